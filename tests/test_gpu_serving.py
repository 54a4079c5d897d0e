"""Rotary positions, the E4M3 cache, decode over it and shared-prefix decode on the GPU against the
fp64 oracle, within the bounds derived in ``oracle/serving_ref.py``; codes, scales and values read back
are compared bit for bit."""
import math

import numpy as np
import pytest

import oracle
import workloads
from oracle import serving_ref as sv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_io_aware_80_b200 as m
    from exact_io_aware_80_b200 import _lib
    _lib.load()
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def normal(shape, dt, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(*shape, generator=g)).to(dt)


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def done(fa):
    torch.cuda.synchronize()
    assert fa.device_status() == 0


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
ROTARY = [
    # B, N, Hq, Hkv, d, rot, dtype, interleaved, first position
    (1, 1, 1, 1, 64, 16, "fp16", False, 0),
    (2, 5, 4, 2, 64, 64, "bf16", False, 7),
    (2, 5, 4, 2, 64, 48, "bf16", True, 7),
    (3, 7, 7, 1, 128, 128, "fp16", False, 100000),
    (3, 7, 7, 1, 128, 128, "fp16", True, 2000000000),
    (1, 130, 9, 3, 128, 112, "bf16", False, -50),
    (1, 130, 32, 8, 128, 16, "bf16", True, 4000000),
    (65, 1, 20, 5, 128, 64, "fp16", False, 12345),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,dt,inter,first", ROTARY)
@pytest.mark.parametrize("back", [False, True])
def test_rotary(fa, B, N, Hq, Hkv, d, rot, dt, inter, first, back):
    q, k = normal((B, N, Hq, d), DT[dt], 1), normal((B, N, Hkv, d), DT[dt], 2)
    pos = np.array([[first + 3 * b + n for n in range(N)] for b in range(B)], dtype=np.int64)
    m = 1.2079441541679836
    kw = dict(scaling="by_parts", factor=8.0, original_len=8192)
    f = sv.frequencies(rot, factor=8.0, original_len=8192)
    run = fa.rotary_bwd if back else fa.rotary_fwd
    qr, kr = run(q.cuda(), k.cuda(), ints(pos), fa.rotary_table(rot, **kw), inter, m)
    done(fa)
    for x, y in ((q, qr), (k, kr)):
        ref = sv.rotary(f64(x), pos, f, inter, m, inverse=back)
        bound = sv.rotary_bound(f64(x), ref, f, inter, m, torch.finfo(DT[dt]).eps, float(np.abs(pos).max()))
        assert np.all(np.abs(f64(y) - ref) <= bound)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


def test_rotary_takes_slices_shared_positions_and_in_place(fa):
    B, N, Hq, Hkv, d = 2, 37, 8, 2, 128
    packed = normal((B, N, Hq + 2 * Hkv, d), torch.bfloat16, 3).cuda()
    q, k, _ = packed.split([Hq, Hkv, Hkv], dim=2)
    table = fa.rotary_table(d)
    pos = ints(list(range(500, 500 + N)))
    a, b = fa.rotary_fwd(q, k, pos, table)
    before = packed.clone()
    qc, kc = q.contiguous(), k.contiguous()
    a2, b2 = fa.rotary_fwd(qc, kc, pos.expand(B, N).contiguous(), table)
    assert torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(packed, before)
    ip = fa.rotary_fwd(qc, kc, pos, table, q_out=qc, k_out=kc)
    assert ip[0] is qc and ip[1] is kc and torch.equal(qc, a) and torch.equal(kc, b)
    only, none = fa.rotary_fwd(q, None, pos, table)
    assert none is None and torch.equal(only, a)
    # a gradient that is one row broadcast over the tokens
    g = normal((1, 1, Hq, d), torch.bfloat16, 4).cuda().expand(B, N, Hq, d)
    assert torch.equal(fa.rotary_bwd(g, None, pos, table)[0], fa.rotary_bwd(g.contiguous(), None, pos, table)[0])
    done(fa)


def test_rotary_refuses_what_it_cannot_read(fa):
    q = torch.zeros(2, 4, 4, 64, device="cuda", dtype=torch.float16)
    pos, table = torch.zeros(2, 4, device="cuda", dtype=torch.int32), fa.rotary_table(64)
    with pytest.raises(ValueError):  # heads not contiguous
        fa.rotary_fwd(q.transpose(1, 2), None, pos, table)
    with pytest.raises(TypeError):
        fa.rotary_fwd(q, None, pos.long(), table)
    with pytest.raises(ValueError):
        fa.rotary_fwd(q, None, pos[:, :3], table)
    with pytest.raises(TypeError):
        fa.rotary_fwd(q, q.bfloat16(), pos, table)
    with pytest.raises(fa.FAError):  # table wider than the head
        fa.rotary_fwd(q, None, pos, fa.rotary_table(128))
    with pytest.raises(fa.FAError):
        fa.rotary_fwd(q, None, pos, fa.rotary_table(24))
    with pytest.raises(fa.FAError):  # output over the other input
        k = q.clone()
        fa.rotary_fwd(q, k, pos, table, q_out=k)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_in_a_training_step(fa, inter):
    """rotary_fwd -> attention_fwd -> attention_bwd -> rotary_bwd against the oracle's chain rule."""
    B, N, Hq, Hkv, d, rot = 1, 200, 4, 2, 128, 64
    q, k, v, do = workloads.make_inputs(B, Hq, Hkv, N, N, d, torch.bfloat16, seed_base=5, with_do=True)
    table, pos = fa.rotary_table(rot), ints(list(range(N)))
    qr, kr = fa.rotary_fwd(q.cuda(), k.cuda(), pos, table, inter)
    o, lse = fa.attention_fwd(qr, kr, v.cuda(), True)
    dq, dk, dv = fa.attention_bwd(qr, kr, v.cuda(), o, do.cuda(), lse, True)
    dq, dk = fa.rotary_bwd(dq, dk, pos, table, inter)
    done(fa)
    f, p = sv.frequencies(rot), np.arange(N)
    s = 1 / math.sqrt(d)
    rq, rk = sv.rotary(f64(q), p, f, inter), sv.rotary(f64(k), p, f, inter)
    O, _ = oracle.attention_fwd(rq, rk, f64(v), True, s)
    DQ, DK, DV = oracle.attention_bwd(rq, rk, f64(v), f64(do), True, s)
    DQ, DK = sv.rotary(DQ, p, f, inter, inverse=True), sv.rotary(DK, p, f, inter, inverse=True)
    # as for attention alone (1e-2, 2e-2), whose 16-bit operands here also carry one rounding of q and k
    assert np.abs(f64(o) - O).max() <= 2e-2
    for g, G in ((dq, DQ), (dk, DK), (dv, DV)):
        assert np.linalg.norm(f64(g) - G) / np.linalg.norm(G) <= 2e-2


# ---------------------------------------------------------------------------
# the E4M3 cache
# ---------------------------------------------------------------------------
def empty_cache(B, N, H, d, seed=11):
    """A cache full of arbitrary bytes, NaN codes and NaN scales among them."""
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (B, N, H, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.full((B, H, N), float("nan")).cuda() for _ in range(2)]
    return codes + scales


APPEND = [
    # B, n, Hkv, d, Nk_max, dtype, start, counts
    (1, 1, 1, 64, 1, "bf16", [0], None),
    (3, 1, 2, 128, 50, "fp16", [0, 49, 17], None),
    (4, 33, 3, 64, 40, "bf16", [0, 5, 7, 3], [33, 0, 1, 20]),
    (2, 70, 8, 128, 100, "fp16", [30, 0], [70, 69]),
    (3, 9, 5, 128, 12, "bf16", [-4, 8, 12], [9, 99, -3]),  # partly outside the cache, counts clamped
    (3, 1700, 8, 64, 2000, "fp16", [250, 0, 1999], [1700, 333, 1]),  # enough rows to take K and V together
    (2, 1300, 8, 128, 1400, "bf16", [-7, 101], None),
]


@pytest.mark.parametrize("B,n,H,d,Nk,dt,start,counts", APPEND)
def test_append_and_read(fa, B, n, H, d, Nk, dt, start, counts):
    k, v = normal((B, n, H, d), DT[dt], 21), normal((B, n, H, d), DT[dt], 22, size=300.0)
    k[:, 0, 0] = 0  # a row of zeros
    v[0, 0, 0, 1:] = -0.0  # a single value among negative zeros, whose sign a code keeps
    k[-1, -1, -1] *= 1e-6  # fp16: values below its normal range
    cache = empty_cache(B, Nk, H, d)
    want = [c.cpu().numpy().copy() for c in cache]
    fa.fp8_cache_append(k.cuda(), v.cuda(), *cache, ints(start), None if counts is None else ints(counts))
    done(fa)
    for i, x in enumerate((k, v)):
        codes, scales = sv.quantize_rows(x.float().numpy())
        for b in range(B):
            for r in range(max(0, min(n, counts[b])) if counts else n):
                t = start[b] + r
                if 0 <= t < Nk:
                    want[i][b, t] = codes[b, r]
                    want[2 + i][b, :, t] = scales[b, r]
    for got, ref in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True)
    # read back what is there: rows past a length are zeros, whatever the cache holds
    lens = [max(0, min(Nk, start[b] + (n if counts is None else min(counts[b], n)))) for b in range(B)]
    lens = [x if start[b] >= 0 else 0 for b, x in enumerate(lens)]
    for b in range(B):  # rows in front of `start` hold arbitrary bytes: give them scales
        want[2][b, :, :start[b] if start[b] > 0 else 0] = 0.5
        want[3][b, :, :start[b] if start[b] > 0 else 0] = 3.0
    cache[2].copy_(torch.from_numpy(want[2]))
    cache[3].copy_(torch.from_numpy(want[3]))
    for rows in (Nk, max(1, Nk - 3)):
        for out in (torch.bfloat16, torch.float16):
            got = fa.fp8_cache_read(*cache, ints(lens), rows, out)
            done(fa)
            for i, y in enumerate(got):
                c8 = torch.from_numpy(want[i]).view(torch.float8_e4m3fn).float()[:, :rows]
                ref = c8 * torch.from_numpy(want[2 + i]).transpose(1, 2)[:, :rows].unsqueeze(-1)
                live = (torch.arange(rows)[None] < torch.tensor(lens)[:, None])[..., None, None]
                ref = torch.where(live, ref, torch.zeros(())).to(out)
                assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(ref, nan=7.0))


def test_append_takes_slices_and_marks_rows_that_are_not_finite(fa):
    B, n, H, d, Nk = 2, 6, 3, 128, 8
    packed = normal((B, n, 4 + 2 * H, d), torch.bfloat16, 31)
    packed[0, 1, 4, 5] = float("nan")
    packed[1, 2, 4 + H, 7] = float("inf")
    dev = packed.cuda()
    _, k, v = dev.split([4, H, H], dim=2)
    a, b = empty_cache(B, Nk, H, d), empty_cache(B, Nk, H, d)
    fa.fp8_cache_append(k, v, *a, ints([0, 2]))
    fa.fp8_cache_append(k.contiguous(), v.contiguous(), *b, ints([0, 2]))
    for x, y in zip(a, b):
        assert torch.equal(torch.nan_to_num(x.float(), nan=-1.0), torch.nan_to_num(y.float(), nan=-1.0))
    kr, vr = fa.fp8_cache_read(*a, ints([6, 8]))
    done(fa)
    assert kr[0, 1, 0].isnan().all() and vr[1, 4, 0].isnan().all()
    assert torch.isfinite(kr[0, :6]).sum() == 6 * H * d - d and torch.isfinite(vr[1, 2:8]).sum() == 6 * H * d - d


# ---------------------------------------------------------------------------
# decode over the E4M3 cache
# ---------------------------------------------------------------------------
def filled_cache(fa, B, N, H, d, lens, seed, spread=0.0):
    """An E4M3 cache of random rows (sizes e^(spread N(0,1)) per token and head), NaN past each length."""
    cache = empty_cache(B, N, H, d, seed)
    g = torch.Generator().manual_seed(seed + 1)
    for i in range(2):
        x = torch.randn(B, N, H, d, generator=g) * torch.exp(spread * torch.randn(B, N, H, 1, generator=g))
        codes, scales = sv.quantize_rows(x.numpy())
        for b, n in enumerate(lens):
            cache[i][b, :n] = torch.from_numpy(codes[b, :n]).cuda()
            cache[2 + i][b, :, :n] = torch.from_numpy(scales[b, :n].T.copy()).cuda()
            cache[i][b, n:] = 0x7F  # NaN codes
    k, v = (sv.cache_values(np.where(np.isnan(c.cpu().numpy()).transpose(0, 2, 1)[..., None], 0, x.cpu().numpy()),
                            np.nan_to_num(c.cpu().numpy(), nan=1.0)) for x, c in zip(cache[:2], cache[2:]))
    return cache, k, v


def check_decode(q, k, v, lens, scale, o, lse, half_step, floor):
    O, L = oracle.decode(f64(q), k, v, lens, scale)
    bo, bl = sv.decode_bounds(f64(q), k, v, lens, scale, half_step, torch.finfo(q.dtype).eps / 2, floor)
    got = f64(o)
    assert np.all(np.abs(got - O) <= bo), float(np.max(np.abs(got - O) / np.maximum(bo, 1e-30)))
    gl = lse.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        if n == 0:
            assert np.all(got[b] == 0) and np.all(np.isneginf(gl[b]))
        else:
            assert np.all(np.abs(gl[b] - L[b]) <= bl[b])


# weights times V's scale in fp16: 2^-11, and 2^-39 of the largest scale (not of the contribution)
F8_STEP, F8_FLOOR = 2.0 ** -11, 2.0 ** -25

DECODE = [
    # B, Hq, Hkv, N, d, dtype, lens
    (1, 1, 1, 1, 64, "fp16", [1]),
    (1, 4, 4, 1, 128, "bf16", [1]),
    (2, 16, 1, 65, 128, "bf16", [65, 64]),
    (3, 14, 2, 200, 64, "bf16", [200, 0, 63]),
    (3, 14, 2, 200, 64, "fp16", [0, 0, 129]),
    (4, 8, 8, 1000, 128, "fp16", [1000, 1, 0, 513]),
    (4, 8, 2, 1000, 128, "bf16", [0, 1000, 128, 127]),
    (2, 32, 8, 4099, 128, "bf16", [4099, 2050]),
    (5, 3, 1, 777, 64, "bf16", [777, 64, 65, 128, 600]),
    (1, 4, 1, 9000, 64, "fp16", [8999]),                       # one sequence over many CTAs
    (300, 2, 2, 40, 64, "bf16", [b % 41 for b in range(300)]),  # many sequences to a CTA, more than threads
    (140, 3, 3, 300, 128, "fp16", [(61 * b) % 301 if b % 3 else 0 for b in range(140)]),
    (3, 5, 5, 70, 64, "bf16", [0, 0, 0]),
    # too many keys or sequences for one cluster each
    (1, 16, 1, 9000, 128, "fp16", [8500]),
    (2, 6, 3, 5000, 128, "bf16", [4999, 17]),
    (3, 4, 2, 8200, 64, "bf16", [0, 8200, 130]),
    (90, 10, 5, 140, 64, "fp16", [(37 * b) % 141 for b in range(90)]),
    # more sequences and KV heads than resident clusters: several sequences to a CTA, whole or in part
    (300, 6, 3, 40, 64, "bf16", [b % 41 for b in range(300)]),
    (140, 5, 5, 300, 128, "fp16", [(61 * b) % 301 if b % 3 else 0 for b in range(140)]),
    (400, 2, 2, 130, 64, "fp16", [(b * b) % 131 if b % 50 else 0 for b in range(400)]),
    (57, 72, 8, 150, 128, "bf16", [(37 * b) % 151 for b in range(57)]),
    (250, 2, 2, 700, 128, "bf16", [700 if b == 100 else (b * 7) % 130 for b in range(250)]),
]


@pytest.mark.parametrize("B,Hq,Hkv,N,d,dt,lens", DECODE)
def test_decode_fp8(fa, B, Hq, Hkv, N, d, dt, lens):
    q = normal((B, 1, Hq, d), DT[dt], 41)
    cache, k, v = filled_cache(fa, B, N, Hkv, d, lens, 42, spread=0.5)
    o, lse = fa.decode_fp8(q.cuda(), *cache, ints(lens))
    done(fa)
    check_decode(q, k, v, lens, 1 / math.sqrt(d), o, lse, F8_STEP, F8_FLOOR)


@pytest.mark.parametrize("dt,size,scale", [("bf16", 1e20, 1e-21), ("bf16", 1e-20, 1e19), ("fp16", 2000.0, 1e-4),
                                           ("bf16", 1.0, 0.0), ("bf16", 1.0, 2.0)])
def test_decode_fp8_query_sizes_and_scales(fa, dt, size, scale):
    B, Hq, Hkv, N, d, lens = 2, 8, 2, 300, 128, [300, 211]
    q = normal((B, 1, Hq, d), DT[dt], 43, size=size)
    cache, k, v = filled_cache(fa, B, N, Hkv, d, lens, 44, spread=1.0)
    o, lse = fa.decode_fp8(q.cuda(), *cache, ints(lens), scale=scale)
    done(fa)
    check_decode(q, k, v, lens, scale, o, lse, F8_STEP, F8_FLOOR)


def test_decode_fp8_with_scales_far_apart(fa):
    """V rows from 2^-60 to 2^60 in size, growing, falling and mixed along the keys."""
    B, Hq, Hkv, N, d, lens = 3, 4, 1, 256, 64, [256, 256, 256]
    q = normal((B, 1, Hq, d), torch.bfloat16, 45)
    cache, k, v = filled_cache(fa, B, N, Hkv, d, lens, 46)
    e = np.stack([np.linspace(-60, 60, N).round(), np.linspace(60, -60, N).round(),
                  np.random.default_rng(5).integers(-60, 61, N)])[:, None]
    cache[3].mul_(torch.from_numpy(2.0 ** e).float().cuda())
    v = v * (2.0 ** e).transpose(0, 2, 1)[..., None]
    o, lse = fa.decode_fp8(q.cuda(), *cache, ints(lens))
    done(fa)
    check_decode(q, k, v, lens, 1 / 8, o, lse, F8_STEP, F8_FLOOR)


def test_decode_fp8_passes_on_nan(fa):
    B, Hq, Hkv, N, d = 2, 4, 2, 100, 64
    q = normal((B, 1, Hq, d), torch.float16, 47)
    cache, _, _ = filled_cache(fa, B, N, Hkv, d, [100, 100], 48)
    cache[2][0, 1, 70] = float("nan")  # one key's scale
    cache[3][1, 0, 3] = float("nan")   # one value's
    o, lse = fa.decode_fp8(q.cuda(), *cache, ints([100, 100]))
    done(fa)
    assert o[0, 0, 2:].isnan().all() and lse[0, 2:].isnan().all() and torch.isfinite(o[0, 0, :2]).all()
    assert o[1, 0, :2].isnan().all() and torch.isfinite(lse[1]).all() and torch.isfinite(o[1, 0, 2:]).all()
    q[0, 0, 1] = float("nan")
    o, lse = fa.decode_fp8(q.cuda(), *cache, ints([100, 100]))
    assert o[0, 0, 1].isnan().all() and lse[0, 1].isnan().all() and torch.isfinite(o[0, 0, 0]).all()
    # a NaN past the length does no harm
    o, _ = fa.decode_fp8(q.cuda(), *cache, ints([70, 3]))
    done(fa)
    assert torch.isfinite(o[0, 0, 2:]).all() and torch.isfinite(o[1]).all()


# ---------------------------------------------------------------------------
# decode behind a shared prefix
# ---------------------------------------------------------------------------
PREFIX = [
    # B, Hq, Hkv, Np, Nk_max, d, dtype, fp8, prefix splits
    (1, 1, 1, 1, 1, 64, "fp16", False, None),
    (1, 4, 2, 127, 3, 128, "bf16", True, None),
    (3, 6, 2, 128, 70, 64, "bf16", False, None),      # G = 3: 42 sequences a tile, 126 rows
    (4, 8, 2, 513, 64, 64, "fp16", False, None),
    (2, 32, 2, 129, 65, 128, "bf16", True, 1),           # G = 16
    (32, 8, 2, 300, 40, 128, "fp16", True, 2),        # 128 rows: one full tile
    (33, 8, 2, 300, 40, 128, "bf16", False, None),    # 132 rows: the second tile holds one sequence
    (64, 4, 1, 1000, 20, 64, "bf16", True, 3),           # 256 rows
    (65, 8, 2, 640, 20, 128, "bf16", False, 5),          # 260 rows: a second row block
    (53, 5, 1, 400, 33, 64, "fp16", True, None),      # G = 5: 25 sequences a tile
    (150, 1, 1, 257, 5, 128, "bf16", False, None),    # G = 1
    (120, 8, 4, 600, 130, 64, "fp16", True, 3),       # the caches merged apart
    (60, 8, 8, 200, 30, 128, "bf16", False, None),
    (2, 8, 2, 1500, 30, 64, "bf16", True, 12),        # many prefix splits
    (67, 9, 3, 1100, 40, 64, "fp16", False, 9),       # 603 rows of nine splits and more
    (40, 14, 2, 260, 9, 64, "bf16", False, 1),        # G = 7: 18 sequences a tile, 126 rows
]


def prefix_case(fa, B, Hq, Hkv, Np, Nk, d, dt, fp8, lens, seed):
    q = normal((B, 1, Hq, d), DT[dt], seed)
    kp, vp = normal((1, Np, Hkv, d), DT[dt], seed + 1), normal((1, Np, Hkv, d), DT[dt], seed + 2)
    if fp8:
        (k8, v8, ks, vs), k, v = filled_cache(fa, B, Nk, Hkv, d, lens, seed + 3)
        args = (q.cuda(), kp.cuda(), vp.cuda(), k8, v8, ints(lens), ks, vs)
    else:
        kc, vc = normal((B, Nk, Hkv, d), DT[dt], seed + 4), normal((B, Nk, Hkv, d), DT[dt], seed + 5)
        for b, n in enumerate(lens):
            kc[b, n:] = float("nan")
            vc[b, n:] = float("nan")
        args = (q.cuda(), kp.cuda(), vp.cuda(), kc.cuda(), vc.cuda(), ints(lens))
        k, v = np.nan_to_num(f64(kc)), np.nan_to_num(f64(vc))
    k = np.concatenate([np.broadcast_to(f64(kp), (B,) + kp.shape[1:]), k], axis=1)
    v = np.concatenate([np.broadcast_to(f64(vp), (B,) + vp.shape[1:]), v], axis=1)
    return q, args, k, v


@pytest.mark.parametrize("B,Hq,Hkv,Np,Nk,d,dt,fp8,ps", PREFIX)
def test_decode_shared_prefix(fa, B, Hq, Hkv, Np, Nk, d, dt, fp8, ps):
    lens = [(7 * b + Nk) % (Nk + 1) for b in range(B)]  # 0 among them
    q, args, k, v = prefix_case(fa, B, Hq, Hkv, Np, Nk, d, dt, fp8, lens, 51)
    o, lse = fa.decode_shared_prefix(*args, prefix_splits=ps)
    done(fa)
    # weights in q's type (half a step of it, 2^-25 absolute in fp16) or in fp16
    check_decode(q, k, v, [Np + n for n in lens], 1 / math.sqrt(d), o, lse,
                 max(F8_STEP, torch.finfo(DT[dt]).eps / 2), F8_FLOOR)


# (q's type and size, scale): scale 0 weighs every key alike, keys past the prefix's end not at all
@pytest.mark.parametrize("dt,size,scale", [("bf16", 1.0, 0.0), ("fp16", 1.0, 0.0), ("bf16", 1.0, 2.0),
                                           ("fp16", 2000.0, 1e-4), ("bf16", 1e20, 1e-21), ("bf16", 1e-20, 1e19)])
@pytest.mark.parametrize("Np", [1, 65, 128, 200, 300])
@pytest.mark.parametrize("B", [3, 70])  # one query tile; two of them, the second row block's last one empty
def test_decode_shared_prefix_query_sizes_and_scales(fa, B, Np, dt, size, scale):
    Hq, Hkv, Nk, d = 4, 1, 5, 64
    lens = [b % (Nk + 1) for b in range(B)]
    _, args, k, v = prefix_case(fa, B, Hq, Hkv, Np, Nk, d, dt, False, lens, 57)
    q = normal((B, 1, Hq, d), DT[dt], 58, size=size)
    o, lse = fa.decode_shared_prefix(q.cuda(), *args[1:], scale=scale)
    done(fa)
    check_decode(q, k, v, [Np + n for n in lens], scale, o, lse, max(F8_STEP, torch.finfo(DT[dt]).eps / 2), F8_FLOOR)


@pytest.mark.parametrize("B", [4, 40, 140])  # few rows; one query tile; two
def test_decode_shared_prefix_keeps_a_long_faint_tail(fa, B):
    """One dominant key whose value is 0 and 20000 keys 17.4 to 17.8 nats (25.1 to 25.7 powers of two) below
    it, which together are all of O: 4e-4 of their values.  A weight is kept in fp16 in units in which the
    largest is 2^7 to 2^15, so it is off by at most half of 2^-24 of that unit, 2^-32 of the largest."""
    Np, d = 20001, 64
    g = torch.Generator().manual_seed(59)
    kp, vp = torch.zeros(1, Np, 1, d), 0.5 + torch.rand(1, Np, 1, d, generator=g)
    kp[..., 0] = 2.2 + 0.4 * torch.rand(1, Np, 1, generator=g)
    kp[0, 0, 0, 0], vp[0, 0] = 20.0, 0.0
    q = torch.zeros(B, 1, 1, d)
    q[..., 0] = 1.0
    q, kp, vp = q.half(), kp.half(), vp.half()
    own = torch.full((B, 1, 1, d), float("nan"), dtype=torch.float16).cuda()
    o, lse = fa.decode_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), own, own, ints([0] * B), prefix_splits=1, scale=1.0)
    done(fa)
    assert torch.equal(o, o[:1].expand_as(o)) and torch.equal(lse, lse[:1].expand_as(lse))  # equal queries
    check_decode(q[:1], f64(kp), f64(vp), [Np], 1.0, o[:1], lse[:1], F8_STEP, 2.0 ** -32)


@pytest.mark.parametrize("B", [2, 40])
def test_decode_shared_prefix_passes_on_nan(fa, B):
    """One bad key of the prefix, in every column of a tile's exponentials, makes its KV head's rows NaN
    and no other's; so does a query row, for itself; so does a +inf score."""
    Hq, Hkv, Np, Nk, d = 8, 2, 200, 4, 64
    lens = [b % 5 for b in range(B)]
    q, args, _, _ = prefix_case(fa, B, Hq, Hkv, Np, Nk, d, "bf16", False, lens, 65)
    for key in list(range(0, 16)) + [127, 128, 199]:
        kp = args[1].clone()
        kp[0, key, 1, 3] = float("nan") if key % 2 else float("inf")
        qq = args[0].clone()
        qq[..., 3] = qq[..., 3].abs() + 0.5
        o, lse = fa.decode_shared_prefix(qq, kp, *args[2:])
        assert o[:, 0, 4:].isnan().all() and torch.isfinite(o[:, 0, :4]).all() and torch.isfinite(lse[:, :4]).all()
    qq = args[0].clone()
    qq[B - 1, 0, 2, 7] = float("nan")
    o, lse = fa.decode_shared_prefix(qq, *args[1:])
    bad = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
    bad[B - 1, 2] = True
    assert torch.equal(o[:, 0].isnan().all(-1), bad) and torch.equal(o[:, 0].isnan().any(-1), bad)
    assert torch.equal(lse[:, :, 0].isnan(), bad)
    done(fa)


def test_decode_shared_prefix_with_more_work_than_sms(fa):
    """Work tiles beyond one per SM: 5 row blocks x 8 KV heads x 8 splits, so a CTA takes several."""
    B, Hq, Hkv, Np, Nk, d = 300, 32, 8, 1024, 4, 64
    lens = [b % 5 for b in range(B)]
    q, args, k, v = prefix_case(fa, B, Hq, Hkv, Np, Nk, d, "fp16", False, lens, 61)
    o, lse = fa.decode_shared_prefix(*args, prefix_splits=8)
    o2, lse2 = fa.decode_shared_prefix(*args, prefix_splits=8)
    done(fa)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    some = [0, 31, 32, 63, 64, 150, 255, 256, 299]
    check_decode(q[some], k[some], v[some], [Np + lens[b] for b in some], 1 / 8, o[some], lse[some], F8_STEP, F8_FLOOR)


def test_decode_shared_prefix_equals_decode_over_the_joined_cache(fa):
    """The prefix copied in front of every cache and decoded by the split-KV path: the same up to rounding."""
    B, Hq, Hkv, Np, Nk, d = 7, 8, 2, 700, 100, 128
    lens = [100, 0, 3, 64, 65, 99, 1]
    q, args, k, v = prefix_case(fa, B, Hq, Hkv, Np, Nk, d, "bf16", False, lens, 71)
    o, lse = fa.decode_shared_prefix(*args)
    joined = [torch.cat((args[1 + i].expand(B, -1, -1, -1), torch.nan_to_num(args[3 + i])), 1).contiguous()
              for i in range(2)]
    o2, lse2 = fa.decode(args[0], *joined, ints([Np + n for n in lens]))
    done(fa)
    # two bf16 results of values below 1: two half steps each of P's rounding and the final one
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * o2.float().abs().max()
    assert (lse - lse2).abs().max() <= 1e-4


def test_decode_refusals(fa):
    B, Hq, Hkv, N, d = 2, 4, 2, 64, 64
    q = normal((B, 1, Hq, d), torch.float16, 81).cuda()
    cache, _, _ = filled_cache(fa, B, N, Hkv, d, [64, 64], 82)
    lens = ints([64, 64])
    kp = normal((1, 10, Hkv, d), torch.float16, 83).cuda()
    with pytest.raises(ValueError):
        fa.decode_fp8(q.expand(B, 2, Hq, d), *cache, lens)
    with pytest.raises(TypeError):
        fa.decode_fp8(q, *cache, lens.long())
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q, kp, kp, cache[0], cache[1], lens, cache[2], cache[3],
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.decode_fp8(q, cache[0], cache[1], cache[2].transpose(1, 2), cache[3], lens)
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q, kp, kp, cache[0], cache[1], lens)
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q, kp.expand(B, 10, Hkv, d), kp, cache[0], cache[1], lens, cache[2], cache[3])
    with pytest.raises(TypeError):
        fa.decode_shared_prefix(q, kp.bfloat16(), kp, cache[0], cache[1], lens, cache[2], cache[3])
    with pytest.raises(fa.FAError):
        fa.decode_fp8(q, *cache, lens, scale=float("inf"))
    with pytest.raises(fa.FAError):
        fa.decode_shared_prefix(q, kp, kp, cache[0], cache[1], lens, cache[2], cache[3], prefix_splits=2)
    done(fa)


# ---------------------------------------------------------------------------
# together, as they are used
# ---------------------------------------------------------------------------
def test_serving_steps_together(fa):
    """A prompt and three decode steps: rotary positions, rows quantised into the cache, attention over
    what was read back (prompt) and over the codes behind a shared prefix (steps); the steps run from one
    captured graph whose lengths and positions advance on the device."""
    B, Hq, Hkv, d, Np, n, Nk = 3, 8, 2, 128, 200, 20, 64
    dt = torch.bfloat16
    table, f = fa.rotary_table(d), sv.frequencies(d)
    kp = sv.rotary(f64(normal((1, Np, Hkv, d), dt, 91)), np.arange(Np), f, False)
    kp, vp = torch.from_numpy(kp).to(dt).cuda(), normal((1, Np, Hkv, d), dt, 92).cuda()
    counts = [20, 7, 0]
    cache = empty_cache(B, Nk, Hkv, d)
    prompt = normal((B, n, Hq + 2 * Hkv, d), dt, 93).cuda()
    q, k, v = prompt.split([Hq, Hkv, Hkv], dim=2)
    _, kr = fa.rotary_fwd(q, k, torch.arange(Np, Np + n, dtype=torch.int32, device="cuda"), table)
    fa.fp8_cache_append(kr, v, *cache, ints([0] * B), ints(counts))
    back = fa.fp8_cache_read(*cache, ints(counts), n)
    want_k, want_v = [np.zeros((B, Nk, Hkv, d)) for _ in range(2)]
    for b, m in enumerate(counts):
        want_k[b, :m] = f64(back[0])[b, :m]
        rel = np.abs(want_k[b, :m] - sv.rotary(f64(k), np.arange(Np, Np + n), f, False)[b, :m])
        # half a step of E4M3 at most, and two 16-bit roundings
        assert rel.max(initial=0) <= (2.0 ** -4 + 2.0 ** -6) * np.abs(want_k).max()

    steps = [normal((B, 1, Hq + 2 * Hkv, d), dt, 94 + i).cuda() for i in range(3)]
    x, lens = torch.empty_like(steps[0]), ints(counts)
    pos = (lens + Np).view(B, 1)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    res = {}

    def step():
        q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
        qr, kr = fa.rotary_fwd(q, k, pos, table)
        fa.fp8_cache_append(kr, v, *cache, lens)
        lens.add_(one)
        pos.add_(1)
        res["q"], res["k"] = qr, kr
        res["o"], res["lse"] = fa.decode_shared_prefix(qr, kp, vp, cache[0], cache[1], lens, cache[2], cache[3])

    side = torch.cuda.Stream()
    saved = [t.clone() for t in cache + [lens, pos]]
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        x.copy_(steps[0])
        step()
    torch.cuda.synchronize()
    for t, s in zip(cache + [lens, pos], saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, s in enumerate(steps):
        x.copy_(s)
        graph.replay()
        done(fa)
        n_now = [c + i + 1 for c in counts]
        assert lens.tolist() == n_now
        K, V = fa.fp8_cache_read(*cache, lens)  # bf16 rounding of the values; the decode uses them unrounded
        vals = [sv.cache_values(np.where(np.arange(Nk)[None, :, None, None] < np.array(n_now)[:, None, None, None],
                                         c.cpu().numpy(), 0), np.nan_to_num(sc.cpu().numpy(), nan=1.0))
                for c, sc in zip(cache[:2], cache[2:])]
        for got, ref in zip((K, V), vals):
            assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref))
        P = [np.concatenate([np.broadcast_to(f64(p), (B, Np, Hkv, d)), c], 1) for p, c in zip((kp, vp), vals)]
        check_decode(res["q"], P[0], P[1], [Np + m for m in n_now], 1 / math.sqrt(d), res["o"], res["lse"],
                     2.0 ** -8, F8_FLOOR)


def test_graphs_that_share_a_workspace_and_other_streams(fa):
    """Two captured decodes that share one workspace, replayed in turn on another stream, equal the
    eager calls bit for bit; so does an eager call on that stream."""
    B, Hq, Hkv, N, d, lens = 4, 8, 2, 500, 128, [500, 3, 0, 257]
    cache, _, _ = filled_cache(fa, B, N, Hkv, d, lens, 101)
    q = [normal((B, 1, Hq, d), torch.bfloat16, 102 + i).cuda() for i in range(2)]
    kp, vp = (normal((1, 333, Hkv, d), torch.bfloat16, 104 + i).cuda() for i in range(2))
    sl = ints(lens)
    P = fa.fa_decode_prefix_splits(B, Hq, Hkv, 333, N, d, True)
    ws = torch.empty(fa.fa_decode_fp8_workspace_bytes(B, Hq, Hkv, N, P, d), dtype=torch.uint8, device="cuda")

    def a():
        return fa.decode_fp8(q[0], *cache, sl, workspace=ws)

    def b():
        return fa.decode_shared_prefix(q[1], kp, vp, cache[0], cache[1], sl, cache[2], cache[3], workspace=ws)

    ref = [tuple(t.clone() for t in f()) for f in (a, b)]
    done(fa)
    graphs = []
    for f in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    ws.fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            for g, _ in graphs:
                g.replay()
        eager = [f() for f in (a, b)]
    done(fa)
    for r, (_, out), e in zip(ref, graphs, eager):
        for x, y, z in zip(r, out, e):
            assert torch.equal(x, y) and torch.equal(x, z)


def test_calls_follow_earlier_and_precede_later_work(fa):
    """A chain of calls over the same buffers, each input produced just before by other kernels and each
    output read just after, with nothing waited for in between, equals the same chain with a wait after
    every step, bit for bit (the kernels start as programmatic dependents)."""
    B, Hq, Hkv, N, d = 24, 8, 2, 300, 64
    table = fa.rotary_table(d)
    kp, vp = (normal((1, 700, Hkv, d), torch.float16, 121 + i).cuda() for i in range(2))
    big = normal((2048, 2048), torch.float16, 123).cuda()
    src = [normal((B, 1, Hq + 2 * Hkv, d), torch.float16, 124 + i).cuda() for i in range(12)]
    long_lens = ints([150 + b for b in range(B)])

    def chain(wait):
        cache = empty_cache(B, N, Hkv, d)
        for c in cache[2:]:
            c.fill_(0.01)
        for c in cache[:2]:
            c.fill_(0x38)
        lens, outs = torch.zeros(B, dtype=torch.int32, device="cuda"), []
        x, q = torch.empty_like(src[0]), torch.empty(B, 1, Hq, d, dtype=torch.float16, device="cuda")
        for i, s in enumerate(src):
            y = big
            for _ in range(3):
                y = (y @ big) * 0.01
            x.copy_(s + 0 * y[0, 0])
            qp, k, v = x.split([Hq, Hkv, Hkv], dim=2)
            pos = (lens + 700).view(B, 1)
            _, kr = fa.rotary_fwd(qp, k, pos, table, q_out=q)
            fa.fp8_cache_append(kr, v, *cache, lens)
            lens += 1
            for f in (lambda: fa.decode_fp8(q, *cache, lens), lambda: fa.decode_fp8(q, *cache, long_lens),
                      lambda: fa.decode_shared_prefix(q, kp, vp, cache[0], cache[1], lens, cache[2], cache[3]),
                      lambda: fa.fp8_cache_read(*cache, lens, 20, torch.float16)):
                o = f()
                outs += [t.clone() for t in o]
                for t in o:
                    t.fill_(7)
                if wait:
                    torch.cuda.synchronize()
            x.zero_()
            q.zero_()
        torch.cuda.synchronize()
        return outs

    ref = chain(True)
    for _ in range(3):
        for a, b in zip(ref, chain(False)):
            assert torch.equal(torch.nan_to_num(a.float(), nan=-3.0), torch.nan_to_num(b.float(), nan=-3.0))
    done(fa)


@pytest.mark.parametrize("B,fp8", [(4, True), (4, False), (90, True), (90, False)])  # a cluster a sequence; a merge of its own
def test_decode_shared_prefix_right_behind_what_it_reads(fa, B, fp8):
    """Rotation of q in place and the rewriting of cache rows that the call before has read, followed by the
    call with nothing in between, equal the same steps with a wait after each, bit for bit."""
    Hq, Hkv, N, Np, d, steps = 8, 2, 150, 300, 64, 40
    table = fa.rotary_table(d)
    kp, vp = (normal((1, Np, Hkv, d), torch.float16, 151 + i).cuda() for i in range(2))
    q0 = normal((B, 1, Hq, d), torch.float16, 153).cuda()
    rows = [normal((B, 1, Hkv, d), torch.float16, 154 + i, size=1.0 + i % 5).cuda() for i in range(2 * steps)]
    at = [ints([(37 * i + 11 * b) % N for b in range(B)]) for i in range(steps)]
    pos, lens = ints([[b] for b in range(B)]), ints([N - b % 3 for b in range(B)])

    def chain(wait):
        cache = empty_cache(B, N, Hkv, d)
        for c, x in zip(cache, (0x38, 0x38, 0.01, 0.01)):
            c.fill_(x)
        plain = [torch.zeros(B, N, Hkv, d, dtype=torch.float16, device="cuda") for _ in range(2)]
        q, outs = q0.clone(), []
        torch.cuda.synchronize()
        for i in range(steps):
            fa.fp8_cache_append(rows[2 * i], rows[2 * i + 1], *cache, at[i])
            if wait:
                torch.cuda.synchronize()
            if not fp8:  # the cache's values as a 16-bit cache
                plain = fa.fp8_cache_read(*cache, lens, N, torch.float16)
            fa.rotary_fwd(q, None, pos, table, q_out=q)
            if wait:
                torch.cuda.synchronize()
            outs += fa.decode_shared_prefix(q, kp, vp, *((cache[0], cache[1], lens, cache[2], cache[3]) if fp8 else
                                                         (*plain, lens)))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    ref = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ref, chain(False)))
    done(fa)


def test_two_threads_on_two_streams(fa):
    """Calls made at once by two threads, each on a stream and tensors of its own, equal those made alone."""
    import threading
    shapes = [(40, 8, 2, 300, 64, torch.float16), (6, 16, 2, 200, 128, torch.bfloat16)]
    table = {d: fa.rotary_table(d) for d in (64, 128)}

    def work(i, outs):
        B, Hq, Hkv, N, d, dt = shapes[i]
        with torch.cuda.stream(streams[i]):
            q, kp, vp = (x.clone() for x in data[i][:3])
            cache = [c.clone() for c in data[i][3]]
            lens = data[i][4].clone()
            for step in range(30):
                qr, kr = fa.rotary_fwd(q, kp[:, step:step + 1].expand(B, 1, Hkv, d), (lens + 400).view(B, 1), table[d])
                fa.fp8_cache_append(kr, kr, *cache, lens)
                lens += 1
                outs += fa.decode_shared_prefix(qr, kp, vp, cache[0], cache[1], lens, cache[2], cache[3])
                outs += fa.decode_fp8(qr, *cache, lens)
            streams[i].synchronize()

    streams = [torch.cuda.Stream() for _ in shapes]
    data = []
    for i, (B, Hq, Hkv, N, d, dt) in enumerate(shapes):
        lens = [(17 * b) % (N - 30) for b in range(B)]
        data.append((normal((B, 1, Hq, d), dt, 161).cuda(), normal((1, 400, Hkv, d), dt, 162 + i).cuda(),
                     normal((1, 400, Hkv, d), dt, 164 + i).cuda(), filled_cache(fa, B, N, Hkv, d, lens, 166 + i)[0], ints(lens)))
    alone, both = [[], []], [[], []]
    torch.cuda.synchronize()
    for i in range(2):
        work(i, alone[i])
    threads = [threading.Thread(target=work, args=(i, both[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done(fa)
    for a, b in zip(alone, both):
        assert len(b) == 4 * 30 and all(torch.equal(x, y) for x, y in zip(a, b))


class Guarded:
    """A tensor between two stretches of sentinel bytes."""
    PAD = 64 * 1024

    def __init__(self, shape, dtype, fill=None):
        self.n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        self.buf = torch.full((2 * self.PAD + (self.n + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.PAD:self.PAD + self.n].view(dtype).view(shape)
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        return bool((self.buf[:self.PAD] == 0xA5).all()) and bool((self.buf[self.PAD + self.n:] == 0xA5).all())


@pytest.mark.parametrize("B,Hq,Hkv,N,d,dt", [(3, 6, 2, 133, 64, "fp16"), (2, 16, 1, 70, 128, "bf16"),
                                             (150, 12, 3, 190, 64, "bf16"), (1, 5, 5, 1, 128, "fp16"),
                                             (2, 8, 2, 9000, 64, "fp16")])
def test_everything_stays_inside_its_outputs(fa, B, Hq, Hkv, N, d, dt):
    t = DT[dt]
    q, k, v = (Guarded((B, 3, H, d), t, normal((B, 3, H, d), t, 131 + i).cuda())
               for i, H in enumerate((Hq, Hkv, Hkv)))
    qo, ko = Guarded((B, 3, Hq, d), t), Guarded((B, 3, Hkv, d), t)
    fa.rotary_fwd(q.t, k.t, torch.arange(3, dtype=torch.int32, device="cuda"), fa.rotary_table(32), q_out=qo.t,
                  k_out=ko.t)
    raw = empty_cache(B, N, Hkv, d)
    cache = [Guarded(c.shape, c.dtype, torch.nan_to_num(c, nan=0.5) if c.is_floating_point() else c & 0x77) for c in raw]
    fa.fp8_cache_append(ko.t, v.t, *(c.t for c in cache), ints([N - 1 - b % 3 for b in range(B)]))
    lens = ints([(N - b * 13) % (N + 1) for b in range(B)])
    rows = [Guarded((B, N, Hkv, d), t) for _ in range(2)]
    from exact_io_aware_80_b200 import _lib
    stream = torch.cuda.current_stream().cuda_stream
    code = _lib.FA_BF16 if dt == "bf16" else _lib.FA_FP16
    _lib.fa_fp8_cache_read(*(c.t.data_ptr() for c in cache), lens.data_ptr(), rows[0].t.data_ptr(),
                           rows[1].t.data_ptr(), B, N, Hkv, N, d, code, stream)
    q1 = Guarded((B, 1, Hq, d), t, qo.t[:, :1])
    kp = Guarded((1, 333, Hkv, d), t, normal((1, 333, Hkv, d), t, 141).cuda())
    everything = [q, k, v, qo, ko, q1, kp] + cache + rows
    for splits in (0, 1, 3):
        need = fa.fa_decode_fp8_workspace_bytes(B, Hq, Hkv, N, splits, d)
        ws = Guarded((max(need, 16),), torch.uint8)
        o, lse = Guarded((B, 1, Hq, d), t), Guarded((B, Hq, 1), torch.float32)
        if splits == 0:
            fa.decode_fp8(q1.t, *(c.t for c in cache), lens, workspace=ws.t, out=o.t, lse=lse.t)
        else:
            fa.decode_shared_prefix(q1.t, kp.t, kp.t, cache[0].t, cache[1].t, lens, cache[2].t, cache[3].t,
                                    prefix_splits=splits, workspace=ws.t, out=o.t, lse=lse.t)
            o16, l16 = Guarded((B, 1, Hq, d), t), Guarded((B, Hq, 1), torch.float32)
            fa.decode_shared_prefix(q1.t, kp.t, kp.t, rows[0].t, rows[1].t, lens, prefix_splits=splits,
                                    workspace=ws.t, out=o16.t, lse=l16.t)
            everything += [o16, l16]
        everything += [ws, o, lse]
    done(fa)
    assert all(g.intact() for g in everything)
    assert all(torch.isfinite(g.t.float()).all() for g in (qo, ko, *rows))


@pytest.mark.slow
def test_decode_fp8_past_two_gigabytes_of_codes(fa):
    """Offsets beyond 2^31: three sequences of 2^20 - 5 keys, 8 heads of 128, sampled heads of the last."""
    B, Hq, Hkv, N, d = 3, 8, 8, (1 << 20) - 5, 128
    g = torch.Generator(device="cuda").manual_seed(111)
    codes = [torch.randint(0, 0x70, (B, N, Hkv, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    for c in codes:
        c.add_(torch.randint(0, 2, (B, N, Hkv, d), generator=g, device="cuda", dtype=torch.uint8) * 128)
    scales = [0.01 * torch.rand(B, Hkv, N, generator=g, device="cuda") + 1e-3 for _ in range(2)]
    q = normal((B, 1, Hq, d), torch.bfloat16, 112)
    lens = [5, 0, N - 3]
    assert codes[0].numel() > 1 << 31
    o, lse = fa.decode_fp8(q.cuda(), *codes, *scales, ints(lens))
    kr, vr = fa.fp8_cache_read(*codes, *scales, ints(lens), 6)
    done(fa)
    assert torch.isfinite(kr).all() and (kr[1] == 0).all() and (vr[0, 5:] == 0).all()
    for h in (0, 7):
        k, v = (sv.cache_values(c[2:, :, h:h + 1].cpu().numpy(), s[2:, h:h + 1].cpu().numpy())
                for c, s in zip(codes, scales))
        check_decode(q[2:, :, h:h + 1], k, v, lens[2:], 1 / math.sqrt(d), o[2:, :, h:h + 1], lse[2:, h:h + 1], F8_STEP,
                     F8_FLOOR)
