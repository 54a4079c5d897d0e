"""Rotary positions, the E4M3 cache and shared-prefix decode without a GPU: refusals of the C entry
points and of the Python calls (nothing is launched; fake pointers are never touched), the host-side
plans, and pins of their oracle."""
import math

import numpy as np
import pytest

import oracle
from oracle import serving_ref as sv

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_80_b200 import build, _lib
    build.build()
    return _lib.load()


def _rejects(fn, base, changes):
    for where, code in changes:
        bad = list(base)
        for i, v in where.items():
            bad[i] = v
        assert fn(*bad) == code, (where, code)


def test_rotary_rejects_bad_arguments(lib):
    q, k, qo, ko = FAKE, FAKE + (1 << 20), FAKE + (2 << 20), FAKE + (3 << 20)
    # q, k, q_out, k_out, pos, turns, B, N, Hq, Hkv, d, rot, inter, inverse, mag, qbs, qts, kbs, kts, pbs, dt, stream
    base = [q, k, qo, ko, 4 * FAKE, 8 * FAKE, 2, 8, 4, 2, 128, 64, 0, 0, 1.0, 8 * 512, 512, 8 * 256, 256, 8, 1, None]
    _rejects(lib.fa_rotary, base, [
        ({0: 0}, -1), ({1: 0}, -1), ({3: 0}, -1), ({4: 0}, -1), ({5: 0}, -1), ({6: 0}, -1), ({7: 0}, -1), ({8: 0}, -1),
        ({9: -1}, -1), ({11: 0}, -1), ({11: 144}, -1), ({14: math.inf}, -1), ({14: math.nan}, -1), ({15: -8}, -1),
        ({19: 7}, -1), ({18: -8}, -1),
        ({10: 96, 11: 96}, -2), ({10: 256}, -2), ({11: 24}, -2), ({20: 5}, -2), ({6: 65536}, -2), ({8: 65536}, -2),
        ({6: 2, 7: 1 << 30, 19: 0}, -2),
        ({0: q + 8}, -3), ({2: qo + 2}, -3), ({4: FAKE + 2}, -3), ({5: FAKE + 4}, -3), ({16: 516}, -3),
        ({17: 8 * 256 + 4}, -3),
        ({2: q + 16}, -1),                 # overlaps its input without being it
        ({2: q, 16: 768, 15: 8 * 768}, -1),  # in place on a strided tensor
        ({2: k}, -1), ({3: qo}, -1), ({3: q}, -1),
    ])


def test_cache_append_rejects_bad_arguments(lib):
    # k, v, k8, v8, ks, vs, start, counts, B, n, Hkv, Nk_max, d, kbs, kts, vbs, vts, dt, stream
    base = [FAKE] * 7 + [0, 2, 5, 2, 64, 128, 5 * 256, 256, 5 * 256, 256, 1, None]
    _rejects(lib.fa_fp8_cache_append, base, [
        ({0: 0}, -1), ({2: 0}, -1), ({5: 0}, -1), ({6: 0}, -1), ({8: 0}, -1), ({9: 0}, -1), ({10: 0}, -1),
        ({11: 0}, -1), ({13: -8}, -1), ({16: -8}, -1), ({12: 96}, -2), ({17: 2}, -2), ({8: 65536}, -2),
        ({11: (1 << 30) + 1}, -2), ({8: 4, 9: 1 << 30}, -2),
        ({0: FAKE + 8}, -3), ({3: FAKE + 8}, -3), ({4: FAKE + 2}, -3), ({6: FAKE + 2}, -3), ({7: FAKE + 2}, -3),
        ({14: 252}, -3),
    ])


def test_cache_read_rejects_bad_arguments(lib):
    # k8, v8, ks, vs, seqlens, k, v, B, Nk, Hkv, Nk_max, d, dt, stream
    base = [FAKE] * 7 + [2, 5, 2, 64, 128, 1, None]
    _rejects(lib.fa_fp8_cache_read, base, [
        ({0: 0}, -1), ({4: 0}, -1), ({6: 0}, -1), ({7: 0}, -1), ({8: 0}, -1), ({8: 65}, -1), ({9: 0}, -1),
        ({11: 32}, -2), ({12: 9}, -2), ({7: 65536}, -2), ({5: FAKE + 8}, -3), ({4: FAKE + 1}, -3),
    ])


def test_decode_fp8_rejects_bad_arguments(lib):
    # q, k8, v8, ks, vs, seqlens, o, lse, ws, B, Hq, Hkv, Nk_max, d, scale, dt, stream
    base = [FAKE] * 9 + [200, 32, 8, 1024, 128, 0.1, 1, None]
    _rejects(lib.fa_decode_fp8, base, [
        ({0: 0}, -1), ({3: 0}, -1), ({8: 0}, -1), ({10: 33}, -1), ({9: 0}, -1), ({12: 0}, -1),
        ({14: -0.1}, -1), ({14: math.inf}, -1), ({14: math.nan}, -1),
        ({10: 64, 11: 2}, -2), ({13: 96}, -2), ({15: 3}, -2), ({9: 65536}, -2), ({12: (1 << 30) + 1}, -2),
        ({1: FAKE + 8}, -3), ({4: FAKE + 2}, -3), ({5: FAKE + 2}, -3), ({7: FAKE + 2}, -3), ({8: FAKE + 8}, -3),
    ])


def test_decode_shared_prefix_rejects_bad_arguments(lib):
    # q, kp, vp, kc, vc, ks, vs, seqlens, o, lse, ws, B, Hq, Hkv, Np, Nk_max, d, scale, psplits, dt, stream
    base = [FAKE] * 5 + [0, 0] + [FAKE] * 4 + [2, 32, 8, 1000, 1024, 128, 0.1, 4, 1, None]
    _rejects(lib.fa_decode_shared_prefix, base, [
        ({0: 0}, -1), ({1: 0}, -1), ({4: 0}, -1), ({10: 0}, -1), ({5: FAKE}, -1), ({6: FAKE}, -1), ({12: 33}, -1),
        ({14: 0}, -1), ({15: 0}, -1), ({18: 0}, -1), ({18: 9}, -1), ({17: -1.0}, -1),
        ({14: 1200, 18: 9}, -1),  # nine splits of two tiles: the last four would be empty
        ({12: 64, 13: 2}, -2), ({16: 96}, -2), ({19: 2}, -2), ({14: (1 << 30) + 1}, -2),
        ({2: FAKE + 8}, -3), ({7: FAKE + 2}, -3), ({5: FAKE + 2, 6: FAKE}, -3), ({10: FAKE + 4}, -3),
    ])


def test_split_plans_are_accepted_shapes(lib):
    from exact_io_aware_80_b200 import _lib
    for B, Hkv, G in ((1, 1, 1), (4, 2, 4), (64, 8, 4), (250, 8, 4), (33, 3, 7), (9, 16, 16)):
        for N in (1, 64, 127, 128, 129, 513, 4096, 12345, 100000):
            for Nk, fp8 in ((1, 0), (1000, 1), (30000, 0)):
                s = _lib.fa_decode_prefix_splits(B, Hkv * G, Hkv, N, Nk, 128, fp8, 148)
                chunk = -(-(-(-N // s)) // 128) * 128
                assert 1 <= s <= -(-N // 128) and (s - 1) * chunk < N
    ws = _lib.fa_decode_fp8_workspace_bytes
    assert ws(2, 8, 2, 10000, 0, 128) >= (2 * 2 + 1024) * 4 * 129 * 4 + 2 * 8
    assert ws(2, 8, 2, 10000, 3, 64) - ws(2, 8, 2, 10000, 0, 64) >= 2 * 8 * 3 * 65 * 4
    assert ws(2, 8, 2, 1000, 0, 128) == 0 and ws(2, 8, 2, 1000, 1, 128) > 0  # a small batch alone needs none
    assert ws(2, 8, 3, 10000, 0, 64) == 0 and ws(0, 8, 2, 10000, 0, 64) == 0 and ws(2, 8, 2, 10000, -1, 64) == 0


# ---------------------------------------------------------------------------
# Python calls
# ---------------------------------------------------------------------------
def test_python_calls_refuse_cpu_tensors_and_bad_metadata():
    torch = pytest.importorskip("torch")
    import exact_io_aware_80_b200 as fa
    q = torch.zeros(2, 8, 4, 64, dtype=torch.float16)
    pos = torch.zeros(2, 8, dtype=torch.int32)
    table = fa.rotary_table(64, device="cpu")
    with pytest.raises(ValueError):
        fa.rotary_fwd(q, q, pos, table)
    with pytest.raises(TypeError):
        fa.rotary_fwd(q.float(), None, pos, table)
    codes, scales = torch.zeros(2, 16, 2, 64, dtype=torch.uint8), torch.ones(2, 2, 16)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fp8_cache_append(q, q, codes, codes, scales, scales, lens)
    with pytest.raises(ValueError):
        fa.fp8_cache_read(codes, codes, scales, scales, lens)
    with pytest.raises(ValueError):
        fa.decode_fp8(q[:, :1], codes, codes, scales, scales, lens)
    with pytest.raises(ValueError):
        fa.decode_shared_prefix(q[:, :1], q[:1], q[:1], q, q, lens)


def test_python_decode_calls_leave_bad_sizes_to_the_library(lib, monkeypatch):
    """Sizes for which no workspace is planned reach the C entry, whose refusal is the error raised (host
    tensors in place of device ones: validation fails before any of them is touched)."""
    torch = pytest.importorskip("torch")
    import exact_io_aware_80_b200 as fa
    from exact_io_aware_80_b200 import serving
    serving._torch()
    monkeypatch.setattr(serving, "_device", lambda t: t.device)
    monkeypatch.setattr(serving, "_get_device", lambda: None)
    monkeypatch.setattr(serving, "_get_stream", lambda index: None)

    def refused(Hq=4, Hkv=2, Nk=64, Np=10, fp8=True, splits=1, prefix=True):
        q, lens = torch.zeros(2, 1, Hq, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
        codes, scales = torch.zeros(2, Nk, Hkv, 64, dtype=torch.uint8), torch.ones(2, Hkv, Nk)
        kp, own = torch.zeros(1, Np, Hkv, 64, dtype=torch.float16), torch.zeros(2, Nk, Hkv, 64, dtype=torch.float16)
        with pytest.raises(fa.FAError):
            if not prefix:
                fa.decode_fp8(q, codes, codes, scales, scales, lens)
            elif fp8:
                fa.decode_shared_prefix(q, kp, kp, codes, codes, lens, scales, scales, prefix_splits=splits)
            else:
                fa.decode_shared_prefix(q, kp, kp, own, own, lens, prefix_splits=splits)

    for fp8 in (True, False):
        refused(Hq=5, fp8=fp8)
        refused(Nk=0, fp8=fp8)
        refused(Np=0, fp8=fp8)
        for splits in (0, -1, 2, 1 << 30):  # the last: no workspace of 2 TB is asked for first
            refused(fp8=fp8, splits=splits)
        refused(Nk=9000, fp8=fp8, splits=0)
    refused(Hq=5, prefix=False)
    refused(Nk=0, prefix=False)


def test_rotary_table_holds_turns_per_position():
    fa = pytest.importorskip("exact_io_aware_80_b200")
    for kw, ref in ((dict(), dict()), (dict(base=500000.0), dict(base=500000.0)),
                    (dict(scaling="by_parts", factor=8.0, original_len=8192),
                     dict(factor=8.0, original_len=8192)),
                    (dict(scaling="by_parts", factor=4.0, original_len=4096, low_turns=1.0, high_turns=4.0),
                     dict(factor=4.0, original_len=4096, low=1.0, high=4.0))):
        t = fa.rotary_table(64, device="cpu", **kw).numpy().astype(np.uint64)
        f = sv.frequencies(64, **ref)
        # the entry is rounded to 2^-64 of a turn: half of that, and a few fp64 roundings
        assert np.allclose(t.astype(np.float64) * 2.0 ** -64 * 2 * np.pi, f, rtol=1e-14, atol=2.0 ** -65 * 2 * np.pi)
    lin = fa.rotary_table(64, scaling="linear", factor=4.0, device="cpu").numpy().astype(np.uint64).astype(np.float64)
    assert np.allclose(lin * 2.0 ** -64 * 2 * np.pi, sv.frequencies(64) / 4, rtol=1e-14,
                       atol=2.0 ** -65 * 2 * np.pi)
    ntk = fa.rotary_table(64, scaling="ntk", factor=4.0, device="cpu").numpy().astype(np.uint64).astype(np.float64)
    f = ntk * 2.0 ** -64 * 2 * np.pi
    assert np.isclose(f[0], 1.0, rtol=1e-14) and np.isclose(f[-1], sv.frequencies(64)[-1] / 4, rtol=1e-12)
    assert fa.rotary_magnitude(1.0) == 1.0 and np.isclose(fa.rotary_magnitude(8.0), 0.1 * math.log(8) + 1)
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, base=0.0), dict(rot_dim=64, factor=-1.0),
               dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="by_parts", factor=2.0),
               dict(rot_dim=64, scaling="by_parts", factor=2.0, original_len=10, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(ValueError):
            fa.rotary_table(device="cpu", **kw)


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_oracle(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 5, 3, 64)), rng.standard_normal((2, 5, 3, 64))
    f = sv.frequencies(48)
    pos = np.arange(5) + 1000
    a, b = sv.rotary(q, pos, f, interleaved), sv.rotary(k, pos, f, interleaved)
    # scores depend on the distance alone
    a2, b2 = sv.rotary(q, pos + 777, f, interleaved), sv.rotary(k, pos + 777, f, interleaved)
    assert np.allclose(np.einsum("bihc,bjhc->bhij", a, b), np.einsum("bihc,bjhc->bhij", a2, b2), atol=1e-9)
    # orthogonal: the inverse is the transpose, the norm is kept, the tail is not touched
    assert np.allclose(sv.rotary(a, pos, f, interleaved, inverse=True), q, atol=1e-12)
    assert np.allclose(np.sum(a * k), np.sum(q * sv.rotary(k, pos, f, interleaved, inverse=True)), atol=1e-9)
    assert np.array_equal(a[..., 48:], q[..., 48:])
    # pair 0 turns by one radian a position
    i, j = (0, 1) if interleaved else (0, 24)
    assert np.allclose(a[0, 2, 0, i], q[0, 2, 0, i] * np.cos(1002.) - q[0, 2, 0, j] * np.sin(1002.), atol=1e-12)
    assert np.allclose(sv.rotary(q, pos, f, interleaved, magnitude=2.0)[..., :48], 2 * a[..., :48], atol=1e-12)


def test_rotary_gradient_by_differences():
    """d/dx of sum(c * softmax-attention(rotary(q), rotary(k), v)) through the inverse rotation."""
    rng = np.random.default_rng(2)
    q, k, v, c = (rng.standard_normal((1, 4, 2, 64)) for _ in range(4))
    f, pos, m = sv.frequencies(32), np.array([3, 4, 9, 10]), 1.2

    def loss(q, k):
        o, _ = oracle.attention_fwd(sv.rotary(q, pos, f, True, m), sv.rotary(k, pos, f, True, m), v, True, 0.125)
        return float(np.sum(c * o))

    dq, dk, _ = oracle.attention_bwd(sv.rotary(q, pos, f, True, m), sv.rotary(k, pos, f, True, m), v, c, True, 0.125)
    dq, dk = sv.rotary(dq, pos, f, True, m, inverse=True), sv.rotary(dk, pos, f, True, m, inverse=True)
    h = 1e-6
    for x, g, at in ((0, dq, (0, 2, 1, 5)), (0, dq, (0, 3, 0, 40)), (1, dk, (0, 1, 1, 0)), (1, dk, (0, 0, 0, 31))):
        up, dn = [q.copy(), k.copy()], [q.copy(), k.copy()]
        up[x][at] += h
        dn[x][at] -= h
        assert abs((loss(*up) - loss(*dn)) / (2 * h) - g[at]) <= 1e-7


def test_quantized_row_oracle():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((6, 64)) * np.exp(3 * rng.standard_normal((6, 1)))).astype(np.float32)
    x[4] = 0
    codes, s = sv.quantize_rows(x)
    assert s[4] == 1 and not codes[4].any()
    back = sv.cache_values(codes[None, :, None], s[None, None])[0, :, 0]
    # half a step of E4M3 (2^-4 relative, 2^-10 of a scale below its normal range)
    assert np.all(np.abs(back - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s[:, None] * 1.001)
    assert np.allclose(np.abs(back).max(-1), np.abs(x).max(-1), rtol=1e-6)


def test_decode_prefix_oracle_is_attention_over_all_keys():
    rng = np.random.default_rng(4)
    q = rng.standard_normal((3, 1, 4, 64))
    kp, vp = rng.standard_normal((2, 9, 2, 64))
    kc, vc = rng.standard_normal((2, 3, 5, 2, 64))
    lens = [5, 0, 2]
    o, lse = sv.decode_prefix(q, kp, vp, kc, vc, lens, 0.125)
    for b, n in enumerate(lens):
        for h in range(4):
            kk = np.concatenate([kp[:, h // 2], kc[b, :n, h // 2]])
            vv = np.concatenate([vp[:, h // 2], vc[b, :n, h // 2]])
            p = np.exp(0.125 * kk @ q[b, 0, h])
            assert np.allclose(o[b, 0, h], p @ vv / p.sum(), atol=1e-12)
            assert np.isclose(lse[b, h, 0], np.log(p.sum()), atol=1e-12)
    # a bound is a bound: fp16 weights and an fp32 score
    k = np.concatenate([np.broadcast_to(kp, (3, 9, 2, 64)), kc], axis=1)
    v = np.concatenate([np.broadcast_to(vp, (3, 9, 2, 64)), vc], axis=1)
    n = [9 + x for x in lens]
    bo, bl = sv.decode_bounds(q, k, v, n, 0.125, 2.0 ** -11, 2.0 ** -11, 2.0 ** -25)
    for b in range(3):
        for h in range(4):
            x = (k[b, :n[b], h // 2].astype(np.float32) @ q[b, 0, h].astype(np.float32)) * np.float32(0.125)
            p = np.exp((x - x.max()).astype(np.float32))
            w = p.astype(np.float16).astype(np.float64)
            got = (w @ v[b, :n[b], h // 2] / float(p.sum())).astype(np.float16)
            assert np.all(np.abs(got - o[b, 0, h]) <= bo[b, 0, h])
            assert abs(float(x.max()) + math.log(float(p.sum())) - lse[b, h, 0]) <= bl[b, h, 0]
