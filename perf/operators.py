"""What the serving and rotary operators cost: cases, inputs, their plain forms and their definition in 64 bits.

Six kinds of call:

* ``rotary``: rotary positions applied to (or, with ``back``, taken back from the gradients of) q and k;
* ``append``: new K and V rows quantised to E4M3 with one scale per (token, head) as they enter a cache;
* ``read``: a range of such a cache read back as 16-bit K and V;
* ``decode``: one-token attention over such a cache;
* ``prefix``: one-token attention of a batch whose sequences share one prefix, followed by a ragged
  suffix of each sequence's own, held in 16 bits or in E4M3.

With ``own`` false, ``run`` computes them in elementary torch operations in fp32 (rotary angles in
fp64) and rounds once; with ``own`` true it calls this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a training step's q and k as slices of one packed projection, the GQA training shape
        dict(name="rotary-train", kind="rotary", B=1, N=8192, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaled=False, back=False, packed=True, far=0, dtype="bf16"),
        # its backward pass at the MHA shape: half of each head rotated, in pairs of neighbours, scaled frequencies
        dict(name="rotary-train-back", kind="rotary", B=4, N=2048, Hq=16, Hkv=16, d=128, rot=64, interleaved=True,
             scaled=True, back=True, packed=False, far=0, dtype="fp16"),
        # one new token of each of 64 sequences, far into a long context: what a launch costs
        dict(name="rotary-token", kind="rotary", B=64, N=1, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaled=True, back=False, packed=True, far=1000000, dtype="bf16"),
        # one new token of each of 64 sequences enters the cache
        dict(name="append-token", kind="append", B=64, n=1, Hkv=8, d=128, Nk=4096, ragged=False, dtype="bf16"),
        # three padded prompts of odd lengths enter the cache, d = 64
        dict(name="append-prompt", kind="append", B=3, n=8001, Hkv=8, d=64, Nk=12000, ragged=True, dtype="fp16"),
        # a short history read back for the next chunk of a prompt
        dict(name="read-short", kind="read", B=2, N=333, Hkv=4, d=64, Nk=512, ragged=True, dtype="fp16"),
        # a long one, 134 MB of codes
        dict(name="read-long", kind="read", B=4, N=16384, Hkv=8, d=128, Nk=16384, ragged=False, dtype="bf16"),
        # a single short request: what the launches cost
        dict(name="decode-one", kind="decode", B=1, Hq=8, Hkv=2, d=64, Nk=1000, empty=False, dtype="fp16"),
        # the split-KV decode shape, its cache in E4M3 (half the sequences full, half ragged)
        dict(name="decode-batch", kind="decode", B=64, Hq=32, Hkv=8, d=128, Nk=32768, empty=False, dtype="bf16"),
        # a few requests behind a short system prompt, one with nothing of its own yet
        dict(name="prefix-few", kind="prefix", B=4, Hq=8, Hkv=2, d=64, Np=513, Nk=64, empty=True, fp8=False,
             dtype="fp16"),
        # 64 requests behind a long document
        dict(name="prefix-batch", kind="prefix", B=64, Hq=32, Hkv=8, d=128, Np=32768, Nk=1024, empty=False, fp8=False,
             dtype="bf16"),
        # 250 samples of one prompt, each with its own E4M3 suffix: more query rows than one K/V read serves
        dict(name="prefix-many", kind="prefix", B=250, Hq=32, Hkv=8, d=128, Np=8192, Nk=512, empty=True, fp8=True,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary", "append", "read", "decode", "decode", "prefix", "prefix"])
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while Hkv * G > 64:
        G = rng.choice([1, 2, 3, 4])
    B = _log(rng, 1, 64)
    c = dict(kind=kind, B=B, Hkv=Hkv, d=d, dtype=dtype)
    if kind == "rotary":
        N = _log(rng, 1, max(1, min(8192, (1 << 25) // (B * Hkv * (G + 1) * d))))
        c.update(N=N, Hq=Hkv * G, rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5,
                 scaled=rng.random() < 0.5, back=rng.random() < 0.5, packed=rng.random() < 0.5,
                 far=rng.choice([0, 0, 100000, 2000000]))
    elif kind == "append":
        n = _log(rng, 1, max(1, min(8192, (1 << 23) // (B * Hkv * d))))
        c.update(n=n, Nk=n + _log(rng, 1, 4096), ragged=rng.random() < 0.6)
    elif kind == "read":
        N = _log(rng, 1, max(1, min(32768, (1 << 26) // (B * Hkv * d))))
        c.update(N=N, Nk=N + rng.choice([0, 1, 100, 1000]), ragged=rng.random() < 0.6)
    elif kind == "decode":
        c.update(Hq=Hkv * G, Nk=_log(rng, 1, max(1, min(32768, (1 << 30) // (B * Hkv * d)))), empty=rng.random() < 0.3)
    else:
        c["B"] = B = _log(rng, 1, 250)
        rows = B * Hkv * G
        c.update(Hq=Hkv * G, Np=_log(rng, 1, max(1, min(65536, (1 << 26) // rows, (1 << 26) // (Hkv * d)))),
                 Nk=_log(rng, 1, max(1, min(2048, (1 << 27) // (B * Hkv * d)))), empty=rng.random() < 0.3,
                 fp8=rng.random() < 0.5)
    return c


# --------------------------------------------------------------------------- inputs
def _lengths(c, N, empty):
    """Sequence lengths of a ragged batch: the first half full, the others spread over 1..N; the last empty if asked."""
    B = c["B"]
    lens = [N if 2 * b < B else 1 + int((N - 1) * ((b + 1) * 0.6180339887 % 1.0)) for b in range(B)]
    if empty:
        lens[-1] = 0
    return lens


def _counts(c):
    """Rows that each sequence appends, and the length that its cache has before."""
    n, room = c["n"], c["Nk"] - c["n"]
    counts = _lengths(c, n, c["ragged"] and c["B"] > 2) if c["ragged"] else [n] * c["B"]
    return counts, [int(room * ((b + 1) * 0.6180339887 % 1.0)) for b in range(c["B"])]


def _read_lengths(c):
    return _lengths(c, c["N"], c["B"] > 2) if c["ragged"] else [c["N"]] * c["B"]


def _frequencies(c):
    """Radians per position of each pair, fp64, on the host: base 10000, and for long contexts a
    frequency-dependent interpolation by 8 of an original context of 8192."""
    freqs = []
    for i in range(c["rot"] // 2):
        f = 10000.0 ** (-2.0 * i / c["rot"])
        if c["scaled"]:
            turns = 8192 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            f = keep * f + (1.0 - keep) * f / 8.0
        freqs.append(f)
    return freqs


def _magnitude(c):
    return 0.1 * math.log(8.0) + 1.0 if c["scaled"] else 1.0


def _table(c, device):
    """The rotary plan that a program keeps: turns per position of each pair as a 64-bit fraction of one turn."""
    t = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in _frequencies(c)]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in t], dtype=torch.int64, device=device)


def _quantised(x):
    """E4M3 codes of x [..., d] (float8_e4m3fn) and one fp32 scale per row: amax / 448, 1 for a row of zeros."""
    s = torch.div(x.abs().amax(-1), torch.full((), 448.0, device=x.device))
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn), s


def _fp8_cache(c, N, g, device):
    """Codes [B, N, Hkv, d] (uint8) and scales [B, Hkv, N] of rows whose size varies from token to token."""
    B, H, d = c["B"], c["Hkv"], c["d"]
    codes = torch.empty(B, N, H, d, dtype=torch.uint8, device=device)
    scales = torch.empty(B, H, N, dtype=torch.float32, device=device)
    for b in range(B):
        x = torch.randn(N, H, d, generator=g, device=device)
        q, s = _quantised(x * torch.exp(0.3 * torch.randn(N, H, 1, generator=g, device=device)))
        codes[b] = q.view(torch.uint8)
        scales[b] = s.t()
    return codes, scales


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    B, Hkv, d, kind = c["B"], c["Hkv"], c["d"], c["kind"]
    s = {"case": c, "dtype": dt, "kind": kind}
    if kind == "rotary":
        N, Hq = c["N"], c["Hq"]
        if c["packed"]:
            s["q"], s["k"], _ = normal(B, N, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], dim=2)
        else:
            s["q"], s["k"] = normal(B, N, Hq, d), normal(B, N, Hkv, d)
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=dev, dtype=torch.int32)
        s["positions"] = (first + torch.arange(N, dtype=torch.int32, device=dev)).contiguous()
        s["table"], s["magnitude"] = _table(c, dev), _magnitude(c)
        s["frequencies"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=dev)
    elif kind == "append":
        counts, start = _counts(c)
        s["k"] = normal(B, c["n"], Hkv, d)
        s["v"] = normal(B, c["n"], Hkv, d)
        s["k8"], s["ks"] = _fp8_cache(c, c["Nk"], g, dev)
        s["v8"], s["vs"] = _fp8_cache(c, c["Nk"], g, dev)
        s["start"], s["counts"] = ints(start), ints(counts)
    elif kind == "read":
        s["k8"], s["ks"] = _fp8_cache(c, c["Nk"], g, dev)
        s["v8"], s["vs"] = _fp8_cache(c, c["Nk"], g, dev)
        s["lens"] = ints(_read_lengths(c))
    else:
        s["q"] = normal(B, 1, c["Hq"], d)
        s["lens"] = ints(_lengths(c, c["Nk"], c["empty"]))
        if kind == "decode" or c["fp8"]:
            s["k8"], s["ks"] = _fp8_cache(c, c["Nk"], g, dev)
            s["v8"], s["vs"] = _fp8_cache(c, c["Nk"], g, dev)
        else:
            s["kc"], s["vc"] = normal(B, c["Nk"], Hkv, d), normal(B, c["Nk"], Hkv, d)
        if kind == "prefix":
            s["kp"], s["vp"] = normal(1, c["Np"], Hkv, d), normal(1, c["Np"], Hkv, d)
    return s


# --------------------------------------------------------------------------- the package's calls
def _run_own(s):
    import exact_io_aware_80_b200 as fa

    c, kind = s["case"], s["kind"]
    if kind == "rotary":
        f = fa.rotary_bwd if c["back"] else fa.rotary_fwd
        return f(s["q"], s["k"], s["positions"], s["table"], c["interleaved"], s["magnitude"])
    if kind == "append":
        fa.fp8_cache_append(s["k"], s["v"], s["k8"], s["v8"], s["ks"], s["vs"], s["start"], s["counts"])
        return s["k8"].view(torch.float8_e4m3fn), s["v8"].view(torch.float8_e4m3fn), s["ks"], s["vs"]
    if kind == "read":
        return fa.fp8_cache_read(s["k8"], s["v8"], s["ks"], s["vs"], s["lens"], c["N"], s["dtype"])
    if kind == "decode":
        return fa.decode_fp8(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["lens"])
    if c["fp8"]:
        return fa.decode_shared_prefix(s["q"], s["kp"], s["vp"], s["k8"], s["v8"], s["lens"], s["ks"], s["vs"])
    return fa.decode_shared_prefix(s["q"], s["kp"], s["vp"], s["kc"], s["vc"], s["lens"])


# --------------------------------------------------------------------------- the plain forms
def _rotated(x, cos, sin, rot, interleaved, dt):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)
    return torch.cat((y, x[..., rot:]), -1).to(dt)


def _appended(x, cache, scale, start, counts):
    B, n = x.shape[:2]
    codes, sc = _quantised(x.float())
    src = torch.minimum(torch.arange(n, device=x.device), counts.unsqueeze(1) - 1).clamp(min=0).long()  # [B, n]
    b = torch.arange(B, device=x.device).unsqueeze(1).expand(B, n)
    dst = start.unsqueeze(1).long() + src
    any_row = (counts > 0).view(B, 1, 1)
    cache[b, dst] = torch.where(any_row.unsqueeze(-1), codes.view(torch.uint8)[b, src], cache[b, dst])
    rows = scale.transpose(1, 2)
    rows[b, dst] = torch.where(any_row, sc[b, src], rows[b, dst])


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale.transpose(1, 2).unsqueeze(-1)


def _weighed(q, parts, d):
    """O and LSE over parts of (scores [B, Hkv, G, n] already scaled and masked, their product with V)."""
    m = torch.stack([x.amax(-1) for x, _ in parts]).amax(0)
    mu = torch.where(torch.isinf(m), torch.zeros_like(m), m).unsqueeze(-1)
    ps = [torch.exp(x - mu) for x, _ in parts]
    total = torch.stack([p.sum(-1) for p in ps]).sum(0)
    out = torch.stack([times(p) for p, (_, times) in zip(ps, parts)]).sum(0)
    out = torch.where(total.unsqueeze(-1) > 0, out / total.unsqueeze(-1), torch.zeros_like(out))
    B, Hkv, G = m.shape
    return out.reshape(B, 1, Hkv * G, d).to(q.dtype), (mu.squeeze(-1) + torch.log(total)).reshape(B, Hkv * G, 1)


def _suffix(s, k, v):
    """Masked scores over a batch's own keys, and the product of weights with their values."""
    q = s["q"].float()
    B, _, Hq, d = q.shape
    N, Hkv = k.shape[1:3]
    x = torch.matmul(q.view(B, Hkv, Hq // Hkv, d), k.permute(0, 2, 3, 1)) / math.sqrt(d)
    out = torch.arange(N, device=q.device) >= s["lens"].view(B, 1, 1, 1)
    return x.masked_fill(out, -math.inf), lambda p: torch.matmul(p, v.transpose(1, 2))


def _prefix(s):
    """The same over the one prefix of all: the batch's rows side by side."""
    q, k, v = s["q"].float(), s["kp"][0].float(), s["vp"][0].float()
    B, _, Hq, d = q.shape
    N, Hkv, _ = k.shape
    G = Hq // Hkv
    rows = q.view(B, Hkv, G, d).transpose(0, 1).reshape(Hkv, B * G, d)
    x = torch.matmul(rows, k.permute(1, 2, 0)) / math.sqrt(d)
    back = lambda t: t.view(Hkv, B, G, -1).transpose(0, 1)  # noqa: E731
    return back(x), lambda p: back(torch.matmul(p.transpose(0, 1).reshape(Hkv, B * G, N), v.transpose(0, 1)))


def _run_plain(s):
    c, kind = s["case"], s["kind"]
    if kind == "rotary":
        angle = s["positions"].double().unsqueeze(-1) * s["frequencies"]
        cos = (torch.cos(angle) * s["magnitude"]).float().unsqueeze(2)
        sin = (torch.sin(angle) * s["magnitude"]).float().unsqueeze(2)
        sin = -sin if c["back"] else sin
        return tuple(_rotated(s[n], cos, sin, c["rot"], c["interleaved"], s["dtype"]) for n in ("q", "k"))
    if kind == "append":
        _appended(s["k"], s["k8"], s["ks"], s["start"], s["counts"])
        _appended(s["v"], s["v8"], s["vs"], s["start"], s["counts"])
        return s["k8"].view(torch.float8_e4m3fn), s["v8"].view(torch.float8_e4m3fn), s["ks"], s["vs"]
    if kind == "read":
        N = c["N"]
        live = (torch.arange(N, device=s["lens"].device) < s["lens"].unsqueeze(1)).view(-1, N, 1, 1)
        k = torch.where(live, _values(s["k8"][:, :N], s["ks"][:, :, :N]), 0.0).to(s["dtype"])
        return k, torch.where(live, _values(s["v8"][:, :N], s["vs"][:, :, :N]), 0.0).to(s["dtype"])
    if kind == "decode" or c["fp8"]:
        parts = [_suffix(s, _values(s["k8"], s["ks"]), _values(s["v8"], s["vs"]))]
    else:
        parts = [_suffix(s, s["kc"].float(), s["vc"].float())]
    if kind == "prefix":
        parts.append(_prefix(s))
    return _weighed(s["q"], parts, c["d"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, kind = case, case["kind"]
    d, Hkv, B = c["d"], c["Hkv"], c["B"]
    row8 = d + 4  # one cached K or V row of a head: codes and scale
    if kind == "rotary":
        n = B * c["N"] * (c["Hq"] + Hkv)
        return {"bytes": 4 * n * d + 4 * B * c["N"] + 4 * c["rot"], "flops": 3 * n * c["rot"]}
    if kind == "append":
        n = 2 * sum(_counts(c)[0]) * Hkv
        return {"bytes": n * (2 * d + row8) + 8 * B, "flops": 2 * n * d}
    if kind == "read":
        live = sum(_read_lengths(c))
        return {"bytes": 2 * Hkv * (live * row8 + B * c["N"] * 2 * d) + 4 * B, "flops": 2 * Hkv * live * d}
    own_keys = sum(_lengths(c, c["Nk"], c["empty"]))
    qo = B * c["Hq"] * (4 * d + 4) + 4 * B
    if kind == "decode":
        return {"bytes": 2 * own_keys * Hkv * row8 + qo, "flops": 4 * own_keys * c["Hq"] * d}
    own_row = row8 if c["fp8"] else 2 * d
    return {"bytes": 2 * own_keys * Hkv * own_row + 4 * c["Np"] * Hkv * d + qo,
            "flops": 4 * (own_keys + B * c["Np"]) * c["Hq"] * d}


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_rows(x):
    """The quotients that codes stand for, and the scales."""
    s = x.abs().amax(-1) / 448
    s = torch.where(s > 0, s, torch.ones_like(s))
    return x / s.unsqueeze(-1), s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind, d, Hkv, B = c["kind"], c["d"], c["Hkv"], c["B"]
    if kind == "rotary":
        turn = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
        angle = s["positions"].double()[..., None] * turn
        z = torch.polar(torch.full_like(angle, s["magnitude"]), -angle if c["back"] else angle)[:, :, None]
        out = []
        for x in (s["q"].double(), s["k"].double()):
            y, r = x.clone(), c["rot"]
            if c["interleaved"]:
                y[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * z
                                                ).flatten(-2)
            else:
                w = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * z
                y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
            out.append(y)
        return tuple(out)
    if kind == "append":
        counts, start = _counts(c)
        out = [s["k8"].view(torch.float8_e4m3fn).double(), s["v8"].view(torch.float8_e4m3fn).double(),
               s["ks"].double(), s["vs"].double()]
        for b in range(B):
            at = slice(start[b], start[b] + counts[b])
            for i, x in enumerate((s["k"], s["v"])):
                out[i][b, at], sc = _exact_rows(x[b, :counts[b]].double())
                out[2 + i][b, :, at] = sc.t()
        return tuple(out)

    def cached(codes, scales, b, n):
        return codes[b, :n].view(torch.float8_e4m3fn).double() * scales[b, :, :n].double().t()[..., None]

    if kind == "read":
        out = []
        for codes, scales in ((s["k8"], s["ks"]), (s["v8"], s["vs"])):
            x = torch.zeros(B, c["N"], Hkv, d, dtype=torch.float64, device="cuda")
            for b, n in enumerate(_read_lengths(c)):
                x[b, :n] = cached(codes, scales, b, n)
            out.append(x)
        return tuple(out)
    Hq = c["Hq"]
    o = torch.zeros(B, 1, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, 1), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c, c["Nk"], c["empty"])):
        if kind == "decode" or c["fp8"]:
            k, v = cached(s["k8"], s["ks"], b, n), cached(s["v8"], s["vs"], b, n)
        else:
            k, v = s["kc"][b, :n].double(), s["vc"][b, :n].double()
        if kind == "prefix":
            k, v = torch.cat((s["kp"][0].double(), k)), torch.cat((s["vp"][0].double(), v))
        if not len(k):
            continue
        q = s["q"][b, 0].double().view(Hkv, Hq // Hkv, d)
        x = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(d)
        lse[b, :, 0] = torch.logsumexp(x, -1).flatten()
        o[b, 0] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(Hq, d)
    return o, lse
