"""fp64 CPU oracle of rotary positions, the E4M3 cache and decode behind a shared prefix.

TEST INFRASTRUCTURE ONLY, like the other modules here: never imported by the
product, and sharing no code, table or constant with it.

* Rotary positions: pair i of a head, (x[i], x[i + r/2]) or (x[2i], x[2i+1]), is
  multiplied as a complex number by m e^{i p f_i}.
* E4M3 cache: row scale s = amax / 448 (1 for zeros) and codes of x / s, both
  divisions rounded to fp32 (the codes are decisions taken in fp32).
* Shared prefix: plain attention over the prefix's keys followed by the
  sequence's own.

The error bounds at the end state how far a kernel that rounds its weights to
16 bits and sums in fp32 may be from these.
"""
from __future__ import annotations

import numpy as np

from .attn_ref import decode
from .fp8_ref import e4m3_decode, e4m3_encode

__all__ = ["frequencies", "rotary", "quantize_rows", "cache_values", "decode_prefix", "decode_bounds", "rotary_bound"]


def frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, original_len=None, low=1.0, high=32.0):
    """base^(-2i / rot); with original_len, interpolated by parts (divided by ``factor`` below ``low``
    turns over original_len, kept above ``high``, linear between)."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if original_len is not None:
        ramp = np.clip((original_len * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = ramp * f + (1 - ramp) * f / factor
    return f


def rotary(x, positions, freqs, interleaved: bool, magnitude: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [B, N, H, d]; positions [N] or [B, N]."""
    x = np.array(x, dtype=np.float64)
    r = 2 * len(freqs)
    pos = np.broadcast_to(np.asarray(positions, dtype=np.float64), x.shape[:2])
    z = magnitude * np.exp((-1j if inverse else 1j) * pos[:, :, None, None] * np.asarray(freqs))
    if interleaved:
        y = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * z
        x[..., 0:r:2], x[..., 1:r:2] = y.real, y.imag
    else:
        y = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * z
        x[..., :r // 2], x[..., r // 2:r] = y.real, y.imag
    return x


def rotary_bound(x, y, freqs, interleaved: bool, magnitude: float, eps: float, reach: float = 0.0) -> np.ndarray:
    """|error| of one rotation computed in fp32 and rounded once to a type with machine epsilon eps.

    The half turn in fp32 is off by 2^-25 of itself (at most 1), i.e. pi 2^-25 < 2^-23 radians, sine and
    cosine by 2^-23 each, two products and a sum by 3 x 2^-24: together under 2^-20 m (|x0| + |x1|).
    ``reach`` = max |p f|: both sides' fp64 frequencies and angles carry a few roundings of 2^-53, up to
    16 together, 2^-49 reach radians.  The final rounding moves y by at most eps / 2 |y| (2^-25 absolute
    below fp16's normal range).
    """
    a = np.abs(np.asarray(x, dtype=np.float64))
    r = 2 * len(freqs)
    s = np.zeros_like(a)
    if interleaved:
        both = a[..., 0:r:2] + a[..., 1:r:2]
        s[..., 0:r:2] = s[..., 1:r:2] = both
    else:
        both = a[..., :r // 2] + a[..., r // 2:r]
        s[..., :r // 2] = s[..., r // 2:r] = both
    return (2.0 ** -20 + 2.0 ** -49 * reach) * abs(magnitude) * s + (eps / 2) * np.abs(y) * (1 + 2.0 ** -10) + 2.0 ** -25


def quantize_rows(x):
    """E4M3 codes [..., d] (uint8) and fp32 scales [...] of the rows of x."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(axis=-1)
    s = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
    return e4m3_encode((x / s[..., None]).astype(np.float32)), s


def cache_values(codes, scales) -> np.ndarray:
    """fp64 values of codes [B, N, H, d] with scales [B, H, N]."""
    return e4m3_decode(codes) * np.asarray(scales, dtype=np.float64).transpose(0, 2, 1)[..., None]


def decode_prefix(q, k_prefix, v_prefix, k_cache, v_cache, seqlens, scale: float):
    """One-token attention over the prefix [Np, H, d] and then each sequence's own keys."""
    B, Np = len(seqlens), k_prefix.shape[0]
    out = []
    for b in range(B):
        n = int(seqlens[b])
        k = np.concatenate([k_prefix, k_cache[b, :n]])[None]
        v = np.concatenate([v_prefix, v_cache[b, :n]])[None]
        out.append(decode(q[b:b + 1], k, v, [Np + n], scale))
    return np.concatenate([o for o, _ in out]), np.concatenate([x for _, x in out])


def decode_bounds(q, k, v, seqlens, scale: float, half_step: float, out_half_step: float, floor: float):
    """Per-element bounds (O [B,1,Hq,d], LSE [B,Hq,1]) for one-token attention whose weights are rounded.

    k, v [B, N, H, d] fp64, the values the kernel's operands stand for.
    Scores: products are exact in fp32, sums of d of them are off by at most d 2^-23 sum |q k| each
    (2^-23: a tensor core may truncate), scaling and the exponent's argument add 4 x 2^-24 of the largest
    |t|; call the sum delta (natural-log units).  A weight is then off by a factor e^{2 delta} (score and
    maximum), 2^-20 for the exponential and the sums, half_step for its rounding, and ``floor``
    absolute (relative to the largest weight) where the type's normal range ends.  Hence
      |dO| <= (2 delta + 2^-20 + half_step) (sum_j p_j |v_j| / l + |O|) + floor sum_j |v_j| + out_half_step |O|,
    where l >= 1 relative to the largest weight, and |dLSE| <= 2 delta + 2^-20 (1 + |LSE|).
    """
    B, _, Hq, d = q.shape
    H = k.shape[2]
    G = Hq // H
    bo = np.zeros((B, 1, Hq, d))
    bl = np.zeros((B, Hq, 1))
    for b in range(B):
        n = int(seqlens[b])
        if n == 0:
            continue
        for h in range(Hq):
            kk, vv, qq = k[b, :n, h // G], v[b, :n, h // G], q[b, 0, h]
            x = scale * (kk @ qq)
            delta = scale * d * 2.0 ** -23 * np.max(np.abs(kk) @ np.abs(qq)) + 4 * 2.0 ** -24 * np.max(np.abs(x)) * 1.5
            p = np.exp(x - x.max())
            l = p.sum()
            o = np.abs(p @ vv) / l
            spread = (p @ np.abs(vv)) / l
            bo[b, 0, h] = ((2 * delta + 2.0 ** -20 + half_step) * (spread + o) + floor * np.abs(vv).sum(0)
                           + out_half_step * o * (1 + 2.0 ** -7) + 2.0 ** -25)
            bl[b, h, 0] = 2 * delta + 2.0 ** -20 * (1 + abs(x.max() + np.log(l)))
    return bo, bl
