"""Rotary positions, an E4M3 key/value cache, and decode over it or behind a shared prefix.

PyTorch-facing wrappers of the entry points of the same kinds in ``include/fa.h``.
As in the package's other wrappers only tensor metadata is checked, outputs and
workspaces are allocated with PyTorch, and raw pointers plus the current CUDA
stream go to libfa.so; there is no CPU or PyTorch fallback.

Layouts: q, o [B, N, Hq, d]; k, v [B, N, Hkv, d]; an E4M3 cache is k8, v8
[B, Nk_max, Hkv, d] uint8 with k_scale, v_scale [B, Hkv, Nk_max] float32;
seqlens_k, start, counts int32 [B].
"""
from __future__ import annotations

import functools
import math

from . import _lib

__all__ = ["rotary_table", "rotary_magnitude", "rotary_fwd", "rotary_bwd", "fp8_cache_append", "fp8_cache_read",
           "decode_fp8", "decode_shared_prefix"]

# These calls serve single tokens, where the host's share of a pass is the larger one: checks pass on
# one expression and take a bad tensor apart only to say what is wrong with it, and what every call
# looks up is looked up once.
torch = None
_entries: dict = {}
_get_device = _get_stream = None


def _torch():
    global torch, _get_device, _get_stream
    if torch is None:
        import torch as module
        _get_device, _get_stream = module._C._cuda_getDevice, module._C._cuda_getCurrentRawStream
        torch = module
    return torch


def _dt(t):
    dtype = t.dtype
    if dtype is (torch or _torch()).bfloat16:
        return _lib.FA_BF16
    if dtype is torch.float16:
        return _lib.FA_FP16
    raise TypeError(f"attention tensors must be fp16 or bf16, got {dtype}")


def _device(t):
    if not t.is_cuda:
        raise ValueError("libfa.so takes CUDA tensors only (no CPU path)")
    return t.device


def _check(name, t, dtype, shape, dev, contiguous=True):
    if t.dtype is dtype and t.shape == shape and t.device == dev and (not contiguous or t.is_contiguous()):
        return
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, the device of the first argument, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _call(dev, name, *args):
    """The C entry point with ``dev`` current, on its current stream."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(_lib.load(), name)
    index = dev.index
    if index == _get_device():
        rc = fn(*args, _get_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _get_stream(index))
    if rc != 0:  # FA_OK
        raise _lib.FAError(name, rc)


def _strides(name, t, B, N, H, d):
    """(batch, token) strides of [B, N, H, d] whose heads are contiguous."""
    if t.is_contiguous():
        return N * H * d, H * d
    sb, sn, sh, sd = t.stride()
    if (sh != d and H > 1) or (sd != 1 and d > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return (sb if B > 1 else 0), (sn if N > 1 else 0)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rotary_table(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original_len: int | None = None, low_turns: float = 1.0, high_turns: float = 32.0, device="cuda"):
    """The frequencies f_i = base^(-2i / rot_dim) as the int64 table that the rotary calls take.

    Entry i is f_i / (2 pi), turns per position, as a 64-bit fraction of one turn.  For contexts
    longer than the trained one:

    * ``scaling="linear"``: positions divided by ``factor``;
    * ``scaling="ntk"``: base grown to base * factor^(rot_dim / (rot_dim - 2)), which divides the
      lowest frequency by ``factor`` and leaves the highest;
    * ``scaling="by_parts"``: with r = original_len f_i / (2 pi) turns over the trained context, f_i
      is divided by ``factor`` for r <= low_turns, kept for r >= high_turns, and blended linearly in
      r between them (see also :func:`rotary_magnitude`).
    """
    torch = _torch()
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not (base > 0 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if scaling not in (None, "linear", "ntk", "by_parts"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'by_parts', got {scaling!r}")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("scaling='ntk' needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    if scaling == "by_parts" and (original_len is None or original_len < 1 or not 0 <= low_turns < high_turns):
        raise ValueError("scaling='by_parts' needs original_len >= 1 and 0 <= low_turns < high_turns")
    turns = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            r = original_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (r - low_turns) / (high_turns - low_turns)))
            f = keep * f + (1.0 - keep) * f / factor
        u = int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64)
        turns.append(u - (1 << 64) if u >= 1 << 63 else u)
    return torch.tensor(turns, dtype=torch.int64, device=device)


def rotary_magnitude(factor: float) -> float:
    """0.1 ln(factor) + 1 (1 for factor <= 1): the ``magnitude`` that goes with ``by_parts`` scaling."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _rotary(q, k, positions, table, interleaved, magnitude, inverse, q_out, k_out):
    dt, dev, dtype, shape = _dt(q), _device(q), q.dtype, q.shape
    B, N, Hq, d = shape
    each = positions.dim() == 2
    _check("positions", positions, torch.int32, (B, N) if each else (N,), dev)
    pairs = table.numel()
    _check("table", table, torch.int64, (pairs,), dev)
    q_bs, q_ts = _strides("q", q, B, N, Hq, d)
    k_bs = k_ts = Hkv = kp = kop = 0
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _check("q_out", q_out, dtype, shape, dev)
    if k is not None:
        Hkv = k.shape[2]
        shape = (B, N, Hkv, d)
        _check("k", k, dtype, shape, dev, contiguous=False)
        k_bs, k_ts = _strides("k", k, B, N, Hkv, d)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        else:
            _check("k_out", k_out, dtype, shape, dev)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    _call(dev, "fa_rotary", q.data_ptr(), kp, q_out.data_ptr(), kop, positions.data_ptr(), table.data_ptr(), B, N,
          Hq, Hkv, d, 2 * pairs, bool(interleaved), inverse, magnitude, q_bs, q_ts, k_bs, k_ts,
          N if each else 0, dt)
    return q_out, k_out


def rotary_fwd(q, k, positions, table, interleaved: bool = False, magnitude: float = 1.0, q_out=None, k_out=None):
    """q and k turned by their tokens' positions, via ``fa_rotary``; returns (q, k).

    ``positions``: int32 [B, N], or [N] shared by the batch; ``table``: from :func:`rotary_table`, its
    rot_dim at most d (later values of each head are copied).  q and k may be slices of one packed
    projection (heads contiguous); k may be None.  Outputs are contiguous; ``q_out=q`` (``k_out=k``)
    works in place on a contiguous tensor.
    """
    return _rotary(q, k, positions, table, interleaved, magnitude, False, q_out, k_out)


def rotary_bwd(dq, dk, positions, table, interleaved: bool = False, magnitude: float = 1.0, q_out=None, k_out=None):
    """Gradients with respect to :func:`rotary_fwd`'s q and k from those of its outputs: the transpose
    of the rotation, with the same positions, table, layout and magnitude."""
    return _rotary(dq, dk, positions, table, interleaved, magnitude, True, q_out, k_out)


# ---------------------------------------------------------------------------
# the E4M3 cache
# ---------------------------------------------------------------------------
def _check_cache(k8, v8, k_scale, v_scale, B, Hkv, d, dev):
    Nk_max = k8.shape[1]
    u8, f32, codes, scales = torch.uint8, torch.float32, (B, Nk_max, Hkv, d), (B, Hkv, Nk_max)
    if not (k8.dtype is u8 and v8.dtype is u8 and k_scale.dtype is f32 and v_scale.dtype is f32 and
            k8.shape == codes and v8.shape == codes and k_scale.shape == scales and v_scale.shape == scales and
            k8.device == dev and v8.device == dev and k_scale.device == dev and v_scale.device == dev and
            k8.is_contiguous() and v8.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()):
        _check("k8", k8, u8, codes, dev)
        _check("v8", v8, u8, codes, dev)
        _check("k_scale", k_scale, f32, scales, dev)
        _check("v_scale", v_scale, f32, scales, dev)
    return Nk_max


def fp8_cache_append(k, v, k8, v8, k_scale, v_scale, start, counts=None):
    """Quantise k, v [B, n, Hkv, d] into rows start[b] .. of an E4M3 cache, in place, via ``fa_fp8_cache_append``.

    ``counts``: int32 [B], rows that each sequence appends (None: all n).  Rows that fall outside the
    cache are dropped.  k and v may be slices of one packed projection (heads contiguous).
    """
    dt, dev = _dt(k), _device(k)
    B, n, Hkv, d = k.shape
    _check("v", v, k.dtype, k.shape, dev, contiguous=False)
    Nk_max = _check_cache(k8, v8, k_scale, v_scale, B, Hkv, d, dev)
    _check("start", start, torch.int32, (B,), dev)
    if counts is not None:
        _check("counts", counts, torch.int32, (B,), dev)
    _call(dev, "fa_fp8_cache_append", k.data_ptr(), v.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), start.data_ptr(), 0 if counts is None else counts.data_ptr(), B, n, Hkv, Nk_max, d,
          *_strides("k", k, B, n, Hkv, d), *_strides("v", v, B, n, Hkv, d), dt)


def fp8_cache_read(k8, v8, k_scale, v_scale, seqlens_k, Nk: int | None = None, dtype=None):
    """The first Nk rows (None: all) of an E4M3 cache as (k, v) [B, Nk, Hkv, d] in ``dtype`` (bf16 by
    default), rows past seqlens_k[b] zero, via ``fa_fp8_cache_read``."""
    _torch()
    dev = _device(k8)
    B, Nk_max, Hkv, d = k8.shape
    _check_cache(k8, v8, k_scale, v_scale, B, Hkv, d, dev)
    _check("seqlens_k", seqlens_k, torch.int32, (B,), dev)
    Nk = Nk_max if Nk is None else Nk
    k = k8.new_empty((B, Nk, Hkv, d), dtype=torch.bfloat16 if dtype is None else dtype)
    v = torch.empty_like(k)
    _call(dev, "fa_fp8_cache_read", k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
          seqlens_k.data_ptr(), k.data_ptr(), v.data_ptr(), B, Nk, Hkv, Nk_max, d, _dt(k))
    return k, v


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def _plan(device, B, Hq, Hkv, Np, Nk_max, d, fp8, prefix_splits):
    """Prefix splits (None: the library's suggestion) and workspace bytes: functions of the sizes alone."""
    if prefix_splits is None:
        with _torch().cuda.device(device):
            prefix_splits = _lib.fa_decode_prefix_splits(B, Hq, Hkv, Np, Nk_max, d, fp8)
    # (more splits than tiles are refused by the call itself, not for want of memory)
    return prefix_splits, _lib.fa_decode_fp8_workspace_bytes(B, Hq, Hkv, Nk_max, min(prefix_splits, -(-Np // 128)), d)


def _decode_buffers(q, seqlens_k, need, workspace, out, lse):
    dev, dtype = q.device, q.dtype
    B, _, Hq, d = q.shape
    shape = (B, 1, Hq, d)
    _check("q", q, dtype, shape, dev)
    _check("seqlens_k", seqlens_k, torch.int32, (B,), dev)
    if workspace is None:
        workspace = q.new_empty(need, dtype=torch.uint8) if need else None
    elif workspace.device != dev or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be contiguous, on the device of q and hold {need} bytes")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, dtype, shape, dev)
    if lse is None:
        lse = q.new_empty((B, Hq, 1), dtype=torch.float32)
    else:
        _check("lse", lse, torch.float32, (B, Hq, 1), dev)
    return workspace, out, lse


def decode_fp8(q, k8, v8, k_scale, v_scale, seqlens_k, scale: float | None = None, workspace=None, out=None,
               lse=None):
    """One-token attention over an E4M3 cache; returns O [B, 1, Hq, d] and LSE [B, Hq, 1] (``fa_decode_fp8``)."""
    dt, dev = _dt(q), _device(q)
    B, _, Hq, d = q.shape
    Hkv = k8.shape[2]
    Nk_max = _check_cache(k8, v8, k_scale, v_scale, B, Hkv, d, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _, need = _plan(dev.index, B, Hq, Hkv, 0, Nk_max, d, True, 0)
    workspace, out, lse = _decode_buffers(q, seqlens_k, need, workspace, out, lse)
    _call(dev, "fa_decode_fp8", q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
          seqlens_k.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr() if need else 0, B, Hq,
          Hkv, Nk_max, d, scale, dt)
    return out, lse


def decode_shared_prefix(q, k_prefix, v_prefix, k_cache, v_cache, seqlens_k, k_scale=None, v_scale=None,
                         prefix_splits: int | None = None, scale: float | None = None, workspace=None, out=None,
                         lse=None):
    """One-token attention of a batch behind one prefix; returns O [B, 1, Hq, d] and LSE [B, Hq, 1].

    Every sequence sees all of ``k_prefix``, ``v_prefix`` [1, Np, Hkv, d] and then the first
    seqlens_k[b] rows (0 allowed) of its own cache, [B, Nk_max, Hkv, d] in q's type, or uint8 E4M3
    codes with ``k_scale`` and ``v_scale`` (``fa_decode_shared_prefix``).  The GPU is divided between the
    prefix and the caches by Nk_max: caches with far more room than their sequences use slow the call.
    """
    dt, dev, dtype = _dt(q), _device(q), q.dtype
    B, _, Hq, d = q.shape
    _, Np, Hkv, _ = k_prefix.shape
    shape = (1, Np, Hkv, d)
    _check("k_prefix", k_prefix, dtype, shape, dev)
    _check("v_prefix", v_prefix, dtype, shape, dev)
    if k_cache.dtype == torch.uint8:
        if k_scale is None or v_scale is None:
            raise ValueError("an E4M3 cache comes with k_scale and v_scale")
        Nk_max = _check_cache(k_cache, v_cache, k_scale, v_scale, B, Hkv, d, dev)
        ksp, vsp = k_scale.data_ptr(), v_scale.data_ptr()
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale go with uint8 E4M3 caches")
        Nk_max = k_cache.shape[1]
        shape = (B, Nk_max, Hkv, d)
        _check("k_cache", k_cache, dtype, shape, dev)
        _check("v_cache", v_cache, dtype, shape, dev)
        ksp = vsp = 0
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    prefix_splits, need = _plan(dev.index, B, Hq, Hkv, Np, Nk_max, d, bool(ksp), prefix_splits)
    workspace, out, lse = _decode_buffers(q, seqlens_k, need, workspace, out, lse)
    _call(dev, "fa_decode_shared_prefix", q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), ksp, vsp, seqlens_k.data_ptr(), out.data_ptr(), lse.data_ptr(),
          0 if workspace is None else workspace.data_ptr(), B, Hq, Hkv, Np, Nk_max, d, scale, prefix_splits, dt)
    return out, lse
