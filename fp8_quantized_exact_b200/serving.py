"""Binding of the serving calls of the C ABI: rotary positions, the quantised
paged cache, and the attention of new or drafted tokens over it.

Argument marshalling only, as in the package's ``__init__``, whose namespace
holds these functions too.  A decode step makes three short calls per layer, so
what they spend on the host counts: each tensor's attributes are read once.

A cache is a tuple ``(k, k_scale, v, v_scale)``: codes int8 or float8_e4m3fn
[pages, H, page_size, D], scales float32 [pages, H, page_size], contiguous.
Tensors must be on the current CUDA device, on which the library launches.
"""
from __future__ import annotations

import ctypes

import torch

import fp8_quantized_exact_b200 as _sage
from fp8_quantized_exact_b200 import (SAGE_CACHE_E4M3, SAGE_CACHE_INT8, SAGE_ROPE_HALF, SAGE_ROPE_PLAIN, SageError,
                                      sage_cache, sage_rope_config, sage_view_bf16)

_BF16, _I32, _F32, _F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
_FORMAT = {torch.int8: SAGE_CACHE_INT8, torch.float8_e4m3fn: SAGE_CACHE_E4M3}
_NO_VIEW = sage_view_bf16(None, 0, 0, 0)


def _device(what):
    if not torch.cuda.is_initialized():
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    return torch._C._cuda_getDevice()


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(rc, what):
    if rc:
        raise SageError(rc, what)


def _bf16(t, shape, dev, what, name):
    """(address, strides) of a BF16 view with unit stride over its last dimension."""
    st = t.stride()
    if t.dtype != _BF16 or t.shape != shape or len(st) != 4 or st[3] != 1 or t.get_device() != dev:
        raise ValueError(f"{what}: {name} must be bfloat16 {tuple(shape)} with unit stride over D on the current CUDA "
                         f"device {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr(), st[0], st[1], st[2]


def _plain(t, dtype, shape, dev, what, name):
    """Address of a contiguous tensor."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what}: {name} must be contiguous {dtype} {tuple(shape)} on the current CUDA device {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cache(cache, dev, what) -> sage_cache:
    k, ks, v, vs = cache
    shape = k.shape
    kf, vf = _FORMAT.get(k.dtype), _FORMAT.get(v.dtype)
    if len(shape) != 4 or kf is None or vf is None:
        raise ValueError(f"{what}: the cache's codes must be int8 or float8_e4m3fn [pages, H, page_size, D]")
    rows = shape[:3]
    return sage_cache(_plain(k, k.dtype, shape, dev, what, "k"), _plain(ks, _F32, rows, dev, what, "k_scale"),
                      _plain(v, v.dtype, shape, dev, what, "v"), _plain(vs, _F32, rows, dev, what, "v_scale"),
                      kf, vf, shape[0], shape[2], shape[1], shape[3])


def _table(t, B, dev, what):
    shape = t.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"{what}: page_table must be int32 [{B}, pages of a sequence]")
    return _plain(t, _I32, shape, dev, what, "page_table"), shape[1]


def _workspace(t, dev, what):
    if not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what}: the workspace must be contiguous on the current CUDA device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def sage_rope_freqs(rot_dim, base=10000.0, scaling=SAGE_ROPE_PLAIN, factor=1.0, trained_len=4096.0, beta_fast=32.0,
                    beta_slow=1.0, device="cuda"):
    """(inv_freq, mscale) for sage_rope: FP64 [rot_dim/2] on `device`, and a float."""
    out = torch.empty(max(rot_dim // 2, 1), dtype=_F64)
    mscale = ctypes.c_float(1.0)
    cfg = sage_rope_config(int(scaling), int(rot_dim), float(base), float(factor), float(trained_len),
                           float(beta_fast), float(beta_slow))
    _check(_sage.lib().sage_rope_freqs(ctypes.byref(cfg), out.data_ptr(), ctypes.byref(mscale)), "sage_rope_freqs")
    return out.to(device), mscale.value


def sage_rope(q, k, q_out, k_out, positions, inv_freq, mscale=1.0, layout=SAGE_ROPE_HALF, rot_dim=None, inverse=False,
              stream=None):
    """Rotary positions on q and k (k and k_out may be None).  positions:
    int32 [B, N], [N] (shared by the batch) or None (0 .. N-1); rot_dim None:
    2 * len(inv_freq)."""
    what = "sage_rope"
    dev = _device(what)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"{what}: q must be [B, N, H, D]")
    B, N, Hq, D = shape
    freqs = inv_freq.shape
    if rot_dim is None:
        rot_dim = 2 * freqs[0]
    if len(freqs) != 1 or 2 * freqs[0] != rot_dim:
        raise ValueError(f"{what}: inv_freq must be float64 [rot_dim / 2]")
    f = _plain(inv_freq, _F64, freqs, dev, what, "inv_freq")
    pos, pos_stride = None, 0
    if positions is not None:
        st = positions.stride()
        if len(st) == 2:
            pos_stride = st[0]
        if positions.dtype != _I32 or tuple(positions.shape) != ((B, N) if len(st) == 2 else (N,)) or \
                (N > 1 and st[-1] != 1) or positions.get_device() != dev:
            raise ValueError(f"{what}: positions must be int32 [B, N] or [N] with unit stride over N on the current "
                             f"CUDA device {dev}")
        pos = positions.data_ptr()
    vq = sage_view_bf16(*_bf16(q, shape, dev, what, "q"))
    oq = _bf16(q_out, shape, dev, what, "q_out")
    if k is None:
        vk, ok, Hk = _NO_VIEW, (None, 0, 0, 0), 0
    else:
        kshape = k.shape
        if len(kshape) != 4 or kshape[0] != B or kshape[1] != N or kshape[3] != D:
            raise ValueError(f"{what}: q and k must agree in B, N and D")
        vk = sage_view_bf16(*_bf16(k, kshape, dev, what, "k"))
        ok, Hk = _bf16(k_out, kshape, dev, what, "k_out"), kshape[2]
    _check(_sage.lib().sage_rope(vq, Hq, *oq, vk, Hk, *ok, pos, pos_stride, f, mscale, layout, rot_dim,
                                 1 if inverse else 0, B, N, D, _raw_stream(stream, dev)), what)


def sage_cache_append(cache, k, v, page_table, start, count, workspace, stream=None):
    """Quantise the first count[b] tokens of k and v [B, N, H, D] into the
    slots from start[b] on (start, count: int32 [B]; None: 0 and N)."""
    what = "sage_cache_append"
    dev = _device(what)
    c = _cache(cache, dev, what)
    shape = k.shape
    if len(shape) != 4 or shape[2] != c.H or shape[3] != c.D:
        raise ValueError(f"{what}: k and v must be [B, N, H, D] with the cache's H and D")
    B, N = shape[0], shape[1]
    vk, vv = sage_view_bf16(*_bf16(k, shape, dev, what, "k")), sage_view_bf16(*_bf16(v, shape, dev, what, "v"))
    table, per = _table(page_table, B, dev, what)
    first = None if start is None else _plain(start, _I32, (B,), dev, what, "start")
    n = None if count is None else _plain(count, _I32, (B,), dev, what, "count")
    ws, ws_bytes = _workspace(workspace, dev, what)
    _check(_sage.lib().sage_cache_append(ctypes.addressof(c), vk, vv, table, per, first, n, B, N, ws, ws_bytes,
                                         _raw_stream(stream, dev)), what)


def sage_cache_read(cache, page_table, start, count, k_out, v_out, workspace, stream=None):
    """Slots start[b] .. start[b] + count[b] - 1 of each sequence as BF16 into
    the first rows of k_out and v_out [B, N, H, D] (either may be None); the
    other rows are left as they were."""
    what = "sage_cache_read"
    dev = _device(what)
    c = _cache(cache, dev, what)
    like = k_out if k_out is not None else v_out
    if like is None or like.dim() != 4:
        raise ValueError(f"{what}: k_out or v_out must be [B, N, H, D]")
    B, N = like.shape[:2]
    shape = (B, N, c.H, c.D)
    table, per = _table(page_table, B, dev, what)
    first = None if start is None else _plain(start, _I32, (B,), dev, what, "start")
    n = None if count is None else _plain(count, _I32, (B,), dev, what, "count")
    ok = (None, 0, 0, 0) if k_out is None else _bf16(k_out, shape, dev, what, "k_out")
    ov = (None, 0, 0, 0) if v_out is None else _bf16(v_out, shape, dev, what, "v_out")
    ws, ws_bytes = _workspace(workspace, dev, what)
    _check(_sage.lib().sage_cache_read(ctypes.addressof(c), table, per, first, n, *ok, *ov, B, N, ws, ws_bytes,
                                       _raw_stream(stream, dev)), what)


def sage_cache_attn(q, cache, page_table, context, count, mask, out, lse, sm_scale, workspace, stream=None):
    """Attention of the T new or drafted tokens of each sequence, q [B, T, Hq,
    D], over its context[b] cached tokens and, by mask (int32 [B, T,
    ceil(T/32)]; None: j <= i), the drafted ones in the slots behind them.
    count: int32 [B] or None (T); lse: float32 [B, T, Hq] or None."""
    what = "sage_cache_attn"
    dev = _device(what)
    c = _cache(cache, dev, what)
    shape = q.shape
    if len(shape) != 4 or shape[3] != c.D or c.H == 0 or shape[2] % c.H:
        raise ValueError(f"{what}: q must be [B, T, Hq, D] with the cache's D and a multiple of its heads")
    B, T, Hq, D = shape
    if context is None:
        raise ValueError(f"{what}: context is missing")
    vq, o = sage_view_bf16(*_bf16(q, shape, dev, what, "q")), _bf16(out, shape, dev, what, "out")
    table, per = _table(page_table, B, dev, what)
    ctx = _plain(context, _I32, (B,), dev, what, "context")
    n = None if count is None else _plain(count, _I32, (B,), dev, what, "count")
    m = None if mask is None else _plain(mask, _I32, (B, T, (T + 31) // 32), dev, what, "mask")
    ls = None if lse is None else _plain(lse, _F32, (B, T, Hq), dev, what, "lse")
    ws, ws_bytes = _workspace(workspace, dev, what)
    _check(_sage.lib().sage_cache_attn(vq, ctypes.addressof(c), table, per, ctx, n, m, *o, ls, B, T, Hq, sm_scale, ws,
                                       ws_bytes, _raw_stream(stream, dev)), what)


def sage_clear_device_status(workspace, stream=None):
    what = "sage_clear_device_status"
    dev = _device(what)
    ws, _ = _workspace(workspace, dev, what)
    _check(_sage.lib().sage_clear_device_status(ws, _raw_stream(stream, dev)), what)


def cache_buffers(pages: int, H: int, page_size: int, D: int, k_format: int = SAGE_CACHE_INT8,
                  v_format: int = SAGE_CACHE_E4M3, device="cuda"):
    """An empty cache: (k, k_scale, v, v_scale)."""
    dtype = {f: t for t, f in _FORMAT.items()}
    codes = lambda f: torch.empty((pages, H, page_size, D), dtype=dtype[f], device=device)
    scale = lambda: torch.empty((pages, H, page_size), dtype=_F32, device=device)
    return codes(k_format), scale(), codes(v_format), scale()
