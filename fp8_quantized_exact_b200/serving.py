"""Binding of the serving calls of the C ABI: rotary positions, the quantised
paged cache, and the attention of new or drafted tokens over it.

Argument marshalling only, as in the package's ``__init__``, whose namespace
holds these functions too.  The four calls of a decode step go through a small
CPython module (``csrc/serving_py.c``), because what ctypes and Python spend on
their many arguments is more than their kernels take.

A cache is a tuple ``(k, k_scale, v, v_scale)``: codes int8 or float8_e4m3fn
[pages, H, page_size, D], scales float32 [pages, H, page_size], contiguous.
Tensors must be on the current CUDA device, on which the library launches; a
tensor that is elsewhere, or of another type or shape than its argument, raises
ValueError, and a code that the library returns raises SageError.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

import fp8_quantized_exact_b200 as _sage
from fp8_quantized_exact_b200 import build
from fp8_quantized_exact_b200 import (SAGE_CACHE_E4M3, SAGE_CACHE_INT8, SAGE_ROPE_HALF, SAGE_ROPE_PLAIN,
                                      SAGE_STATUS_BYTES, SageError, sage_rope_config)

_FORMAT = {torch.int8: SAGE_CACHE_INT8, torch.float8_e4m3fn: SAGE_CACHE_E4M3}
_bound = None
_native = None


def _calls():
    """The CPython module, bound to the loaded library."""
    global _bound, _native
    lib = _sage.lib()
    if _bound is not lib:
        if _native is None:
            path = build.SERVING
            if not os.path.exists(path):
                raise RuntimeError(f"serving module not built: {path} is missing (run __graft_entry__.build())")
            loader = importlib.machinery.ExtensionFileLoader("_sage_serving", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_sage_serving", loader))
            loader.exec_module(module)
            _native = module
        _native.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                       for n in ("sage_rope", "sage_cache_append", "sage_cache_read", "sage_cache_attn")], SageError)
        _bound = lib
    return _native


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _check(rc, what):
    if rc:
        raise SageError(rc, what)


def sage_rope_freqs(rot_dim, base=10000.0, scaling=SAGE_ROPE_PLAIN, factor=1.0, trained_len=4096.0, beta_fast=32.0,
                    beta_slow=1.0, device="cuda"):
    """(inv_freq, mscale) for sage_rope: FP64 [rot_dim/2] on `device`, and a float."""
    out = torch.empty(max(rot_dim // 2, 1), dtype=torch.float64)
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
    _calls().rope(q, k, q_out, k_out, positions, inv_freq, mscale, layout, rot_dim, inverse, _handle(stream))


def sage_cache_append(cache, k, v, page_table, start, count, workspace, stream=None):
    """Quantise the first count[b] tokens of k and v [B, N, H, D] into the
    slots from start[b] on (start, count: int32 [B]; None: 0 and N)."""
    _calls().append(cache, k, v, page_table, start, count, workspace, _handle(stream))


def sage_cache_read(cache, page_table, start, count, k_out, v_out, workspace, stream=None):
    """Slots start[b] .. start[b] + count[b] - 1 of each sequence as BF16 into
    the first rows of k_out and v_out [B, N, H, D] (either may be None); the
    other rows are left as they were."""
    _calls().read(cache, page_table, start, count, k_out, v_out, workspace, _handle(stream))


def sage_cache_attn(q, cache, page_table, context, count, mask, out, lse, sm_scale, workspace, stream=None):
    """Attention of the T new or drafted tokens of each sequence, q [B, T, Hq,
    D], over its context[b] cached tokens and, by mask (int32 [B, T,
    ceil(T/32)]; None: j <= i), the drafted ones in the slots behind them.
    count: int32 [B] or None (T); lse: float32 [B, T, Hq] or None."""
    _calls().attn(q, cache, page_table, context, count, mask, out, lse, sm_scale, workspace, _handle(stream))


def sage_clear_device_status(workspace, stream=None):
    """Zero the workspace's status block."""
    if (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous() or
            workspace.numel() * workspace.element_size() < SAGE_STATUS_BYTES):
        raise ValueError("sage_clear_device_status: workspace must be a contiguous CUDA tensor of at least "
                         f"{SAGE_STATUS_BYTES} bytes")
    _check(_sage.lib().sage_clear_device_status(workspace.data_ptr(), _sage._stream(stream)), "sage_clear_device_status")


def cache_buffers(pages: int, H: int, page_size: int, D: int, k_format: int = SAGE_CACHE_INT8,
                  v_format: int = SAGE_CACHE_E4M3, device="cuda"):
    """An empty cache: (k, k_scale, v, v_scale)."""
    dtype = {f: t for t, f in _FORMAT.items()}
    codes = lambda f: torch.empty((pages, H, page_size, D), dtype=dtype[f], device=device)
    scale = lambda: torch.empty((pages, H, page_size), dtype=torch.float32, device=device)
    return codes(k_format), scale(), codes(v_format), scale()
