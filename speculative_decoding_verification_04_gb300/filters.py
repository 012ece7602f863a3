"""Binding of the filtered distributions (argument marshalling only): min-p,
top-k and top-p, in that order, over rows of logits.

  logits       [B, V], or [B, S, V] for spec_filter_logits; float32 or bfloat16,
               contiguous
  temperature  [B] float32 (0: the argmax alone)
  top_k        [B] int32 (0: off); top_p [B] float32 (1: off); min_p [B] float32
               (0: off); each may be None

See ``include/specverify.h`` for the definitions and for rows that cannot be
used.  A call's tensors (and its stream) are those of the current device.
Every step runs in the CUDA library; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _load, kv_cache
from .kv_cache import _code, _empty

_P, _I32 = ctypes.c_void_p, ctypes.c_int32
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _load()
        lib.spec_sample_filtered.argtypes = [_P, ctypes.c_int, _P, _P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P]
        lib.spec_filter_logits.argtypes = [_P, ctypes.c_int, _P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _P, _P]
        lib.spec_sample_filtered.restype = lib.spec_filter_logits.restype = ctypes.c_int
        _lib = lib
    return _lib


def _ptr(t, name, dtype, shape, dev):
    """The address of an optional contiguous tensor of device `dev`, checked."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the logits and the current device are cuda:{dev}")
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _rows(logits, dims):
    """Dtype code, shape and device of the logits, checked."""
    dev = logits.get_device()
    if dev < 0 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA tensor")
    if dev != kv_cache._current_device():   # the library launches on the current one
        raise ValueError(f"logits are on cuda:{dev}, the current device is cuda:{kv_cache._current_device()}")
    shape = logits.shape
    if len(shape) not in dims:
        raise ValueError("logits must be [B, V]" + (" or [B, S, V]" if 3 in dims else ""))
    return _code(logits.dtype), shape, dev


def _settings(temperature, top_k, top_p, min_p, B, dev):
    one = (B,)
    if temperature is None:
        raise ValueError("temperature must be a [B] tensor")
    return (_ptr(temperature, "temperature", torch.float32, one, dev), _ptr(top_k, "top_k", torch.int32, one, dev),
            _ptr(top_p, "top_p", torch.float32, one, dev), _ptr(min_p, "min_p", torch.float32, one, dev))


def _like(t, dtype, stream):
    """A new tensor of t's shape that belongs to the call's stream."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    return _empty(t, t.shape, dtype, stream)


def spec_sample_filtered(logits, uniforms, temperature, top_k=None, top_p=None, min_p=None, out_tokens=None, out_prob=None,
                         out_kept=None, stream=None):
    """One token per row of ``logits`` [B, V] from the tokens that the filters
    keep, at ``uniforms`` [B] in [0, 1): returns (tokens int32 [B], each one's
    share of the kept mass float32 [B], how many were kept int32 [B])."""
    code, (B, V), dev = _rows(logits, (2,))
    if uniforms is None:
        raise ValueError("uniforms must be a [B] tensor")
    one = (B,)
    if out_tokens is None:
        out_tokens = _like(uniforms, torch.int32, stream)
    if out_prob is None:
        out_prob = _like(uniforms, torch.float32, stream)
    if out_kept is None:
        out_kept = _like(uniforms, torch.int32, stream)
    st = (_lib or _library()).spec_sample_filtered(
        logits.data_ptr(), code, _ptr(uniforms, "uniforms", torch.float32, one, dev),
        *_settings(temperature, top_k, top_p, min_p, B, dev), B, V, _ptr(out_tokens, "out_tokens", torch.int32, one, dev),
        _ptr(out_prob, "out_prob", torch.float32, one, dev), _ptr(out_kept, "out_kept", torch.int32, one, dev),
        kv_cache._raw_stream(stream, dev))
    if st:
        _check(st, "spec_sample_filtered")
    return out_tokens, out_prob, out_kept


def spec_filter_logits(logits, temperature, top_k=None, top_p=None, min_p=None, n_rows=None, out=None, out_kept=None, stream=None):
    """``logits`` [B, S, V] (or [B, V]) with -inf for every token that the
    filters drop; returns (out, how many each row kept int32 [B, S] or [B]).
    ``n_rows`` [B] int32: how many of a sequence's S rows are real; the others
    are not written (kept 0).  ``out`` may be ``logits``."""
    code, shape, dev = _rows(logits, (2, 3))
    B, S, V = shape[0], shape[1] if len(shape) == 3 else 1, shape[-1]
    if out is None:
        out = _empty(logits, shape, logits.dtype, stream)
    if out_kept is None:
        out_kept = _empty(logits, shape[:-1], torch.int32, stream)
    st = (_lib or _library()).spec_filter_logits(
        logits.data_ptr(), code, *_settings(temperature, top_k, top_p, min_p, B, dev), B, S,
        _ptr(n_rows, "n_rows", torch.int32, (B,), dev), V, _ptr(out, "out", logits.dtype, shape, dev),
        _ptr(out_kept, "out_kept", torch.int32, shape[:-1], dev), kv_cache._raw_stream(stream, dev))
    if st:
        _check(st, "spec_filter_logits")
    return out, out_kept
