"""Binding of the cache's pages (argument marshalling only): reserving pages
for new tokens, with their slots, and giving pages back.

  page_table  [B, max_pages] int32; the first held[b] entries are sequence b's
  kv_len      [B] int32, each sequence's context length
  held        [B] int32, how many pages each sequence has
  free_pages  [capacity] int32, a stack: its first free_count entries are free
              pages, the last of them on top
  free_count  one int32

``held`` and ``free_count`` are updated in place, or left alone where
``held_out`` and ``free_count_out`` are given.  ``errors`` (an int32 CUDA
tensor of at least one element, zeroed once) gets bit 3 set when pages ran out,
bit 2 when a call met lengths or counts it cannot use; see
``include/specverify.h``.  A call's tensors (and its stream) are those of the
current device.  Every step runs in the CUDA library; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _check, _load, kv_cache

_P, _I32 = ctypes.c_void_p, ctypes.c_int32


class SVKvPool(ctypes.Structure):
    _fields_ = [("page_table", _P), ("held", _P), ("free_pages", _P), ("free_count", _P), ("B", _I32), ("max_pages", _I32),
                ("page_size", _I32), ("capacity", _I32)]


_PACK_POOL = struct.Struct("4P4i").pack
assert struct.calcsize("4P4i") == ctypes.sizeof(SVKvPool)

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _load()
        lib.spec_kv_reserve.argtypes = [_P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P]
        lib.spec_kv_release.argtypes = [_P, _P, _P, _P, _P, _P]
        lib.spec_kv_reserve.restype = lib.spec_kv_release.restype = ctypes.c_int
        _lib = lib
    return _lib


def _ptr(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of device `dev`, checked."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the page table and the current device are cuda:{dev}")
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _pool(page_table, kv_len, held, free_pages, free_count, page_size, held_out, free_count_out, errors):
    """The packed sv_kv_pool, the arguments both calls share, B and the device."""
    table, dev = page_table.shape, page_table.get_device()
    if dev < 0 or len(table) != 2:
        raise ValueError("page_table must be a CUDA tensor [B, max_pages]")
    if dev != kv_cache._current_device():   # the library launches on the current one
        raise ValueError(f"page_table is on cuda:{dev}, the current device is cuda:{kv_cache._current_device()}")
    B, i32 = table[0], torch.int32
    one, stack = (B,), free_pages.shape
    if len(stack) != 1:
        raise ValueError("free_pages must be [capacity]")
    if free_count.numel() != 1 or (free_count_out is not None and free_count_out.numel() != 1):
        raise ValueError("free_count must have one element")
    if errors is not None and errors.numel() < 1:
        raise ValueError("errors must have an element")
    hp = _ptr(held, "held", i32, one, dev)
    fp = _ptr(free_count, "free_count", i32, free_count.shape, dev)
    ho = hp if held_out is None else _ptr(held_out, "held_out", i32, one, dev)
    fo = fp if free_count_out is None else _ptr(free_count_out, "free_count_out", i32, free_count_out.shape, dev)
    p = _PACK_POOL(_ptr(page_table, "page_table", i32, table, dev), hp, _ptr(free_pages, "free_pages", i32, stack, dev), fp, B,
                   table[1], page_size, stack[0])
    ep = 0 if errors is None else _ptr(errors, "errors", i32, errors.shape, dev)
    return p, _ptr(kv_len, "kv_len", i32, one, dev), ho, fo, ep, B, dev


def spec_kv_reserve(page_table, kv_len, held, free_pages, free_count, page_size, S=None, n_new=None, row_start=None, slots=None,
                    held_out=None, free_count_out=None, errors=None, stream=None):
    """Pages for new tokens behind each sequence's context, from the stack into
    the page table; returns the new held counts.

    ``S`` tokens a sequence (``n_new`` [B]: how many of the S are real), or
    packed rows with ``row_start`` [B + 1].  ``slots`` int64 [B, S] (or [rows],
    packed; optional) receives each token's place in the cache,
    page * page_size + position within it; -1 for tokens that are not real and
    for sequences whose request the stack could not serve."""
    p, kv, ho, fo, ep, B, dev = _pool(page_table, kv_len, held, free_pages, free_count, page_size, held_out, free_count_out, errors)
    nn = starts = sp = rows = 0
    if row_start is None:
        if S is None or not 0 <= S <= 0x7fffffff:
            raise ValueError("S (tokens a sequence) or row_start must be given")
        if n_new is not None:
            nn = _ptr(n_new, "n_new", torch.int32, (B,), dev)
        rows = B * S
        if slots is not None:
            sp = _ptr(slots, "slots", torch.int64, (B, S), dev)
    else:
        if S is not None or n_new is not None:
            raise ValueError("packed rows (row_start) go without S and n_new")
        S = 0
        starts = _ptr(row_start, "row_start", torch.int32, (B + 1,), dev)
        if slots is None:
            rows = 0x7fffffff   # any: the starts alone say how many there are
        else:
            if slots.dim() != 1:
                raise ValueError("packed slots must be [rows]")
            rows = slots.shape[0]
            sp = _ptr(slots, "slots", torch.int64, slots.shape, dev)
    st = (_lib or _library()).spec_kv_reserve(p, kv, nn, starts, S, rows, ho, fo, sp, ep, kv_cache._raw_stream(stream, dev))
    if st:
        _check(st, "spec_kv_reserve")
    return held if held_out is None else held_out


def spec_kv_release(page_table, kv_len, held, free_pages, free_count, page_size, held_out=None, free_count_out=None, errors=None,
                    stream=None):
    """The pages behind each sequence's kv_len positions go back onto the stack
    (kv_len 0: all of them); returns the new held counts."""
    p, kv, ho, fo, ep, _, dev = _pool(page_table, kv_len, held, free_pages, free_count, page_size, held_out, free_count_out, errors)
    st = (_lib or _library()).spec_kv_release(p, kv, ho, fo, ep, kv_cache._raw_stream(stream, dev))
    if st:
        _check(st, "spec_kv_release")
    return held if held_out is None else held_out
