"""Binding of the paged key/value cache operators (argument marshalling only).

``spec_kv_append`` -> ``spec_tree_attention`` -> verification ->
``spec_kv_commit`` is one decode step over a tree of drafted tokens;
``spec_kv_read`` returns ranges of the cache.  Shapes, as in
``include/specverify.h``:

  k_cache, v_cache   [num_pages, n_kv_heads, page_size, head_dim], bfloat16 or
                     float8_e4m3fn, contiguous (a layer's slice of a
                     [layers, ...] tensor is)
  k_scale, v_scale   [num_pages, n_kv_heads, page_size] float32 with
                     float8_e4m3fn caches, None with bfloat16
  page_table         [B, max_pages] int32
  kv_len             [B] int32, each sequence's context length

``errors`` (an int32 CUDA tensor of at least one element, zeroed once) gets
bit 2 set when a call met unusable device data; see the header for what the
outputs then hold.  A call's tensors (and its stream) are those of the current
device.  Every step runs in the CUDA library; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import SV_DTYPE_BF16, SV_DTYPE_F32, _check, _load

SV_KV_BF16 = 0
SV_KV_E4M3 = 1
SV_ATTENTION_WAITS = 14

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class SVKvCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("page_table", _P),
                ("max_pages", _I32), ("format", _I32), ("layers", _I32), ("num_pages", _I32),
                ("n_kv_heads", _I32), ("page_size", _I32), ("head_dim", _I32)]


class SVKvTokens(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("q_stride", _I64), ("k_stride", _I64),
                ("v_stride", _I64), ("q_norm", _P), ("k_norm", _P), ("cos_sin", _P), ("parent", _P),
                ("n_new", _P), ("row_start", _P), ("q_out", _P), ("dtype", _I32), ("n_heads", _I32),
                ("B", _I32), ("S", _I32), ("rows", _I32), ("max_positions", _I32),
                ("rotary_dim", _I32), ("interleaved", _I32), ("eps", ctypes.c_float)]


# The calls pass the two structs as packed bytes: one call packs what would be a
# dozen attribute assignments, which at the smallest shapes cost more than the
# kernels run.
_PACK_CACHE = struct.Struct("5P7i4x").pack
_PACK_TOKENS = struct.Struct("3P3q7P8if4x").pack
assert struct.calcsize("5P7i4x") == ctypes.sizeof(SVKvCache)
assert struct.calcsize("3P3q7P8if4x") == ctypes.sizeof(SVKvTokens)

_lib = None
_workspace_sizes: dict = {}


def _library():
    global _lib
    if _lib is None:
        lib = _load()
        lib.spec_kv_append.argtypes = [_P, _P, _P, _P, _P]
        lib.spec_tree_attention.argtypes = [_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32,
                                            ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]
        lib.spec_tree_attention_ex.argtypes = [*lib.spec_tree_attention.argtypes[:-1], ctypes.c_uint32, _P]
        lib.spec_kv_commit.argtypes = [_P, _P, _P, _P, _I32, _I32, _P, _P, _P]
        lib.spec_kv_read.argtypes = [_P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P]
        for f in (lib.spec_kv_append, lib.spec_tree_attention, lib.spec_tree_attention_ex, lib.spec_kv_commit,
                  lib.spec_kv_read):
            f.restype = ctypes.c_int
        lib.sv_attention_workspace_size.argtypes = [_I32, _I32, _I32, _I32]
        lib.sv_attention_workspace_size.restype = ctypes.c_size_t
        _lib = lib
    return _lib


def _refuse(t, name, dtype, shape, dev):
    """The exception for a tensor that _ptr does not take."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    _same_device(t, name, dev)
    raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _same_device(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the cache and the current device are cuda:{dev}")


def _ptr(t, name, dtype, shape, dev):
    """The address of an optional contiguous tensor of device `dev`, checked."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _errors_ptr(errors, dev):
    if errors is None:
        return 0
    if errors.numel() < 1:
        raise ValueError("errors must have an element")
    return _ptr(errors, "errors", torch.int32, errors.shape, dev)


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, layered=False):
    """The packed sv_kv_cache, the cache's shape, the table's batch and the device."""
    shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.get_device()
    if dev < 0:
        raise ValueError("k_cache must be a contiguous CUDA tensor")
    if dev != _current_device():   # the library launches on the current one
        raise ValueError(f"k_cache is on cuda:{dev}, the current device is cuda:{_current_device()}")
    n = len(shape)
    if n != 4 and not (layered and n == 5):
        raise ValueError("k_cache must be [num_pages, n_kv_heads, page_size, head_dim]"
                         + (" or [layers, ...]" if layered else ""))
    ks = vs = 0
    if dtype is torch.bfloat16:
        code = SV_KV_BF16
        if k_scale is not None or v_scale is not None:
            raise ValueError("bfloat16 caches have no scales")
    elif dtype is torch.float8_e4m3fn:
        code = SV_KV_E4M3
        if k_scale is None or v_scale is None:
            raise ValueError("float8_e4m3fn caches need k_scale and v_scale")
        rows = shape[:-1]
        ks = _ptr(k_scale, "k_scale", torch.float32, rows, dev)
        vs = _ptr(v_scale, "v_scale", torch.float32, rows, dev)
    else:
        raise TypeError(f"the cache must be bfloat16 or float8_e4m3fn, got {dtype}")
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    return _PACK_CACHE(_ptr(k_cache, "k_cache", dtype, shape, dev), _ptr(v_cache, "v_cache", dtype, shape, dev), ks, vs,
                       _ptr(page_table, "page_table", torch.int32, table, dev), table[1], code,
                       shape[0] if n == 5 else 1, *shape[-4:-2], *shape[-2:]), shape, table[0], dev


def _heads(t, name, dtype, lead, dev):
    """Address, token stride and head count of [*lead, heads, head_dim] rows
    whose heads are adjacent (tokens may be strided, evenly)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    n = len(lead)
    if (not t.is_cuda or len(shape) != n + 2 or shape[:n] != lead or st[-1] != 1
            or (shape[-2] > 1 and st[-2] != shape[-1])):
        raise ValueError(f"{name} must be a CUDA tensor {list(lead)} + [heads, head_dim] with contiguous heads")
    if t.get_device() != dev:
        _same_device(t, name, dev)
    if n == 2:
        if lead[0] > 1 and lead[1] > 1 and st[0] != lead[1] * st[1]:
            raise ValueError(f"{name}'s tokens must be evenly strided")
        return t.data_ptr(), st[1] if lead[1] > 1 else st[0], shape[-2]
    return t.data_ptr(), st[0], shape[-2]


def _code(dtype):
    if dtype is torch.bfloat16:
        return SV_DTYPE_BF16
    if dtype is torch.float32:
        return SV_DTYPE_F32
    raise TypeError(f"rows must be float32 or bfloat16, got {dtype}")


# the current device, and its current stream's handle without a Stream object around it
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, dev):
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError(f"the stream is of cuda:{stream.device_index}, the cache and the current device are cuda:{dev}")
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _empty(like, shape, dtype, stream):
    """A new tensor that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def spec_kv_append(k, v, k_cache, v_cache, page_table, kv_len, n_new=None, q=None, q_norm=None, k_norm=None,
                   eps=1e-6, cos_sin=None, interleaved=False, parent=None, row_start=None, k_scale=None,
                   v_scale=None, q_out=None, errors=None, stream=None):
    """Write new tokens' keys and values behind each sequence's context, with
    the heads' norms and the position rotation of queries and keys in the same
    pass; returns the queries (None without ``q``).

    k, v: [B, S, n_kv_heads, head_dim] (``n_new`` [B]: how many of the S are
    real; ``parent`` [B, S]: they are a tree's nodes), or with ``row_start``
    [B + 1] packed rows [rows, n_kv_heads, head_dim]; q likewise with its
    heads.  Tokens may be strided: slices of one fused projection work as they
    are.  ``cos_sin`` [max_positions, rotary_dim] float32 holds each position's
    cosines, then its sines."""
    c, cache, B, dev = _cache(k_cache, v_cache, k_scale, v_scale, page_table)
    dtype, D = k.dtype, cache[-1]
    code = _code(dtype)
    S = nn = par = starts = 0
    if row_start is None:
        if k.dim() != 4 or k.shape[0] != B:
            raise ValueError("k must be [B, S, n_kv_heads, head_dim]")
        S = k.shape[1]
        lead, rows = (B, S), B * S
        nn = _ptr(n_new, "n_new", torch.int32, (B,), dev)
        par = _ptr(parent, "parent", torch.int32, lead, dev)
    else:
        if k.dim() != 3 or n_new is not None or parent is not None:
            raise ValueError("packed k must be [rows, n_kv_heads, head_dim], without n_new and parent")
        rows = k.shape[0]
        lead = (rows,)
        starts = _ptr(row_start, "row_start", torch.int32, (B + 1,), dev)
    kp, k_stride, hk = _heads(k, "k", dtype, lead, dev)
    vp, v_stride, hv = _heads(v, "v", dtype, lead, dev)
    if hk != cache[-3] or hv != hk or k.shape[-1] != D or v.shape[-1] != D:
        raise ValueError("k and v must have the cache's heads and head_dim")
    qp = q_stride = hq = op = qn = kn = cs = positions = rot = 0
    if q is not None:
        qp, q_stride, hq = _heads(q, "q", dtype, lead, dev)
        if q.shape[-1] != D:
            raise ValueError("q must have the cache's head_dim")
        if q_out is None:
            q_out = _empty(q, q.shape, dtype, stream)
            op = q_out.data_ptr()
        else:
            op = _ptr(q_out, "q_out", dtype, q.shape, dev)
        qn = _ptr(q_norm, "q_norm", dtype, (D,), dev)
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm go with q")
    kn = _ptr(k_norm, "k_norm", dtype, (D,), dev)
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_positions, rotary_dim]")
        positions, rot = cos_sin.shape
        cs = _ptr(cos_sin, "cos_sin", torch.float32, (positions, rot), dev)
    t = _PACK_TOKENS(qp, kp, vp, q_stride, k_stride, v_stride, qn, kn, cs, par, nn, starts, op, code, hq, B, S,
                     rows, positions, rot, 1 if interleaved else 0, eps)
    st = (_lib or _library()).spec_kv_append(c, t, _ptr(kv_len, "kv_len", torch.int32, (B,), dev), _errors_ptr(errors, dev),
                                             _raw_stream(stream, dev))
    if st:
        _check(st, "spec_kv_append")
    return q_out


def sv_attention_workspace_size(Nmax: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(_library().sv_attention_workspace_size(int(Nmax), int(n_heads), int(n_kv_heads), int(head_dim)))


def spec_tree_attention(q, k_cache, v_cache, page_table, kv_len, n_nodes=None, parent=None, scale=None,
                        k_scale=None, v_scale=None, out=None, workspace=None, errors=None, stream=None,
                        expire_waits=0):
    """Attention of each sequence's tree nodes, q [B, Nmax, n_heads, head_dim]
    (bfloat16; tokens may be strided), to its context and their ancestors;
    returns out of q's shape, zeros past ``n_nodes``.  ``parent`` None is the
    chain; Nmax = 1 an ordinary decode step.  ``scale`` defaults to
    head_dim ** -0.5.  ``workspace``: a uint8 CUDA tensor of at least
    sv_attention_workspace_size bytes (allocated when omitted).
    ``expire_waits`` (testing only): bits of SV_ATTENTION_WAITS kinds of waits
    inside the kernel that are made to run out, to exercise the timeout path."""
    c, cache, B, dev = _cache(k_cache, v_cache, k_scale, v_scale, page_table)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, Nmax, n_heads, head_dim]")
    _, Nmax, Hq, D = shape
    if B != shape[0] or D != cache[-1]:
        raise ValueError("q must have the page table's B and the cache's head_dim")
    dtype = q.dtype
    code = _code(dtype)
    qp, q_stride, _ = _heads(q, "q", dtype, (B, Nmax), dev)
    lib = _lib or _library()
    if out is None:
        out = _empty(q, shape, dtype, stream)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dtype, shape, dev)
    if workspace is None:
        key = (Nmax, Hq, cache[-3], D)
        need = _workspace_sizes.get(key)
        if need is None:
            need = _workspace_sizes[key] = max(256, lib.sv_attention_workspace_size(*key))
        workspace = _empty(q, need, torch.uint8, stream)
        wp = workspace.data_ptr()
    else:
        need = workspace.numel()
        wp = _ptr(workspace, "workspace", torch.uint8, workspace.shape, dev)
    st = lib.spec_tree_attention_ex(c, _ptr(kv_len, "kv_len", torch.int32, (B,), dev),
                                    _ptr(n_nodes, "n_nodes", torch.int32, (B,), dev),
                                    _ptr(parent, "parent", torch.int32, (B, Nmax), dev), qp, q_stride, code, Hq, B,
                                    Nmax, D ** -0.5 if scale is None else scale, op, _errors_ptr(errors, dev), wp, need,
                                    expire_waits, _raw_stream(stream, dev))
    if st:
        _check(st, "spec_tree_attention")
    return out


def spec_kv_commit(k_cache, v_cache, page_table, kv_len, out_path, out_len, k_scale=None, v_scale=None,
                   kv_len_out=None, errors=None, stream=None):
    """Move the kept path of each verified tree (out_path [B, Nmax] and out_len
    [B] of spec_verify_tree) behind its root, in every layer of the caches
    ([layers, num_pages, ...], or one layer's [num_pages, ...]), and return the
    lengths kv_len + 1 + out_len: in ``kv_len`` itself, or in ``kv_len_out``."""
    c, _, B, dev = _cache(k_cache, v_cache, k_scale, v_scale, page_table, layered=True)
    path = out_path.shape
    if len(path) != 2:
        raise ValueError("out_path must be [B, Nmax]")
    Nmax, one = path[1], (B,)
    if kv_len_out is None:
        kv_len_out = kv_len
    st = (_lib or _library()).spec_kv_commit(c, _ptr(kv_len, "kv_len", torch.int32, one, dev),
                                             _ptr(out_path, "out_path", torch.int32, (B, Nmax), dev),
                                             _ptr(out_len, "out_len", torch.int32, one, dev), B, Nmax,
                                             _ptr(kv_len_out, "kv_len_out", torch.int32, one, dev),
                                             _errors_ptr(errors, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "spec_kv_commit")
    return kv_len_out


def spec_kv_read(k_cache, v_cache, page_table, start, row_start, rows, dtype=torch.bfloat16, k_scale=None,
                 v_scale=None, k_out=None, v_out=None, errors=None, stream=None):
    """The entries of sequence b at positions start[b], start[b] + 1, ... as the
    dense rows row_start[b] .. row_start[b + 1] - 1 of (k_out, v_out)
    [rows, n_kv_heads, head_dim]; rows of no sequence are zeros."""
    c, cache, B, dev = _cache(k_cache, v_cache, k_scale, v_scale, page_table)
    rows = int(rows)
    shape = (rows, cache[-3], cache[-1])
    code = _code(dtype)
    if k_out is None:
        k_out = _empty(k_cache, shape, dtype, stream)
    if v_out is None:
        v_out = _empty(k_cache, shape, dtype, stream)
    st = (_lib or _library()).spec_kv_read(c, _ptr(start, "start", torch.int32, (B,), dev),
                                           _ptr(row_start, "row_start", torch.int32, (B + 1,), dev), B, rows, code,
                                           _ptr(k_out, "k_out", dtype, shape, dev), _ptr(v_out, "v_out", dtype, shape, dev),
                                           _errors_ptr(errors, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "spec_kv_read")
    return k_out, v_out
