"""Thin ctypes binding over the C ABI in include/attn.h.

The attention step of a decode over a paged cache.  As in :mod:`.moe`, each
function carries the C entry point's name, checks types and devices, allocates
what the caller does not pass, and hands device pointers plus the current CUDA
stream to the library.  A serving loop makes one :func:`attn_cache` handle per
layer and keeps its workspaces; the calls then touch no allocator when every
output is passed.  The cache's device has to be the current one.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import moe as _moe
from .moe import DEV_TIMEOUT, MoeError, _check  # noqa: F401

BF16 = 0
FP16 = 1

DEV_BAD_PAGE = 32
DEV_BAD_LENGTH = 64

EXPORTS = (
    "attn_qk_norm_rope",
    "attn_tree_decode_workspace",
    "attn_tree_decode",
    "attn_cache_weights",
    "attn_cache_evict_workspace",
    "attn_cache_evict",
)

_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16}


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong), ("page_table", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_vp, _i, _ll, _d, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_double, ctypes.c_size_t
_cp = ctypes.POINTER(_CacheStruct)

_SIGS = {
    "attn_qk_norm_rope": (_i, [_vp, _vp, _vp, _ll, _ll, _ll, _vp, _vp, _vp, _i, _i, _vp, _vp, _d, _vp, _i, _i, _d,
                               _vp, _vp, _i, _cp, _vp, _vp]),
    "attn_tree_decode_workspace": (_sz, [_cp]),
    "attn_tree_decode": (_i, [_vp, _ll, _vp, _vp, _i, _i, _vp, _i, _d, _cp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "attn_cache_weights": (_i, [_vp, _ll, _vp, _vp, _vp, _i, _i, _vp, _i, _d, _cp, _vp, _d, _vp, _i, _vp, _vp]),
    "attn_cache_evict_workspace": (_sz, [_cp, _i]),
    "attn_cache_evict": (_i, [_cp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
}

_LIB = None


def load():
    """The library of :func:`.moe.load` with this module's signatures set."""
    global _LIB
    if _LIB is None:
        lib = _moe.load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


class AttnCache:
    """Handle of a paged cache: the C description plus the tensors it points
    into, which it keeps alive."""

    def __init__(self, k, v, page_table):
        self.k, self.v, self.page_table = k, v, page_table
        pages, heads, size, dim = k.shape
        sp, sh, sr, _ = k.stride()
        self.batch, self.kv_heads, self.head_dim = page_table.shape[0], heads, dim
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self.lens_shape, self.cu_shape = (self.batch,), (self.batch + 1,)
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), sp, sh, sr, page_table.data_ptr(), page_table.shape[0],
                                   page_table.shape[1], pages, size, heads, dim, _DTYPES[k.dtype])
        self.ref = ctypes.byref(self.struct)


def attn_cache(k, v, page_table) -> AttnCache:
    """Describes a cache.  k, v [pages, kv_heads, page_size, D]: any strides
    with D contiguous, the same for both (a [pages, page_size, kv_heads, D]
    cache is passed as its transposed view); page_table [batch, max_pages]
    int32."""
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise MoeError(f"{name} must be a CUDA tensor")
        if t.dim() != 4 or t.dtype not in _DTYPES or t.stride(3) != 1:
            raise MoeError(f"{name} must be [pages, kv_heads, page_size, D] of bfloat16 or float16, D contiguous")
    if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.device != v.device:
        raise MoeError("k and v must have the same shape, strides, type and device")
    _moe._cuda(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.device != k.device:
        raise MoeError("page_table must be [batch, max_pages] on the cache's device")
    _fit(batch=page_table.shape[0], max_pages=page_table.shape[1], pages=k.shape[0], kv_heads=k.shape[1],
         page_size=k.shape[2], head_dim=k.shape[3])
    return AttnCache(k, v, page_table)


# The checks below run on every call of a decode step, so each is a handful of
# attribute reads; the words for a refusal are only put together when there is
# one.

_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_i32, _i64, _f32, _f64, _u8 = torch.int32, torch.int64, torch.float32, torch.float64, torch.uint8


def _on(stream, cache):
    """Handle of the stream to launch on.  A launch goes to the device that is
    current: any other than the cache's is refused, before anything else is done."""
    index = cache.index
    if _current() != index:
        raise MoeError(f"the cache is on {cache.device}, cuda:{_current()} is current")
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise MoeError(f"the cache is on {cache.device}, the stream on cuda:{stream.device_index}")
    return stream.cuda_stream


def _rows(t, name, heads, cache):
    """Token stride of a [tokens, heads, D] tensor whose heads and elements are
    contiguous (heads None: any number)."""
    try:
        T, h, D = t.shape
        st, sh, sd = t.stride()
        if (t.dtype is cache.dtype and t.get_device() == cache.index and D == cache.head_dim
                and (heads is None or h == heads) and sd == 1 and (h == 1 or sh == D)):
            # the stride of one token is of no account; a packed one satisfies the checks
            return st if T > 1 else h * D
    except (AttributeError, TypeError, ValueError):
        pass
    raise MoeError(f"{name} must be a [tokens, {heads or 'heads'}, {cache.head_dim}] tensor of {cache.dtype} on "
                   f"{cache.device}, heads and elements contiguous")


def _array(t, name, shape, dtype, cache):
    """Address of a contiguous tensor of just this shape and type."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == cache.index:
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    raise MoeError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {cache.device}")


def _size(t, name):
    """Elements of the last axis of a tensor whose shape is checked later."""
    try:
        return t.shape[-1]
    except (AttributeError, IndexError):
        pass
    raise MoeError(f"{name} must be a tensor with a shape")


def _tree(tree, tokens, cache):
    """tree [tokens, words] int64: bit j % 64 of word j // 64 of a row is set
    if the token sees draft j of its sequence."""
    if tree is None:
        return None, 0
    words = _size(tree, "tree")
    if len(tree.shape) != 2 or words == 0:
        raise MoeError("tree must be [tokens, words], of one word or more")
    at = _array(tree, "tree", (tokens, words), _i64, cache)
    return (at, words) if tokens else (None, 0)


_MOST = (1 << 31) - 1


def _fit(**sizes):
    """ctypes drops what passes 32 bits without a word."""
    for name, x in sizes.items():
        if not 0 <= x <= _MOST:
            raise MoeError(f"{name} must be 0 to 2^31 - 1, got {x}")


def _status(dev_status, cache):
    return None if dev_status is None else _array(dev_status, "dev_status", (1,), _i32, cache)


def _elsewhere(stream):
    """Context for allocating on the stream the call runs on, so that the
    allocator never hands the memory to another stream while the call uses it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


_HERE = contextlib.nullcontext()
_empty = torch.empty


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def attn_qk_norm_rope(q, k, v, pos, cu, lens, cache: AttnCache, inv_freq, q_weight=None, k_weight=None,
                      eps: float = 1e-6, interleaved: bool = False, magnitude: float = 1.0, slot_pos=None, q_out=None,
                      dev_status=None, stream=None):
    """Head norm and rotation of q and k, append of k and v.  inv_freq [rot /
    2] FP64: radians per position.  Returns q_out [tokens, q_heads, D]."""
    on = _on(stream, cache)
    sq, sk, sv = _rows(q, "q", None, cache), _rows(k, "k", cache.kv_heads, cache), _rows(v, "v", cache.kv_heads, cache)
    T, hq, D = q.shape
    if k.shape[0] != T or v.shape[0] != T:
        raise MoeError("q, k and v must hold the same tokens")
    half = _size(inv_freq, "inv_freq")
    if q_weight is None and k_weight is None:
        wq = wk = None
    else:
        wq = _array(q_weight, "q_weight", (D,), cache.dtype, cache)
        wk = _array(k_weight, "k_weight", (D,), cache.dtype, cache)
    at, cap = None, 0
    if slot_pos is not None:
        cap = _size(slot_pos, "slot_pos")
        if cap > _MOST:
            _fit(slot_cap=cap)
        at = _array(slot_pos, "slot_pos", (cache.batch, cache.kv_heads, cap), _i32, cache)
    if q_out is None:
        with _elsewhere(stream):
            q_out = _empty((T, hq, D), dtype=cache.dtype, device=cache.device)
        to = q_out.data_ptr()
    else:
        to = _array(q_out, "q_out", (T, hq, D), cache.dtype, cache)
    rc = (_LIB or load()).attn_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), sq, sk, sv, _array(pos, "pos", (T,), _i32, cache),
        _array(cu, "cu", cache.cu_shape, _i32, cache), _array(lens, "lens", cache.lens_shape, _i32, cache),
        T, hq, wq, wk, eps, _array(inv_freq, "inv_freq", (half,), _f64, cache), 2 * half, interleaved,
        magnitude, to, at, cap, cache.ref,
        _status(dev_status, cache), on)
    if rc:
        _check(rc, "attn_qk_norm_rope")
    return q_out


def attn_tree_decode_workspace(cache: AttnCache):
    """A workspace for :func:`attn_tree_decode` on the cache's device."""
    with torch.cuda.device(cache.device):
        n = int(load().attn_tree_decode_workspace(cache.ref))
    if n == 0:
        raise MoeError("attn_tree_decode does not support this cache")
    return torch.empty(n, dtype=_u8, device=cache.device)


def attn_tree_decode(q, cu, lens, cache: AttnCache, tree=None, scale: float | None = None, out=None, lse=None,
                     workspace=None, dev_status=None, stream=None):
    """Attention of the tokens in flight over the cache; tree = None: a chain.
    Returns (out [tokens, q_heads, D], lse [tokens, q_heads])."""
    on = _on(stream, cache)
    sq = _rows(q, "q", None, cache)
    T, hq, D = q.shape
    words, count = _tree(tree, T, cache)
    if out is None or lse is None or workspace is None:
        with _elsewhere(stream):
            if out is None:
                out = _empty((T, hq, D), dtype=cache.dtype, device=cache.device)
            if lse is None:
                lse = _empty((T, hq), dtype=_f32, device=cache.device)
            if workspace is None:
                workspace = attn_tree_decode_workspace(cache)
    size = _size(workspace, "workspace")
    rc = (_LIB or load()).attn_tree_decode(
        q.data_ptr(), sq, _array(cu, "cu", cache.cu_shape, _i32, cache),
        _array(lens, "lens", cache.lens_shape, _i32, cache), T, hq, words, count,
        D ** -0.5 if scale is None else scale, cache.ref, _array(out, "out", (T, hq, D), cache.dtype, cache),
        _array(lse, "lse", (T, hq), _f32, cache),
        _array(workspace, "workspace", (size,), _u8, cache), size, _status(dev_status, cache), on)
    if rc:
        _check(rc, "attn_tree_decode")
    return out, lse


def attn_cache_weights(q, lse, cu, lens, cache: AttnCache, acc, tree=None, scale: float | None = None,
                       decay: float = 1.0, acc_out=None, dev_status=None, stream=None):
    """acc_out = decay * acc + the softmax weight each slot received.  acc
    [batch, kv_heads, slot_cap]; acc_out may be acc; entries past a sequence's
    end are not written (a new acc_out starts as zeros)."""
    on = _on(stream, cache)
    sq = _rows(q, "q", None, cache)
    T, hq, D = q.shape
    words, count = _tree(tree, T, cache)
    shape = (cache.batch, cache.kv_heads, _size(acc, "acc"))
    if shape[2] > _MOST:
        _fit(slot_cap=shape[2])
    if acc_out is None:
        with _elsewhere(stream):
            acc_out = torch.zeros(shape, dtype=_f32, device=cache.device)
    rc = (_LIB or load()).attn_cache_weights(
        q.data_ptr(), sq, _array(lse, "lse", (T, hq), _f32, cache),
        _array(cu, "cu", cache.cu_shape, _i32, cache), _array(lens, "lens", cache.lens_shape, _i32, cache),
        T, hq, words, count, D ** -0.5 if scale is None else scale, cache.ref,
        _array(acc, "acc", shape, _f32, cache), decay, _array(acc_out, "acc_out", shape, _f32, cache),
        shape[2], _status(dev_status, cache), on)
    if rc:
        _check(rc, "attn_cache_weights")
    return acc_out


def attn_cache_evict_workspace(cache: AttnCache, budget: int):
    """A workspace for :func:`attn_cache_evict` with this budget."""
    _fit(budget=budget)
    n = int(load().attn_cache_evict_workspace(cache.ref, budget))
    if n == 0:
        raise MoeError("attn_cache_evict does not support this cache or budget")
    return torch.empty(n, dtype=_u8, device=cache.device)


def attn_cache_evict(cache: AttnCache, acc, slot_pos, lens, next_pos, budget: int, sinks: int = 0, recent: int = 0,
                     acc_out=None, pos_out=None, lens_out=None, workspace=None, dev_status=None, stream=None):
    """Keeps the `budget` slots of each sequence and KV head with the most
    weight and moves their rows below the budget, in place.  Returns
    (lens_out, acc_out, pos_out)."""
    on = _on(stream, cache)
    shape = (cache.batch, cache.kv_heads, _size(acc, "acc"))
    if not (shape[2] <= _MOST and 0 <= budget <= _MOST and 0 <= sinks <= _MOST and 0 <= recent <= _MOST):
        _fit(slot_cap=shape[2], budget=budget, sinks=sinks, recent=recent)
    if acc_out is None or pos_out is None or lens_out is None or workspace is None:
        with _elsewhere(stream):
            if acc_out is None:
                acc_out = torch.zeros(shape, dtype=_f32, device=cache.device)
            if pos_out is None:
                pos_out = torch.zeros(shape, dtype=_i32, device=cache.device)
            if lens_out is None:
                lens_out = _empty(cache.lens_shape, dtype=_i32, device=cache.device)
            if workspace is None:
                workspace = attn_cache_evict_workspace(cache, budget)
    size = _size(workspace, "workspace")
    rc = (_LIB or load()).attn_cache_evict(
        cache.ref, _array(acc, "acc", shape, _f32, cache), _array(slot_pos, "slot_pos", shape, _i32, cache),
        shape[2], _array(lens, "lens", cache.lens_shape, _i32, cache),
        _array(next_pos, "next_pos", cache.lens_shape, _i32, cache), budget, sinks, recent,
        _array(acc_out, "acc_out", shape, _f32, cache), _array(pos_out, "pos_out", shape, _i32, cache),
        _array(lens_out, "lens_out", cache.lens_shape, _i32, cache),
        _array(workspace, "workspace", (size,), _u8, cache), size, _status(dev_status, cache), on)
    if rc:
        _check(rc, "attn_cache_evict")
    return lens_out, acc_out, pos_out
