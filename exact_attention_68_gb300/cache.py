"""ctypes binding to the C ABI of include/attn_cache.h (argument marshalling only).

An 8-bit key/value cache in pages and the operators on it, beside
``binding.attn_fwd``: ``cache_append`` stores the step's new keys and values,
``cache_fwd`` is the attention of the new tokens' queries over the cache,
``cache_select`` picks the pages a long context's heads should read and
``cache_evict`` keeps each head's most attended tokens.  The meaning of every
argument, the layout and the errors are those of the header; tensors are
checked here, all arithmetic runs in the CUDA library, and there is no fallback.

    cache = cache_alloc(pages=4096, heads=8, head_dim=128)
    cache_append(cache, k, v, table, lens)            # lens counts the new tokens
    out, lse = cache_fwd(q, cache, table, lens)       # q [B, Hq, T, D]
    pages, scores = cache_select(q, cache, table, lens, count=64)
    out, lse = cache_fwd(q, cache, table, lens, pages=pages)
    kept, new_lens, new_mass = cache_evict(cache, mass, table, lens, dst_table, keep=4096, recent=256)

Nothing synchronises.  A workspace is allocated per call unless one is passed;
calls that may run at the same time, and graphs, need one each.  With ``stream``,
what a call allocates belongs to that stream, as if it were the current one.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import NamedTuple

import torch

from .binding import (ATTN_BF16, ATTN_DEFAULT_WAIT_TIMEOUT_NS, ATTN_ERR_INVALID_ARG, ATTN_F16, ATTN_OK, AttnError,
                      load_library)

__all__ = ["KVCache8", "cache_alloc", "cache_append", "cache_fwd", "cache_select", "cache_evict",
           "cache_fwd_workspace", "cache_evict_workspace", "CACHE_MAX_TOKENS", "CACHE_SYMBOLS"]

CACHE_MAX_TOKENS = 64
_PAGE_SIZES = (16, 32, 64)
_NO_SPACE = 16  # the size that says no workspace is needed

_i64, _p, _f, _i, _u64, _sz = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_uint64,
                               ctypes.c_size_t)


class _Cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("k_bounds", _p), ("pages", _i64),
                ("heads", _i64), ("head_dim", _i64), ("page", _i64)]


class _Seqs(ctypes.Structure):
    _fields_ = [("table", _p), ("lens", _p), ("fresh", _p), ("batch", _i64), ("width", _i64)]


_c, _s = ctypes.POINTER(_Cache), ctypes.POINTER(_Seqs)
_SIGS = {
    "attn_cache_append": (_i, [_c, _s, _p, _p, _i64, _i, _p]),
    "attn_cache_fwd_workspace": (_sz, [_c, _s, _i64, _i64, _i64, _i]),
    "attn_cache_fwd": (_i, [_c, _s, _p, _p, _i64, _p, _p, _p, _i64, _i64, _f, _i, _p, _sz, _u64, _p]),
    "attn_cache_select": (_i, [_c, _s, _p, _i64, _i64, _i, _i64, _p, _p, _p]),
    "attn_cache_evict_workspace": (_sz, [_c, _s, _i64]),
    "attn_cache_evict": (_i, [_c, _s, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _sz, _p]),
}
CACHE_SYMBOLS = tuple(_SIGS)

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}
_lib = None
_lock = threading.Lock()


def declare(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the signatures of the cache's entry points on a loaded library."""
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                _lib = declare(load_library())
    return _lib


class KVCache8(NamedTuple):
    """A pool of pages; the tensors are the user's own (see include/attn_cache.h).

    k, v uint8 [pages, heads, page, pitch] (e4m3 codes), k_scale, v_scale fp32
    [pages, heads], k_bounds int8 [pages, heads, 2, pitch]; pitch is head_dim
    rounded up to a multiple of 16.
    """
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_bounds: torch.Tensor
    head_dim: int


def cache_alloc(pages: int, heads: int, head_dim: int, page: int = 64, device="cuda") -> KVCache8:
    """A pool of empty pages (codes and bounds zero, scales one)."""
    if page not in _PAGE_SIZES:
        raise ValueError(f"page must be one of {_PAGE_SIZES}")
    if pages < 1 or heads < 1 or head_dim < 8 or head_dim > 256 or head_dim % 8:
        raise ValueError("pages and heads must be positive, head_dim a multiple of 8 up to 256")
    pitch = (head_dim + 15) // 16 * 16
    codes = [torch.zeros((pages, heads, page, pitch), dtype=torch.uint8, device=device) for _ in "kv"]
    scales = [torch.ones((pages, heads), dtype=torch.float32, device=device) for _ in "kv"]
    return KVCache8(*codes, *scales, torch.zeros((pages, heads, 2, pitch), dtype=torch.int8, device=device), head_dim)


def _want(name, t, dtype, shape, device):
    """The address of a tensor that has to be just so."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


_u8, _i8, _i32, _f32 = torch.uint8, torch.int8, torch.int32, torch.float32


def _views(cache, table, lens, fresh):
    """The C structures of a pool and a call's sequences, checked; the device, and
    (heads, head_dim, page, batch, width)."""
    k, v, k_scale, v_scale, k_bounds, head_dim = cache
    try:
        dev, at, shape = k.device, k.get_device(), k.shape
        pages, heads, page, pitch = shape
        batch, width = table.shape
        # everything in one condition: this is much of a small call's time
        if (at < 0 or pitch != (head_dim + 15) // 16 * 16
                or k.dtype is not _u8 or not k.is_contiguous()
                or v.dtype is not _u8 or v.shape != shape or not v.is_contiguous() or v.get_device() != at
                or k_scale.dtype is not _f32 or k_scale.shape != (pages, heads) or not k_scale.is_contiguous()
                or k_scale.get_device() != at
                or v_scale.dtype is not _f32 or v_scale.shape != (pages, heads) or not v_scale.is_contiguous()
                or v_scale.get_device() != at
                or k_bounds.dtype is not _i8 or k_bounds.shape != (pages, heads, 2, pitch)
                or not k_bounds.is_contiguous() or k_bounds.get_device() != at
                or table.dtype is not _i32 or not table.is_contiguous() or table.get_device() != at
                or lens.dtype is not _i32 or lens.shape != (batch,) or not lens.is_contiguous()
                or lens.get_device() != at):
            _refuse(cache, table, lens)
        fresh_p = None if fresh is None else _want("fresh", fresh, _i32, (batch,), dev)
        return (_Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_bounds.data_ptr(),
                       pages, heads, head_dim, page),
                _Seqs(table.data_ptr(), lens.data_ptr(), fresh_p, batch, width), dev,
                heads, head_dim, page, batch, width)
    except (AttributeError, ValueError):
        _refuse(cache, table, lens)
        raise


def _refuse(cache, table, lens):
    """Names what _views found wrong, one tensor after the other."""
    k, v, k_scale, v_scale, k_bounds, head_dim = cache
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise TypeError("the cache must be CUDA tensors")
    if k.dim() != 4:
        raise ValueError("cache.k must be [pages, heads, page, pitch]")
    dev, (pages, heads, page, pitch) = k.device, k.shape
    if pitch != (head_dim + 15) // 16 * 16:
        raise ValueError("the cache's rows must be head_dim rounded up to a multiple of 16")
    _want("cache.k", k, _u8, k.shape, dev)
    _want("cache.v", v, _u8, k.shape, dev)
    _want("cache.k_scale", k_scale, _f32, (pages, heads), dev)
    _want("cache.v_scale", v_scale, _f32, (pages, heads), dev)
    _want("cache.k_bounds", k_bounds, _i8, (pages, heads, 2, pitch), dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 [batch, width] tensor")
    _want("table", table, _i32, table.shape, dev)
    _want("lens", lens, _i32, (table.shape[0],), dev)


def _rows(name, t, batch, head_dim, dev):
    """A contiguous 16-bit [batch, heads, T, head_dim] tensor: its dtype code, heads and T."""
    dt = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dt is None:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    shape = t.shape
    if len(shape) != 4 or shape[0] != batch or shape[3] != head_dim or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous [{batch}, heads, T, {head_dim}] tensor on {dev}")
    return dt, shape[1], shape[2]


# the current device and its current stream's handle, without the objects
# torch.cuda.current_stream makes on the way
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name, dev, stream, *args):
    """The entry point on `stream` (default: the current one) of `dev`."""
    index = dev.index
    if stream is not None:
        st = stream.cuda_stream
    elif _raw_stream is not None:
        st = _raw_stream(index)
    else:
        st = torch.cuda.current_stream(dev).cuda_stream
    fn = getattr(_lib or _library(), name)
    if index == _current_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, st)
    if rc != ATTN_OK:
        raise AttnError(rc, name)


def _size(name, dev, *args):
    fn = getattr(_lib or _library(), name)
    if dev.index == _current_device():
        n = fn(*args)
    else:
        with torch.cuda.device(dev):
            n = fn(*args)
    if n == 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, name)
    return n


def _new(stream, dev, shape, dtype):
    """Memory for a call on `stream`, from that stream's pool: no work of another
    stream can still be using it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _space(workspace, dev):
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    if not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be contiguous, on {dev}")


def cache_append(cache, k, v, table, lens, fresh=None, stream=None) -> None:
    """Quantises the new tokens' keys and values, 16-bit [B, heads, T, D], into
    the cache: token i < fresh[b] (default T) goes to position lens[b] - fresh[b] + i."""
    c, s, dev, kv_heads, D, _, B, _ = _views(cache, table, lens, fresh)
    dt, heads, T = _rows("k", k, B, D, dev)
    if _rows("v", v, B, D, dev) != (dt, heads, T) or heads != kv_heads:
        raise ValueError("k and v must share shape and dtype and have the cache's heads")
    _call("attn_cache_append", dev, stream, c, s, k.data_ptr(), v.data_ptr(), T, dt)


def cache_fwd_workspace(cache, table, lens, q_heads, T, listed=0, with_mass=False) -> int:
    """Bytes of workspace cache_fwd needs for these sizes."""
    c, s, dev = _views(cache, table, lens, None)[:3]
    return _size("attn_cache_fwd_workspace", dev, c, s, listed, q_heads, T, int(with_mass))


def cache_fwd(q, cache, table, lens, fresh=None, scale=None, pages=None, mass=None, out=None, lse=None,
              workspace=None, stream=None, wait_timeout_ns: int | None = None):
    """Attention of the new tokens' queries q [B, Hq, T, D] over the cache.

    Each head reads every page, or the ones `pages` [B, heads, n] lists
    (ascending; negative: none).  `mass` [B, heads, width·page] fp32 gets the
    keys' attention weights added.  Returns (out like q, lse fp32 [B, Hq, T]);
    rows of tokens from fresh[b] on are not written.
    """
    c, s, dev, kv_heads, D, page, B, width = _views(cache, table, lens, fresh)
    dt, heads, T = _rows("q", q, B, D, dev)
    listed, list_p, mass_p = 0, None, None
    if pages is not None:
        if not isinstance(pages, torch.Tensor) or pages.dim() != 3 or pages.shape[2] < 1:
            raise ValueError("pages must be an int32 [batch, heads, n] tensor, n >= 1")
        listed = pages.shape[2]
        list_p = _want("pages", pages, torch.int32, (B, kv_heads, listed), dev)
    if mass is not None:
        mass_p = _want("mass", mass, torch.float32, (B, kv_heads, width * page), dev)
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(stream, dev, q.shape, q.dtype)
    else:
        _want("out", out, q.dtype, q.shape, dev)
    if lse is None:
        lse = _new(stream, dev, (B, heads, T), torch.float32)
    else:
        _want("lse", lse, torch.float32, (B, heads, T), dev)
    if workspace is None:
        space = _size("attn_cache_fwd_workspace", dev, c, s, listed, heads, T, int(mass is not None))
        if space > _NO_SPACE:
            workspace = _new(stream, dev, space, torch.uint8)
    else:
        _space(workspace, dev)
        space = workspace.numel()
    _call("attn_cache_fwd", dev, stream, c, s, q.data_ptr(), list_p, listed, out.data_ptr(), lse.data_ptr(), mass_p,
          heads, T, 1.0 / math.sqrt(D) if scale is None else float(scale), dt,
          None if workspace is None else workspace.data_ptr(), space, ATTN_DEFAULT_WAIT_TIMEOUT_NS if wait_timeout_ns is None else int(wait_timeout_ns))
    return out, lse


def cache_select(q, cache, table, lens, count, fresh=None, pages=None, scores=None, stream=None):
    """The `count` pages each head of each sequence should read for the queries
    q [B, Hq, T, D]: those of the new tokens and the best by an 8-bit bound on
    their scores.  Returns (pages int32 [B, heads, count], ascending, -1 behind
    the last; scores fp32 [B, heads, width])."""
    c, s, dev, kv_heads, D, page, B, width = _views(cache, table, lens, fresh)
    dt, heads, T = _rows("q", q, B, D, dev)
    count = int(count)
    if count < 1:
        raise ValueError("count must be at least 1")
    if pages is None:
        pages = _new(stream, dev, (B, kv_heads, count), torch.int32)
    else:
        _want("pages", pages, torch.int32, (B, kv_heads, count), dev)
    if scores is None:
        scores = _new(stream, dev, (B, kv_heads, width), torch.float32)
    else:
        _want("scores", scores, torch.float32, (B, kv_heads, width), dev)
    _call("attn_cache_select", dev, stream, c, s, q.data_ptr(), heads, T, dt, count, pages.data_ptr(),
          scores.data_ptr())
    return pages, scores


def cache_evict_workspace(cache, table, lens, dst_width) -> int:
    """Bytes of workspace cache_evict needs for these sizes."""
    c, s, dev = _views(cache, table, lens, None)[:3]
    return _size("attn_cache_evict_workspace", dev, c, s, dst_width)


def cache_evict(cache, mass, table, lens, dst_table, keep, recent, kept=None, new_lens=None, new_mass=None,
                workspace=None, stream=None):
    """Keeps, for each head, the last `recent` tokens and those of the largest
    `mass` up to `keep`, and moves them to the pages of dst_table [B, dst_width].
    Returns (kept int32 [B, heads, keep], new_lens int32 [B], new_mass fp32
    [B, heads, dst_width·page]); from then on dst_table and new_lens describe
    the sequences and the old pages are free."""
    c, s, dev, kv_heads, _, page, B, width = _views(cache, table, lens, None)
    mass_p = _want("mass", mass, torch.float32, (B, kv_heads, width * page), dev)
    if not isinstance(dst_table, torch.Tensor) or dst_table.dim() != 2:
        raise ValueError("dst_table must be an int32 [batch, dst_width] tensor")
    dst_width = dst_table.shape[1]
    dst_p = _want("dst_table", dst_table, torch.int32, (B, dst_width), dev)
    keep, recent = int(keep), int(recent)
    if keep < 1 or not 0 <= recent <= keep or keep > dst_width * page:
        raise ValueError("0 <= recent <= keep, 1 <= keep <= dst_width * page")
    if kept is None:
        kept = _new(stream, dev, (B, kv_heads, keep), torch.int32)
    else:
        _want("kept", kept, torch.int32, (B, kv_heads, keep), dev)
    if new_lens is None:
        new_lens = _new(stream, dev, (B,), torch.int32)
    else:
        _want("new_lens", new_lens, torch.int32, (B,), dev)
    if new_mass is None:
        new_mass = _new(stream, dev, (B, kv_heads, dst_width * page), torch.float32)
    else:
        _want("new_mass", new_mass, torch.float32, (B, kv_heads, dst_width * page), dev)
    if workspace is None:
        need = _size("attn_cache_evict_workspace", dev, c, s, dst_width)
        workspace = _new(stream, dev, need, torch.uint8)
    else:
        _space(workspace, dev)
    _call("attn_cache_evict", dev, stream, c, s, mass_p, dst_p, dst_width, keep, recent, kept.data_ptr(),
          new_lens.data_ptr(), new_mass.data_ptr(), workspace.data_ptr(), workspace.numel())
    return kept, new_lens, new_mass
