"""ctypes binding to the C ABI of include/attn_cross.h (argument marshalling only).

Cross-attention, beside ``binding.attn_fwd``: queries [B, Hq, Sq, D] over another
sequence's keys and values [B, Hkv, Sk, D], of which sequence b has lens[b]; query
heads share key heads in groups of Hq / Hkv.  ``cross_bwd`` is the gradient and
``cross_attention`` the differentiable form.  The meaning of every argument and the
errors are those of the header; there is no fallback.

    out, lse = cross_fwd(q, k, v, lens)              # lens int32 [B] on the device, or None
    dq, dk, dv, delta = cross_bwd(q, k, v, out, lse, dout, lens)
    out = cross_attention(q, k, v, lens)             # autograd

A captured backward pass of the differentiable forms needs what torch asks of any: no
eager graph of the same leaves may be alive, since their gradients would be added up
on that graph's stream.  cross_bwd itself has no such bound.  Nothing synchronises.  A
workspace is allocated per call where one is needed, unless one is passed; calls that may
run at the same time, and graphs, need one each.  With ``stream``, what a call allocates
belongs to that stream, as if it were the current one.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
import threading

import torch
from torch.autograd.function import once_differentiable

from .binding import (ATTN_BF16, ATTN_DEFAULT_WAIT_TIMEOUT_NS, ATTN_ERR_INVALID_ARG, ATTN_F16, ATTN_OK, AttnError,
                      load_library)

__all__ = ["cross_fwd", "cross_bwd", "cross_attention", "cross_fwd_workspace", "cross_bwd_workspace", "CROSS_SYMBOLS"]

_NO_SPACE = 16  # the size that says no workspace is needed

_i64, _p, _f, _i, _u64, _sz = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_uint64,
                               ctypes.c_size_t)


# attn_cross_t as bytes: batch, q_heads, heads, Sq, Sk, head_dim
_pack_sizes = struct.Struct("@6q").pack

_s = ctypes.c_char_p
_SIGS = {
    "attn_cross_fwd_workspace": (_sz, [_s]),
    "attn_cross_fwd": (_i, [_s, _p, _p, _p, _p, _p, _p, _f, _i, _p, _sz, _u64, _p]),
    "attn_cross_bwd_workspace": (_sz, [_s]),
    "attn_cross_bwd": (_i, [_s] + [_p] * 11 + [_f, _i, _p, _sz, _u64, _p]),
}
CROSS_SYMBOLS = tuple(_SIGS)

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}
_i32, _f32 = torch.int32, torch.float32
_lib = None
_lock = threading.Lock()


def declare(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the signatures of these entry points on a loaded library."""
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


def _inputs(q, k, v, lens):
    """The sizes packed, q's shape, the dtype and its code, the device and its index, and the address of lens."""
    try:
        dt, qs, ks, at = q.dtype, q.shape, k.shape, q.get_device()
        B, Hq, Sq, D = qs
        _, Hkv, Sk, _ = ks
        # everything in one condition: this is much of a small call's time
        if (at < 0 or dt not in _DTYPES or not q.is_contiguous() or ks[0] != B or ks[3] != D or k.dtype is not dt
                or not k.is_contiguous() or k.get_device() != at or v.shape != ks or v.dtype is not dt
                or not v.is_contiguous() or v.get_device() != at or Hkv < 1 or Hq % Hkv):
            _refuse(q, k, v)
        lens_p = None
        if lens is not None:
            if (lens.dtype is not _i32 or lens.shape != (B,) or not lens.is_contiguous() or lens.get_device() != at):
                _want("lens", lens, _i32, (B,), q.device)
            lens_p = lens.data_ptr()
        return _pack_sizes(B, Hq, Hkv, Sq, Sk, D), qs, dt, _DTYPES[dt], q.device, at, lens_p
    except (AttributeError, ValueError):
        _refuse(q, k, v)
        if lens is not None:
            _want("lens", lens, _i32, (q.shape[0],), q.device)
        raise


def _refuse(q, k, v):
    """Names what _inputs found wrong, one tensor after the other."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError("q must be a bfloat16 or float16 tensor")
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype is not q.dtype:
            raise TypeError(f"{name} must be a tensor of q's dtype")
    if not q.is_cuda or q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous CUDA tensor [B, Hq, Sq, D]")
    for name, t in (("k", k), ("v", v)):
        if (t.dim() != 4 or t.shape[0] != q.shape[0] or t.shape[3] != q.shape[3] or not t.is_contiguous()
                or t.device != q.device or t.shape != k.shape):
            raise ValueError(f"{name} must be a contiguous tensor [{q.shape[0]}, Hkv, Sk, {q.shape[3]}] on {q.device}, "
                             "k and v alike")
    if k.shape[1] < 1 or q.shape[1] % k.shape[1]:
        raise ValueError("q's heads must be a multiple of k's")


def _want(name, t, dtype, shape, dev):
    """The address of a tensor that has to be just so."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


# the current device and its current stream's handle, without the objects
# torch.cuda.current_stream makes on the way
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name, index, stream, *args):
    """The entry point on `stream` (default: the current one) of device `index`."""
    if stream is not None:
        st = stream.cuda_stream
    elif _raw_stream is not None:
        st = _raw_stream(index)
    else:
        st = torch.cuda.current_stream(index).cuda_stream
    fn = getattr(_lib or _library(), name)
    if index == _current_device():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, st)
    if rc != ATTN_OK:
        raise AttnError(rc, name)


@functools.lru_cache(maxsize=4096)
def _size(name, index, sizes):
    """Bytes of workspace: sizes and device alone decide them."""
    fn = getattr(_lib or _library(), name)
    with torch.cuda.device(index):
        n = fn(sizes)
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


def _space(name, workspace, dev, index, sizes, stream):
    """The workspace of a call, its address and bytes."""
    if workspace is None:
        need = _size(name, index, sizes)
        if need <= _NO_SPACE:
            return None, None, 0
        workspace = _new(stream, dev, need, torch.uint8)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be contiguous, on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel()


def cross_fwd_workspace(q, k) -> int:
    """Bytes of workspace cross_fwd needs for these tensors' sizes (16: none)."""
    sizes, _, _, _, _, index, _ = _inputs(q, k, k, None)
    return _size("attn_cross_fwd_workspace", index, sizes)


def cross_bwd_workspace(q, k) -> int:
    """Bytes of workspace cross_bwd needs for these tensors' sizes (16: none)."""
    sizes, _, _, _, _, index, _ = _inputs(q, k, k, None)
    return _size("attn_cross_bwd_workspace", index, sizes)


def cross_fwd(q, k, v, lens=None, scale=None, out=None, lse=None, workspace=None, stream=None,
              wait_timeout_ns: int | None = None):
    """Attention of q [B, Hq, Sq, D] over the first lens[b] of k, v [B, Hkv, Sk, D].
    Returns (out like q, lse fp32 [B, Hq, Sq]); a sequence without keys gives 0 and -inf."""
    sizes, shape, dt, code, dev, index, lens_p = _inputs(q, k, v, lens)
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(stream, dev, shape, dt)
    else:
        _want("out", out, dt, shape, dev)
    if lse is None:
        lse = _new(stream, dev, shape[:3], _f32)
    else:
        _want("lse", lse, _f32, shape[:3], dev)
    workspace, at, space = _space("attn_cross_fwd_workspace", workspace, dev, index, sizes, stream)
    _call("attn_cross_fwd", index, stream, sizes, q.data_ptr(), k.data_ptr(), v.data_ptr(), lens_p, out.data_ptr(),
          lse.data_ptr(), 1.0 / math.sqrt(shape[3]) if scale is None else float(scale), code, at, space,
          ATTN_DEFAULT_WAIT_TIMEOUT_NS if wait_timeout_ns is None else int(wait_timeout_ns))
    return out, lse


def cross_bwd(q, k, v, out, lse, dout, lens=None, scale=None, dq=None, dk=None, dv=None, delta=None, workspace=None,
              stream=None, wait_timeout_ns: int | None = None):
    """Gradient of cross_fwd.  Returns (dq like q; dk, dv like k, 0 for keys that are not
    there; delta = rowsum(dout ⊙ out) fp32 [B, Hq, Sq])."""
    sizes, shape, dt, code, dev, index, lens_p = _inputs(q, k, v, lens)
    ks, rows = k.shape, shape[:3]
    out_p, dout_p = _want("out", out, dt, shape, dev), _want("dout", dout, dt, shape, dev)
    lse_p = _want("lse", lse, _f32, rows, dev)
    if dq is None:
        dq = torch.empty_like(q) if stream is None else _new(stream, dev, shape, dt)
    else:
        _want("dq", dq, dt, shape, dev)
    if dk is None:
        dk = torch.empty_like(k) if stream is None else _new(stream, dev, ks, dt)
    else:
        _want("dk", dk, dt, ks, dev)
    if dv is None:
        dv = torch.empty_like(k) if stream is None else _new(stream, dev, ks, dt)
    else:
        _want("dv", dv, dt, ks, dev)
    if delta is None:
        delta = _new(stream, dev, rows, _f32)
    else:
        _want("delta", delta, _f32, rows, dev)
    workspace, at, space = _space("attn_cross_bwd_workspace", workspace, dev, index, sizes, stream)
    _call("attn_cross_bwd", index, stream, sizes, q.data_ptr(), k.data_ptr(), v.data_ptr(), lens_p, out_p, lse_p, dout_p,
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), delta.data_ptr(),
          1.0 / math.sqrt(shape[3]) if scale is None else float(scale), code, at, space,
          ATTN_DEFAULT_WAIT_TIMEOUT_NS if wait_timeout_ns is None else int(wait_timeout_ns))
    return dq, dk, dv, delta


class _CrossFn(torch.autograd.Function):
    """cross_fwd in forward, cross_bwd in backward (both through the C ABI)."""

    @staticmethod
    def forward(ctx, q, k, v, lens, scale):
        out, lse = cross_fwd(q, k, v, lens, scale)
        ctx.save_for_backward(q, k, v, lens, out, lse)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, lens, out, lse = ctx.saved_tensors
        dq, dk, dv, _ = cross_bwd(q, k, v, out, lse, dout.contiguous(), lens, ctx.scale)
        return dq, dk, dv, None, None


def cross_attention(q, k, v, lens=None, scale=None):
    """Differentiable cross-attention: gradients flow to q, k and v."""
    return _CrossFn.apply(q, k, v, lens, 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale))
