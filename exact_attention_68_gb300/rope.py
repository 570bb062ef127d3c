"""ctypes binding to the C ABI of include/attn_rope.h (argument marshalling only).

The heads' norm and rotation, between a block's projections and its attention:
``rope_fwd`` takes queries, keys and values as a projection leaves them,
[B, S, H, D] views of any strides, and gives the contiguous [B, H, S, D] that
``binding.attn_fwd`` and ``cross.cross_fwd`` take, each head divided by its root
mean square and weighted, and its pairs of channels turned by their positions.
``rope_bwd`` is the gradient, ``norm_rope`` the differentiable form, and
``rotary_attention`` a block's self-attention from the projections on.  The
formulas, the layouts and the errors are the header's; there is no fallback.

    plan = rope_plan((16, 56, 56))                   # channels of time, height, width
    q, k, v = rope_fwd((q, k, v), plan, positions, (wq, wk, None), turn=(True, True, False))
    out = rotary_attention(q, k, v, plan, positions, wq, wk)

A captured backward pass of the differentiable forms needs what torch asks of any: no
eager graph of the same leaves may be alive, since their gradients would be added up
on that graph's stream.  rope_bwd itself has no such bound.  Nothing synchronises.  With
``stream``, what a call allocates belongs to that stream, as if it were the current one.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from .binding import ATTN_BF16, ATTN_ERR_INVALID_ARG, ATTN_F16, ATTN_OK, AttnError, attn_bwd, attn_fwd, load_library

__all__ = ["Rope", "rope_plan", "rope_fwd", "rope_bwd", "rope_bwd_workspace", "norm_rope", "rotary_attention",
           "ROPE_MAX_PARTS", "ROPE_MAX_AXES", "ROPE_SYMBOLS"]

ROPE_MAX_PARTS = 4
ROPE_MAX_AXES = 8
_NO_SPACE = 16  # the size that says no workspace is needed

_i64, _p, _f, _i, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_size_t


# The C structures as bytes: attn_rope_t, attn_rope_positions_t, attn_rope_part_t
# (packing costs a third of what ctypes structures do, and a small call is mostly this).
_pack_rope = struct.Struct("@3qi4x").pack
_pack_positions = struct.Struct("@5q").pack
_pack_part = struct.Struct("@6q2i6q").pack

_b = ctypes.c_char_p
_SIGS = {
    "attn_rope_fwd": (_i, [_b, _i, _b, _b, _i64, _i64, _i64, _f, _i, _p]),
    "attn_rope_bwd_workspace": (_sz, [_b, _i, _i64, _i64, _i64]),
    "attn_rope_bwd": (_i, [_b, _i, _b, _b, _i64, _i64, _i64, _f, _i, _p, _sz, _p]),
}
ROPE_SYMBOLS = tuple(_SIGS)

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}
_f32 = torch.float32
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


class Rope(NamedTuple):
    """A rotation: pair i of ``inv_freq.numel()`` turns by positions[..., axis[i]] ·
    inv_freq[i].  inv_freq float64 and axis uint8 (None: all axis 0) are contiguous
    host tensors [pairs].  The pairs are channels (i, i + pairs), or (2i, 2i + 1)
    where ``interleaved``; channels from 2·pairs on are not turned."""
    inv_freq: torch.Tensor
    axis: Optional[torch.Tensor] = None
    interleaved: bool = False


def rope_plan(dims, base: float = 10000.0, interleaved: bool = False) -> Rope:
    """The usual rotation: axis a turns dims[a] channels (an even number), its pair i of
    n = dims[a] / 2 with inv_freq = base^(-i/n).  ``dims`` is a number for one axis."""
    dims = (dims,) if isinstance(dims, int) else tuple(dims)
    if not 1 <= len(dims) <= ROPE_MAX_AXES or any(d < 0 or d % 2 for d in dims) or not base > 0:
        raise ValueError(f"dims must be 1 to {ROPE_MAX_AXES} even numbers, base positive")
    freq = [base ** (-2 * i / d) for d in dims for i in range(d // 2)]
    axis = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    return Rope(torch.tensor(freq, dtype=torch.float64), torch.tensor(axis, dtype=torch.uint8), bool(interleaved))


def _views(xs, what):
    """B, S, D, the device, its index, the dtype and, of each of a call's [B, S, H, D] tensors,
    (address, strides of batch, token and head, heads)."""
    if not 1 <= len(xs) <= ROPE_MAX_PARTS:
        raise ValueError(f"1 to {ROPE_MAX_PARTS} tensors a call")
    try:
        x0 = xs[0]
        B, S, _, D = x0.shape
        dt, at, got = x0.dtype, x0.get_device(), []
        for x in xs:
            b, s, h, d = x.shape
            u, v, w, c = x.stride()
            if (b != B or s != S or d != D or x.dtype is not dt or x.get_device() != at or (c != 1 and D > 1)):
                _refuse(xs, what)
            # a dimension of one entry has no stride to go by
            got.append((x.data_ptr(), u if B > 1 else 0, v if S > 1 else 0, w if h > 1 else 0, h))
        if dt not in _DTYPES or at < 0:
            _refuse(xs, what)
        return B, S, D, x0.device, at, dt, got
    except (AttributeError, ValueError):
        _refuse(xs, what)
        raise


def _refuse(xs, what):
    """Names what _views found wrong, one tensor after the other."""
    for x in xs:
        if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
            raise TypeError(f"{what} must be bfloat16 or float16 tensors")
        if x.dim() != 4 or not x.is_cuda:
            raise ValueError(f"{what} must be CUDA tensors [B, S, heads, D]")
    B, S, _, D = xs[0].shape
    for x in xs:
        if x.dtype is not xs[0].dtype:
            raise TypeError(f"{what} must share a dtype")
        if x.shape[:2] != (B, S) or x.shape[3] != D or x.device != xs[0].device:
            raise ValueError(f"{what} must be [{B}, {S}, heads, {D}] tensors on {xs[0].device}")
        if D > 1 and x.stride(3) != 1:
            raise ValueError(f"{what} must have adjacent channels")


def _weight(name, w, D, dt, at):
    """The address of a weight and whether it is float32; (0, 0) without one."""
    if w is None:
        return 0, 0
    if not isinstance(w, torch.Tensor) or (w.dtype is not dt and w.dtype is not _f32):
        raise TypeError(f"{name} must be tensors of the heads' dtype or float32")
    if w.shape != (D,) or not w.is_contiguous() or w.get_device() != at:
        raise ValueError(f"{name} must be contiguous [{D}] tensors on the heads' device")
    return w.data_ptr(), w.dtype is _f32


def _rope(plan, positions, B, S, at):
    """The C structures of a rotation and the tokens' positions [B, S] or [B, S, axes] (either of the first two 1)."""
    if plan is None:
        return None, None
    freq, axis, interleaved = plan
    if not isinstance(freq, torch.Tensor) or freq.dtype is not torch.float64 or freq.dim() != 1 or freq.is_cuda \
            or not freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 host tensor [pairs]")
    if axis is not None and (not isinstance(axis, torch.Tensor) or axis.dtype is not torch.uint8 or axis.is_cuda
                             or axis.shape != freq.shape or not axis.is_contiguous()):
        raise TypeError("axis must be a contiguous uint8 host tensor [pairs]")
    if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32:
        raise TypeError("positions must be an int32 tensor")
    shape, stride = positions.shape, positions.stride()
    if len(shape) == 2:
        shape, stride = (*shape, 1), (*stride, 0)
    if len(shape) != 3 or shape[0] not in (1, B) or shape[1] not in (1, S) or positions.get_device() != at:
        raise ValueError(f"positions must be [{B}, {S}] or [{B}, {S}, axes] on the heads' device")
    return (_pack_rope(freq.data_ptr(), 0 if axis is None else axis.data_ptr(), freq.numel(), interleaved),
            _pack_positions(positions.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0,
                            stride[2] if shape[2] > 1 else 0, shape[2]))


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


def _new(stream, dev, shape, dtype):
    """Memory for a call on `stream`, from that stream's pool."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _per_part(values, n, name):
    if values is None:
        return (None,) * n
    if len(values) != n:
        raise ValueError(f"{name} must have an entry for each tensor")
    return values


def _want_rows(name, t, shape, dt, at):
    """The address of a contiguous tensor that has to be just so."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dt:
        raise TypeError(f"{name} must be a {dt} tensor")
    if t.shape != shape or not t.is_contiguous() or t.get_device() != at:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on the heads' device")
    return t.data_ptr()


def rope_fwd(xs, plan, positions=None, weights=None, eps: float = 1e-6, turn=None, ys=None, stream=None):
    """Norm, rotation and layout of 1 to 4 tensors [B, S, H, D] in one pass.

    weights[i] [D], of the heads' dtype or float32, or None: no norm.  turn[i]
    (default: all) rotates by `plan` and `positions`; without a plan nothing
    turns.  Returns the contiguous [B, H, S, D] tensors (``ys`` if given)."""
    B, S, D, dev, at, dt, got = _views(xs, "xs")
    n = len(xs)
    weights, ys = _per_part(weights, n, "weights"), _per_part(ys, n, "ys")
    turn = (plan is not None,) * n if turn is None else _per_part(turn, n, "turn")
    rope, pos = _rope(plan, positions, B, S, at) if any(turn) else (None, None)
    parts, out = [], []
    for x, w, y, t in zip(got, weights, ys, turn):
        shape = (B, x[4], S, D)
        if y is None:
            y = _new(stream, dev, shape, dt)
            y_p = y.data_ptr()
        else:
            y_p = _want_rows("ys", y, shape, dt, at)
        out.append(y)
        w_p, f32 = _weight("weights", w, D, dt, at)
        parts.append(_pack_part(*x, w_p, f32, bool(t), y_p, 0, 0, 0, 0, 0))
    _call("attn_rope_fwd", at, stream, b"".join(parts), n, rope, pos, B, S, D, eps, _DTYPES[dt])
    return out


def rope_bwd_workspace(xs, weights) -> int:
    """Bytes of workspace rope_bwd needs for these sizes (16: none)."""
    B, S, D, _, at, _, got = _views(xs, "xs")
    return _space(b"".join(_pack_part(*x, 0, 0, 0, 0, 0, 0, 0, 0, 0 if w is None else w.data_ptr())
                           for x, w in zip(got, _per_part(weights, len(xs), "weights"))), len(xs), B, S, D, at)


def _space(parts, n, B, S, D, index):
    with torch.cuda.device(index):
        size = _library().attn_rope_bwd_workspace(parts, n, B, S, D)
    if size == 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_rope_bwd_workspace")
    return size


_spaces = {}  # bytes by device, channels and how many weights have a gradient: nothing else decides them


def rope_bwd(dys, xs, plan, positions=None, weights=None, eps: float = 1e-6, turn=None, dxs=None, dweights=None,
             workspace=None, stream=None):
    """The gradient of rope_fwd: from dys [B, H, S, D], contiguous, and the forward's
    other arguments.  ``dxs`` may be views of one packed gradient; by default they are
    new contiguous [B, S, H, D] tensors.  Returns (dxs, dweights); dweights[i] is None
    where weights[i] is."""
    B, S, D, dev, at, dt, got = _views(xs, "xs")
    n = len(xs)
    if len(dys) != n:
        raise ValueError("dys must have an entry for each tensor")
    weights, dweights = _per_part(weights, n, "weights"), _per_part(dweights, n, "dweights")
    if dxs is None:
        dxs = [_new(stream, dev, x.shape, dt) for x in xs]
    into = _views(dxs, "dxs")
    if into[:3] != (B, S, D) or into[4:6] != (at, dt) or [x[4] for x in into[6]] != [x[4] for x in got]:
        raise ValueError("dxs must be tensors of the shapes, dtype and device of xs")
    turn = (plan is not None,) * n if turn is None else _per_part(turn, n, "turn")
    rope, pos = _rope(plan, positions, B, S, at) if any(turn) else (None, None)
    parts, grads, wanted = [], [], 0
    for x, d, dy, w, dw, t in zip(got, into[6], dys, weights, dweights, turn):
        y_p = _want_rows("dys", dy, (B, x[4], S, D), dt, at)
        w_p, f32 = _weight("weights", w, D, dt, at)
        dw_p = 0
        if w is not None:
            wanted += 1
            if dw is None:
                dw = _new(stream, dev, (D,), w.dtype)
                dw_p = dw.data_ptr()
            else:
                dw_p = _want_rows("dweights", dw, (D,), w.dtype, at)
        elif dw is not None:
            raise ValueError("dweights without weights")
        grads.append(dw)
        parts.append(_pack_part(*x, w_p, f32, bool(t), y_p, *d[:4], dw_p))
    parts, space, space_p = b"".join(parts), 0, None
    if wanted:
        if workspace is None:
            space = _spaces.get((at, D, wanted))
            if space is None:
                space = _spaces[at, D, wanted] = _space(parts, n, B, S, D, at)
            workspace = _new(stream, dev, space, torch.uint8)
        elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace must be a uint8 tensor")
        elif not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError(f"workspace must be contiguous, on {dev}")
        space, space_p = workspace.numel(), workspace.data_ptr()
    _call("attn_rope_bwd", at, stream, parts, n, rope, pos, B, S, D, eps, _DTYPES[dt], space_p, space)
    return list(dxs), grads


def _kept(plan):
    """A plan's tensors, to be saved for the backward pass as the others are: torch refuses them once changed."""
    return (None, None) if plan is None else (plan[0], plan[1])


def _plan_of(freq, axis, interleaved):
    return None if freq is None else Rope(freq, axis, interleaved)


class _NormRopeFn(torch.autograd.Function):
    """rope_fwd in forward, rope_bwd in backward (both through the C ABI)."""

    @staticmethod
    def forward(ctx, plan, positions, eps, turn, n, *tensors):
        xs, weights = tensors[:n], tensors[n:]
        ctx.save_for_backward(positions, *_kept(plan), *tensors)
        ctx.interleaved, ctx.eps, ctx.turn, ctx.n = plan and plan[2], eps, turn, n
        return tuple(rope_fwd(xs, plan, positions, weights, eps, turn))

    @staticmethod
    @once_differentiable
    def backward(ctx, *dys):
        positions, freq, axis, *tensors = ctx.saved_tensors
        n, plan = ctx.n, _plan_of(freq, axis, ctx.interleaved)
        dxs, dws = rope_bwd([dy.contiguous() for dy in dys], tensors[:n], plan, positions, tensors[n:], ctx.eps, ctx.turn)
        return (None, None, None, None, None, *dxs, *dws)


def norm_rope(xs, plan, positions=None, weights=None, eps: float = 1e-6, turn=None):
    """Differentiable rope_fwd: gradients flow to xs and weights."""
    n = len(xs)
    turn = (plan is not None,) * n if turn is None else tuple(bool(t) for t in _per_part(turn, n, "turn"))
    return _NormRopeFn.apply(plan, positions, float(eps), turn, n, *xs, *_per_part(weights, n, "weights"))


class _RotaryAttentionFn(torch.autograd.Function):
    """rope_fwd and attn_fwd in forward, attn_bwd and rope_bwd in backward."""

    @staticmethod
    def forward(ctx, q, k, v, plan, positions, wq, wk, eps, scale, causal):
        qh, kh, vh = rope_fwd((q, k, v), plan, positions, (wq, wk, None), eps, (plan is not None, plan is not None, False))
        out, lse = attn_fwd(qh, kh, vh, scale=scale, causal=causal)
        ctx.save_for_backward(q, k, v, positions, *_kept(plan), wq, wk, qh, kh, vh, out, lse)
        ctx.rest = plan and plan[2], eps, scale, causal
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, positions, freq, axis, wq, wk, qh, kh, vh, out, lse = ctx.saved_tensors
        interleaved, eps, scale, causal = ctx.rest
        plan = _plan_of(freq, axis, interleaved)
        dq, dk, dv, _ = attn_bwd(qh, kh, vh, out, lse, dout.contiguous(), scale=scale, causal=causal)
        dxs, dws = rope_bwd((dq, dk, dv), (q, k, v), plan, positions, (wq, wk, None), eps,
                            (plan is not None, plan is not None, False))
        return (*dxs, None, None, dws[0], dws[1], None, None, None)


def rotary_attention(q, k, v, plan=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, scale=None,
                     causal=True):
    """Differentiable self-attention from the projections on: q, k, v [B, S, H, D] views
    are normalised (where a weight is given), turned and laid out by rope_fwd, then
    attended over by attn_fwd, so the three share one number of heads.  Returns out
    [B, H, S, D]; gradients flow to q, k, v and the weights."""
    if not q.shape == k.shape == v.shape:
        raise ValueError("q, k, v must share a shape: heads that share keys and values are not attn_fwd's")
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _RotaryAttentionFn.apply(q, k, v, plan, positions, q_weight, k_weight, float(eps), float(scale), bool(causal))
