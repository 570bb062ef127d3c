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

Nothing synchronises.  With ``stream``, what a call allocates belongs to that
stream, as if it were the current one.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import NamedTuple, Optional

import torch

from .binding import ATTN_BF16, ATTN_ERR_INVALID_ARG, ATTN_F16, ATTN_OK, AttnError, attn_bwd, attn_fwd, load_library

__all__ = ["Rope", "rope_plan", "rope_fwd", "rope_bwd", "rope_bwd_workspace", "norm_rope", "rotary_attention",
           "ROPE_MAX_PARTS", "ROPE_MAX_AXES", "ROPE_SYMBOLS"]

ROPE_MAX_PARTS = 4
ROPE_MAX_AXES = 8
_NO_SPACE = 16  # the size that says no workspace is needed

_i64, _p, _f, _i, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_size_t


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", _p), ("axis", _p), ("pairs", _i64), ("interleaved", _i)]


class _Positions(ctypes.Structure):
    _fields_ = [("at", _p), ("stride_b", _i64), ("stride_s", _i64), ("stride_a", _i64), ("axes", _i64)]


class _Part(ctypes.Structure):
    _fields_ = [("x", _p), ("stride_b", _i64), ("stride_s", _i64), ("stride_h", _i64), ("heads", _i64),
                ("weight", _p), ("weight_f32", _i), ("turn", _i), ("y", _p), ("dx", _p), ("dx_stride_b", _i64),
                ("dx_stride_s", _i64), ("dx_stride_h", _i64), ("dweight", _p)]


_pp, _rp, _ap = ctypes.POINTER(_Part), ctypes.POINTER(_Rope), ctypes.POINTER(_Positions)
_SIGS = {
    "attn_rope_fwd": (_i, [_pp, _i, _rp, _ap, _i64, _i64, _i64, _f, _i, _p]),
    "attn_rope_bwd_workspace": (_sz, [_pp, _i, _i64, _i64, _i64]),
    "attn_rope_bwd": (_i, [_pp, _i, _rp, _ap, _i64, _i64, _i64, _f, _i, _p, _sz, _p]),
}
ROPE_SYMBOLS = tuple(_SIGS)
_ARRAYS = [None] + [_Part * n for n in range(1, ROPE_MAX_PARTS + 1)]

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}
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
    """B, S, D, the heads, the device and the dtype code of a call's [B, S, H, D] tensors."""
    if not 1 <= len(xs) <= ROPE_MAX_PARTS:
        raise ValueError(f"1 to {ROPE_MAX_PARTS} tensors a call")
    x0 = xs[0]
    if not isinstance(x0, torch.Tensor) or x0.dtype not in _DTYPES:
        raise TypeError(f"{what} must be bfloat16 or float16 tensors")
    if x0.dim() != 4 or not x0.is_cuda:
        raise ValueError(f"{what} must be CUDA tensors [B, S, heads, D]")
    B, S, _, D = x0.shape
    dt, dev, heads = x0.dtype, x0.device, []
    for x in xs:
        if not isinstance(x, torch.Tensor) or x.dtype != dt:
            raise TypeError(f"{what} must share a dtype, bfloat16 or float16")
        shape = x.shape
        if len(shape) != 4 or shape[0] != B or shape[1] != S or shape[3] != D or x.device != dev:
            raise ValueError(f"{what} must be [{B}, {S}, heads, {D}] tensors on {dev}")
        if D > 1 and x.stride(3) != 1:
            raise ValueError(f"{what} must have adjacent channels")
        heads.append(shape[2])
    return B, S, D, heads, dev, dt


def _strides(x):
    """Strides of batch, token and head; a dimension of one entry counts as having none to go by."""
    (B, S, H, _), (b, s, h, _) = x.shape, x.stride()
    return (b if B > 1 else 0), (s if S > 1 else 0), (h if H > 1 else 0)


def _weight(name, w, D, dt, dev):
    if w.dtype != dt and w.dtype != torch.float32:
        raise TypeError(f"{name} must have the heads' dtype or be float32")
    if w.shape != (D,) or not w.is_contiguous() or w.device != dev:
        raise ValueError(f"{name} must be a contiguous [{D}] tensor on {dev}")
    return w.data_ptr(), w.dtype == torch.float32


def _rope(plan, positions, B, S, dev):
    """The C structures of a rotation and the tokens' positions [B, S] or [B, S, axes] (either of the first two 1)."""
    if plan is None:
        return None, None
    freq, axis, interleaved = plan
    if not isinstance(freq, torch.Tensor) or freq.dtype != torch.float64 or freq.dim() != 1 or freq.is_cuda \
            or not freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 host tensor [pairs]")
    if axis is not None and (not isinstance(axis, torch.Tensor) or axis.dtype != torch.uint8 or axis.is_cuda
                             or axis.shape != freq.shape or not axis.is_contiguous()):
        raise TypeError("axis must be a contiguous uint8 host tensor [pairs]")
    if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
        raise TypeError("positions must be an int32 tensor")
    shape, stride = positions.shape, positions.stride()
    if len(shape) == 2:
        shape, stride = (*shape, 1), (*stride, 0)
    if len(shape) != 3 or shape[0] not in (1, B) or shape[1] not in (1, S) or positions.device != dev:
        raise ValueError(f"positions must be [{B}, {S}] or [{B}, {S}, axes] on {dev}")
    at = _Positions(positions.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0,
                    stride[2] if shape[2] > 1 else 0, shape[2])
    return _Rope(freq.data_ptr(), None if axis is None else axis.data_ptr(), freq.numel(), interleaved), at


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


def _want_rows(name, t, shape, dt, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dt:
        raise TypeError(f"{name} must be a {dt} tensor")
    if t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on {dev}")
    return t


def rope_fwd(xs, plan, positions=None, weights=None, eps: float = 1e-6, turn=None, ys=None, stream=None):
    """Norm, rotation and layout of 1 to 4 tensors [B, S, H, D] in one pass.

    weights[i] [D], of the heads' dtype or float32, or None: no norm.  turn[i]
    (default: all) rotates by `plan` and `positions`; without a plan nothing
    turns.  Returns the contiguous [B, H, S, D] tensors (``ys`` if given)."""
    B, S, D, heads, dev, dt = _views(xs, "xs")
    n = len(xs)
    weights, ys = _per_part(weights, n, "weights"), _per_part(ys, n, "ys")
    turn = (plan is not None,) * n if turn is None else _per_part(turn, n, "turn")
    rope, at = _rope(plan, positions, B, S, dev) if any(turn) else (None, None)
    parts, out = _ARRAYS[n](), []
    for i, x in enumerate(xs):
        y = ys[i]
        if y is None:
            y = _new(stream, dev, (B, heads[i], S, D), dt)
        else:
            _want_rows("ys", y, (B, heads[i], S, D), dt, dev)
        out.append(y)
        w, f32 = (None, False) if weights[i] is None else _weight("weights", weights[i], D, dt, dev)
        parts[i] = _Part(x.data_ptr(), *_strides(x), heads[i], w, f32, bool(turn[i]), y.data_ptr())
    _call("attn_rope_fwd", dev, stream, parts, n, rope, at, B, S, D, eps, _DTYPES[dt])
    return out


def rope_bwd_workspace(xs, weights) -> int:
    """Bytes of workspace rope_bwd needs for these sizes (16: none)."""
    B, S, D, heads, dev, _ = _views(xs, "xs")
    parts = _ARRAYS[len(xs)]()
    for i, w in enumerate(_per_part(weights, len(xs), "weights")):
        parts[i].heads, parts[i].dweight = heads[i], None if w is None else w.data_ptr()
    return _space(parts, len(xs), B, S, D, dev)


def _space(parts, n, B, S, D, dev):
    with torch.cuda.device(dev):
        size = _library().attn_rope_bwd_workspace(parts, n, B, S, D)
    if size == 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_rope_bwd_workspace")
    return size


def rope_bwd(dys, xs, plan, positions=None, weights=None, eps: float = 1e-6, turn=None, dxs=None, dweights=None,
             workspace=None, stream=None):
    """The gradient of rope_fwd: from dys [B, H, S, D], contiguous, and the forward's
    other arguments.  ``dxs`` may be views of one packed gradient; by default they are
    new contiguous [B, S, H, D] tensors.  Returns (dxs, dweights); dweights[i] is None
    where weights[i] is."""
    B, S, D, heads, dev, dt = _views(xs, "xs")
    n = len(xs)
    if len(dys) != n:
        raise ValueError("dys must have an entry for each tensor")
    weights, dxs, dweights = (_per_part(v, n, m) for v, m in ((weights, "weights"), (dxs, "dxs"), (dweights, "dweights")))
    if any(d is not None for d in dxs):
        if any(d is None for d in dxs) or _views(dxs, "dxs") != (B, S, D, heads, dev, dt):
            raise ValueError("dxs must be tensors of the shapes, dtype and device of xs")
    turn = (plan is not None,) * n if turn is None else _per_part(turn, n, "turn")
    rope, at = _rope(plan, positions, B, S, dev) if any(turn) else (None, None)
    parts, out, grads = _ARRAYS[n](), [], []
    for i, (x, dy) in enumerate(zip(xs, dys)):
        _want_rows("dys", dy, (B, heads[i], S, D), dt, dev)
        dx = dxs[i]
        if dx is None:
            dx = _new(stream, dev, x.shape, dt)
        out.append(dx)
        w, f32, dw = None, False, None
        if weights[i] is not None:
            w, f32 = _weight("weights", weights[i], D, dt, dev)
            dw = dweights[i]
            if dw is None:
                dw = _new(stream, dev, (D,), weights[i].dtype)
            else:
                _want_rows("dweights", dw, (D,), weights[i].dtype, dev)
        elif dweights[i] is not None:
            raise ValueError("dweights without weights")
        grads.append(dw)
        parts[i] = _Part(x.data_ptr(), *_strides(x), heads[i], w, f32, bool(turn[i]), dy.data_ptr(), dx.data_ptr(),
                         *_strides(dx), None if dw is None else dw.data_ptr())
    space, at_ws = 0, None
    if any(g is not None for g in grads):
        if workspace is None:
            workspace = _new(stream, dev, _space(parts, n, B, S, D, dev), torch.uint8)
        elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace must be a uint8 tensor")
        elif not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError(f"workspace must be contiguous, on {dev}")
        space, at_ws = workspace.numel(), workspace.data_ptr()
    _call("attn_rope_bwd", dev, stream, parts, n, rope, at, B, S, D, eps, _DTYPES[dt], at_ws, space)
    return out, grads


class _NormRopeFn(torch.autograd.Function):
    """rope_fwd in forward, rope_bwd in backward (both through the C ABI)."""

    @staticmethod
    def forward(ctx, plan, positions, eps, turn, n, *tensors):
        xs, weights = tensors[:n], tensors[n:]
        ctx.save_for_backward(positions, *tensors)
        ctx.plan, ctx.eps, ctx.turn, ctx.n = plan, eps, turn, n
        return tuple(rope_fwd(xs, plan, positions, weights, eps, turn))

    @staticmethod
    def backward(ctx, *dys):
        positions, *tensors = ctx.saved_tensors
        n = ctx.n
        dxs, dws = rope_bwd([dy.contiguous() for dy in dys], tensors[:n], ctx.plan, positions, tensors[n:], ctx.eps,
                            ctx.turn)
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
        ctx.save_for_backward(q, k, v, positions, wq, wk, qh, kh, vh, out, lse)
        ctx.rest = plan, eps, scale, causal
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, positions, wq, wk, qh, kh, vh, out, lse = ctx.saved_tensors
        plan, eps, scale, causal = ctx.rest
        dq, dk, dv, _ = attn_bwd(qh, kh, vh, out, lse, dout.contiguous(), scale=scale, causal=causal)
        dxs, dws = rope_bwd((dq, dk, dv), (q, k, v), plan, positions, (wq, wk, None), eps,
                            (plan is not None, plan is not None, False))
        return (*dxs, None, None, dws[0], dws[1], None, None, None)


def rotary_attention(q, k, v, plan=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, scale=None,
                     causal=True):
    """Differentiable self-attention from the projections on: q, k, v [B, S, H, D] views
    are normalised (where a weight is given), turned and laid out by rope_fwd, then
    attended over by attn_fwd.  Returns out [B, H, S, D]; gradients flow to q, k, v and
    the weights."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _RotaryAttentionFn.apply(q, k, v, plan, positions, q_weight, k_weight, float(eps), float(scale), bool(causal))
