"""CPU checks of the heads' norm and rotation: the oracle against differences and
hand-worked values, the plan, and the library's refusals (no CUDA call is reached)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, rope
from exact_attention_68_gb300.build import build_library
from oracle import rope as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return rope.declare(binding.load_library(build_library()))


def test_header_declares_the_bound_symbols(lib):
    with open(os.path.join(ROOT, "include", "attn_rope.h")) as f:
        names = re.findall(r"ATTN_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", f.read())
    assert sorted(names) == sorted(rope.ROPE_SYMBOLS)
    for n in names:
        assert hasattr(lib, n)


def test_oracle_hand_worked():
    x = np.array([[[[3.0, 4.0, 0.0, 0.0]]]])
    # mean of squares 25/4; one pair, channels 0 and 1: a quarter turn takes (a, c) to (-c, a)
    y = oracle.rope_fwd(x, [1, 1, 1, 1], np.array([[[1]]]), [np.pi / 2], interleaved=False, eps=0.0)
    np.testing.assert_allclose(y[0, 0, 0], [-1.6, 1.2, 0, 0], atol=1e-15)
    y = oracle.rope_fwd(x, None, np.array([[[2]]]), [np.pi / 2], interleaved=True)
    np.testing.assert_allclose(y[0, 0, 0], [-3, -4, 0, 0], atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_oracle_gradient_against_differences(interleaved, weighted):
    rng = np.random.default_rng(3)
    B, S, H, D, n = 1, 2, 2, 8, 3
    x, w = rng.standard_normal((B, S, H, D)), rng.standard_normal(D)
    pos, freq, axis = rng.integers(-9, 9, (B, S, 2)), rng.random(n), [0, 1, 1]
    dy = rng.standard_normal((B, H, S, D))
    kw = dict(positions=pos, inv_freq=freq, axis=axis, interleaved=interleaved, eps=1e-3)
    f = lambda xx, ww: float((oracle.rope_fwd(xx, ww if weighted else None, **kw) * dy).sum())  # noqa: E731
    dx, dw = oracle.rope_bwd(dy, x, w if weighted else None, **kw)[:2]
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if weighted:
        for d in range(D):
            e = np.zeros(D)
            e[d] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[d]) < 1e-7


def test_plan():
    p = rope.rope_plan((4, 8), base=100.0)
    assert p.inv_freq.tolist() == pytest.approx([1.0, 0.1, 1.0, 100 ** -0.25, 0.1, 100 ** -0.75])
    assert p.axis.tolist() == [0, 0, 1, 1, 1, 1] and not p.interleaved
    assert rope.rope_plan(8).inv_freq.numel() == 4
    for bad in ((3,), (), (-2,), (2,) * 9):
        with pytest.raises(ValueError):
            rope.rope_plan(bad)


# Fake, never dereferenced device addresses: validation runs before any CUDA call.
A, T = 0x7F0000000000, 1 << 30


class _Part(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("x", "stride_b", "stride_s", "stride_h", "heads", "weight")] + \
               [("weight_f32", ctypes.c_int), ("turn", ctypes.c_int)] + \
               [(n, ctypes.c_int64) for n in ("y", "dx", "dx_stride_b", "dx_stride_s", "dx_stride_h", "dweight")]


def _args(n=1, B=2, S=16, D=64, H=4, **over):
    parts = (_Part * max(n, 1))()
    for i in range(n):
        parts[i] = _Part(A + i * T, S * H * D, H * D, D, H, A + 8 * T + i * 1024, 0, 1, A + (10 + i) * T,
                         A + (20 + i) * T, S * H * D, H * D, D, A + 9 * T + i * 1024)
    for name, value in over.items():
        setattr(parts[0], name, value or 0)
    return parts


FREQ = (ctypes.c_double * 32)(*[0.5] * 32)
AXIS = (ctypes.c_uint8 * 32)(*[0] * 32)


def _rope_struct(freq=FREQ, axis=AXIS, pairs=32, interleaved=0):
    return rope._pack_rope(ctypes.addressof(freq) if freq else 0, ctypes.addressof(axis) if axis else 0, pairs, interleaved)


def _at(at=A + 30 * T, b=16, s=1, a=0, axes=1):
    return rope._pack_positions(at, b, s, a, axes)


def _call(lib, bwd, parts, n=1, r=None, at=None, B=2, S=16, D=64, eps=1e-6, dtype=0, ws=A + 31 * T, space=1 << 28):
    r, at, parts = _rope_struct() if r is None else r, _at() if at is None else at, bytes(parts)
    if bwd:
        return lib.attn_rope_bwd(parts, n, r, at, B, S, D, eps, dtype, ws, space, None)
    return lib.attn_rope_fwd(parts, n, r, at, B, S, D, eps, dtype, None)


KEEP = []


def _array(ctype, value):
    """32 equal values that outlive the parametrisation."""
    KEEP.append((ctype * 32)(*[value] * 32))
    return KEEP[-1]


BAD, UNSUP, MIS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED, binding.ATTN_ERR_MISALIGNED


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(x=0), BAD), (dict(y=0), BAD), (dict(heads=0), BAD), (dict(heads=1 << 27), BAD), (dict(turn=2), BAD),
    (dict(weight_f32=-1), BAD), (dict(stride_s=-256), BAD), (dict(stride_h=12), BAD), (dict(stride_b=1 << 41), BAD),
    (dict(x=A + 8), MIS), (dict(y=A + 10 * T + 4), MIS), (dict(weight=A + 8 * T + 2), MIS),
])
def test_refused_parts(lib, bwd, over, code):
    assert _call(lib, bwd, _args(**over)) == code


@pytest.mark.parametrize("over,code", [
    (dict(dx=0), BAD), (dict(dx=A + 20 * T + 8), MIS), (dict(dweight=A + 9 * T + 1), MIS),
    (dict(dx_stride_h=0), BAD),                 # heads share a place
    (dict(dx_stride_s=128), BAD),               # tokens overlap
    (dict(weight=None), BAD),                   # dweight without weight
    (dict(dx=A), BAD),                          # dx is x
    (dict(dx=A + 10 * T), BAD),                 # dx is dy
    (dict(dweight=A + 64), BAD),                # dweight in x
    (dict(dweight=A + 8 * T), BAD),             # dweight is weight
])
def test_refused_gradients(lib, over, code):
    assert _call(lib, True, _args(**over)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), BAD), (dict(n=5), BAD), (dict(B=0), BAD), (dict(S=0), BAD), (dict(B=1 << 20, S=1 << 20), BAD),
    (dict(D=60), UNSUP), (dict(D=264), UNSUP), (dict(D=0), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(dtype=2), BAD),
    (dict(r=_rope_struct(pairs=33)), BAD), (dict(r=_rope_struct(pairs=-1)), BAD), (dict(r=_rope_struct(freq=None)), BAD),
    (dict(r=_rope_struct(interleaved=2)), BAD),
    (dict(r=_rope_struct(freq=_array(ctypes.c_double, float("inf")))), BAD),
    (dict(r=_rope_struct(freq=_array(ctypes.c_double, 2e6))), BAD),
    (dict(r=_rope_struct(axis=_array(ctypes.c_uint8, 1))), BAD),
    (dict(at=_at(at=0)), BAD), (dict(at=_at(at=A + 2)), MIS), (dict(at=_at(axes=0)), BAD), (dict(at=_at(axes=9)), BAD),
    (dict(at=_at(b=-1)), BAD), (dict(at=_at(s=1 << 41)), BAD),
])
def test_refused_calls(lib, kw, code):
    for bwd in (False, True):
        assert _call(lib, bwd, _args(), **kw) == code


def test_refused_overlaps(lib):
    two = _args(2)
    two[1].y = two[0].y + 4096
    assert _call(lib, False, two, n=2) == BAD
    two = _args(2)
    two[1].x = two[0].y + 64
    assert _call(lib, False, two, n=2) == BAD
    one = _args(1)
    assert _call(lib, False, one, at=_at(at=one[0].y + 128)) == BAD
    # gradients of a packed projection lie beside one another; shifted by less than a head they do not
    B, S, H, D = 2, 16, 4, 64
    for shift, code in ((H * D, None), (H * D - 8, BAD), (3 * H * D, BAD)):
        two = _args(2)
        for i in range(2):
            two[i].dx_stride_b, two[i].dx_stride_s = S * 2 * H * D, 2 * H * D
            two[i].dx = A + 20 * T + i * shift * 2
        # a sound layout goes on to the first CUDA call, which fails here
        got = _call(lib, True, two, n=2)
        assert (got == code) if code else (got not in (BAD, MIS))


def test_refused_workspace_overlaps(lib):
    one = _args(1)
    for ws in (one[0].dx + 64, one[0].y, one[0].x, one[0].weight, one[0].dweight, A + 30 * T):
        assert _call(lib, True, one, ws=ws, space=4096) == BAD


def test_workspace_right_behind_a_weight(lib):
    """16-bit weights end after 2 bytes a channel: what lies behind is free."""
    one = _args(1, D=128, dweight=0)
    got = _call(lib, True, one, D=128, ws=one[0].weight + 256, space=1 << 20)
    assert got not in (BAD, MIS)


@pytest.mark.parametrize("over", [dict(stride_b=1 << 50), dict(stride_s=1 << 44), dict(stride_h=1 << 57)])
def test_refused_strides_past_64_bits(lib, over):
    for bwd in (False, True):
        assert _call(lib, bwd, _args(**over), B=1 << 14, S=1 << 15) == BAD


def test_workspace_sizes_without_weights(lib):
    parts = bytes(_args(1, dweight=0))
    assert lib.attn_rope_bwd_workspace(parts, 1, 2, 16, 64) == 16
    assert lib.attn_rope_bwd_workspace(parts, 0, 2, 16, 64) == 0
    assert lib.attn_rope_bwd_workspace(parts, 1, 2, 16, 60) == 0


def test_binding_refuses_bad_tensors():
    x = torch.zeros(1, 4, 2, 8, dtype=torch.bfloat16)
    plan = rope.rope_plan(8)
    with pytest.raises(ValueError):
        rope.rope_fwd((x,), plan, torch.zeros(1, 4, dtype=torch.int32))  # not on the GPU
    with pytest.raises(TypeError):
        rope.rope_fwd((x.float(),), plan, None)
    with pytest.raises(ValueError):
        rope.rope_fwd((), plan, None)


def _packed(lib, B, S, D, views, own=20):
    """The status of a gradient whose parts' dx are views (offset, strides of batch, token and head, heads) of one buffer."""
    parts = _args(len(views), B=B, S=S, D=D, dweight=0)
    for i, (at, sb, ss, sh, h) in enumerate(views):
        parts[i].dx, parts[i].dx_stride_b, parts[i].dx_stride_s, parts[i].dx_stride_h = A + own * T + 2 * at, sb, ss, sh
        parts[i].heads, parts[i].dweight = h, 0
    return _call(lib, True, parts, n=len(views), B=B, S=S, D=D, r=_rope_struct(pairs=4))


B_, S_, H_, D_ = 3, 5, 4, 64
LAYOUTS = {  # of q, k and v in one buffer of B·S·3·H·D values: strides of batch, token and head, and how far apart they begin
    "[B,S,3,H,D]": (S_ * 3 * H_ * D_, 3 * H_ * D_, D_, H_ * D_),
    "[S,B,3,H,D]": (3 * H_ * D_, B_ * 3 * H_ * D_, D_, H_ * D_),
    "[B,S,H,3,D]": (S_ * 3 * H_ * D_, 3 * H_ * D_, 3 * D_, D_),
    "[S,B,H,3,D]": (3 * H_ * D_, B_ * 3 * H_ * D_, 3 * D_, D_),
    "[B,3,H,S,D]": (3 * H_ * S_ * D_, D_, S_ * D_, H_ * S_ * D_),
    "[B,H,3,S,D]": (3 * H_ * S_ * D_, D_, 3 * S_ * D_, S_ * D_),
    "[H,B,S,3,D]": (S_ * 3 * D_, 3 * D_, B_ * S_ * 3 * D_, D_),
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_packed_gradients_of_any_order(lib, layout):
    sb, ss, sh, step = LAYOUTS[layout]
    views = [(i * step, sb, ss, sh, H_) for i in range(3)]
    # a sound layout goes on to the first CUDA call, which fails here
    assert _packed(lib, B_, S_, D_, views) not in (BAD, MIS)
    assert _packed(lib, B_, S_, D_, views[::-1]) not in (BAD, MIS)
    for i in range(3):
        for shift in (8, -8, D_ - 8):
            moved = [(at + (shift if j == i else 0), *rest) for j, (at, *rest) in enumerate(views)]
            assert _packed(lib, B_, S_, D_, moved) == BAD


def test_packed_gradients_of_shared_heads(lib):
    """q's heads, then k's and v's in pairs, of one token after the other; and with batch and tokens swapped."""
    B, S, D, Hq, Hkv = 2, 7, 64, 8, 2
    W = (Hq + 2 * Hkv) * D
    for sb, ss in ((S * W, W), (W, B * W)):
        views = [(0, sb, ss, D, Hq), (Hq * D, sb, ss, 2 * D, Hkv), ((Hq + 1) * D, sb, ss, 2 * D, Hkv)]
        assert _packed(lib, B, S, D, views) not in (BAD, MIS)
        views[1] = (Hq * D - D, sb, ss, 2 * D, Hkv)
        assert _packed(lib, B, S, D, views) == BAD


def _places(view, B, S, D):
    at, sb, ss, sh, h = view
    return {at + b * sb + s * ss + i * sh + d for b in range(B) for s in range(S) for i in range(h) for d in range(D)}


def test_packed_gradients_against_the_places_themselves(lib):
    """Random views: refused where any two values share a place; and taken as parts of a packed tensor with its
    dimensions in random order."""
    rng = np.random.default_rng(17)
    D, shared = 8, 0
    for _ in range(4000):
        B, S, h = (int(x) for x in rng.integers(1, 4, 3))
        sizes, reach, strides = [B, S, h], D, [0, 0, 0]
        for i in rng.permutation(3):  # each dimension past what the inner ones reach, with room or none
            strides[i] = reach + 8 * int(rng.integers(0, 9)) * int(rng.integers(0, 2))
            reach += strides[i] * (sizes[i] - 1)
        views = [(0, *strides, h),
                 (8 * int(rng.integers(-40, 41)), *(x + 8 * int(rng.integers(0, 3)) * int(rng.integers(0, 2)) for x in strides),
                  int(rng.integers(1, h + 1)))]
        if _places(views[0], B, S, D) & _places(views[1], B, S, D):
            shared += 1
            assert _packed(lib, B, S, D, views) == BAD, (B, S, views)
        sizes, inner, strides = [B, S, h, 3], D, [0] * 4
        for i in rng.permutation(4):
            strides[i] = inner
            inner *= sizes[i]
        views = [(p * strides[3], *strides[:3], h) for p in rng.permutation(3)]
        assert _packed(lib, B, S, D, views) not in (BAD, MIS), (B, S, views)
    assert shared > 400


def test_rotary_attention_refuses_shared_heads_at_once():
    """Before the heads are turned, with the reason."""
    q, k = (torch.zeros(1, 4, h, 8, dtype=torch.bfloat16) for h in (4, 2))
    for args in ((q, k, k), (q, q, k), (q, k, q)):
        with pytest.raises(ValueError, match="share a shape"):
            rope.rotary_attention(*args)
