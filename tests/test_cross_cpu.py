"""CPU checks of cross-attention: the oracle against differences and against the
self-attention oracle, and the library's refusals (no CUDA call is reached)."""
import os
import re

import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cross
from exact_attention_68_gb300.build import build_library
from oracle import attention_bwd, attention_fwd
from oracle import cross as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return cross.declare(binding.load_library(build_library()))


def test_header_declares_the_bound_symbols(lib):
    with open(os.path.join(ROOT, "include", "attn_cross.h")) as f:
        names = re.findall(r"ATTN_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", f.read())
    assert sorted(names) == sorted(cross.CROSS_SYMBOLS)
    for n in names:
        assert hasattr(lib, n)


def test_oracle_is_the_self_attention_oracle_where_both_apply():
    rng = np.random.default_rng(1)
    q, k, v, dout = (rng.standard_normal((2, 3, 7, 8)) for _ in range(4))
    ro, rl = attention_fwd(q, k, v, 0.3, False)
    out, lse = oracle.cross_fwd(q, k, v, [7, 7], 0.3)
    np.testing.assert_allclose(out, ro, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(lse, rl, rtol=1e-13)
    got = oracle.cross_bwd(q, k, v, out, lse, dout, [7, 7], 0.3)[:3]
    for a, b in zip(got, attention_bwd(q, k, v, dout, 0.3, False)):
        np.testing.assert_allclose(a, b, rtol=1e-11, atol=1e-13)


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(2)
    B, Hq, Hkv, Sq, Sk, D, lens, scale = 3, 4, 2, 2, 5, 3, [5, 0, 3], 0.7
    q, dout = rng.standard_normal((2, B, Hq, Sq, D))
    k, v = rng.standard_normal((2, B, Hkv, Sk, D))
    out, lse = oracle.cross_fwd(q, k, v, lens, scale)
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
    grads = oracle.cross_bwd(q, k, v, out, lse, dout, lens, scale)[:3]
    args = [q, k, v]
    for which in range(3):
        for i in np.ndindex(args[which].shape):
            d = []
            for sign in (1, -1):
                x = [a.copy() for a in args]
                x[which][i] += sign * 1e-6
                d.append((oracle.cross_fwd(*x, lens, scale)[0] * dout).sum())
            assert abs((d[0] - d[1]) / 2e-6 - grads[which][i]) < 1e-7
    assert (grads[1][2, :, 3:] == 0).all() and (grads[2][1] == 0).all()


# Fake, never dereferenced device addresses: validation runs before any CUDA call.
A, T = 0x7F0000000000, 1 << 30
BAD, UNSUP, MIS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED, binding.ATTN_ERR_MISALIGNED


def _sizes(batch=2, q_heads=8, heads=4, Sq=16, Sk=40, head_dim=64):
    return cross._pack_sizes(batch, q_heads, heads, Sq, Sk, head_dim)


def _fwd(lib, sizes=None, q=A, k=A + T, v=A + 2 * T, lens=A + 3 * T, out=A + 4 * T, lse=A + 5 * T, scale=0.125, dtype=0,
         ws=None, space=0):
    return lib.attn_cross_fwd(sizes or _sizes(), q, k, v, lens, out, lse, scale, dtype, ws, space, 0, None)


def _bwd(lib, sizes=None, q=A, k=A + T, v=A + 2 * T, lens=A + 3 * T, out=A + 4 * T, lse=A + 5 * T, dout=A + 6 * T,
         dq=A + 7 * T, dk=A + 8 * T, dv=A + 9 * T, delta=A + 10 * T, scale=0.125, dtype=0, ws=None, space=0):
    return lib.attn_cross_bwd(sizes or _sizes(), q, k, v, lens, out, lse, dout, dq, dk, dv, delta, scale, dtype, ws, space,
                              0, None)


SIZES = [
    (dict(batch=0), BAD), (dict(heads=0), BAD), (dict(q_heads=0), BAD), (dict(Sq=0), BAD), (dict(Sk=0), BAD),
    (dict(head_dim=0), BAD), (dict(q_heads=6), BAD), (dict(head_dim=60), UNSUP), (dict(head_dim=264), UNSUP),
    (dict(Sq=1 << 31), BAD), (dict(Sk=1 << 31), BAD), (dict(Sq=1 << 30), BAD), (dict(batch=1 << 30), BAD),
    (dict(batch=1 << 20, q_heads=1 << 14, heads=1 << 14), BAD),
]


@pytest.mark.parametrize("kw,code", SIZES)
def test_refused_sizes(lib, kw, code):
    s = _sizes(**kw)
    assert _fwd(lib, s) == code and _bwd(lib, s) == code
    assert lib.attn_cross_fwd_workspace(s) == 0 and lib.attn_cross_bwd_workspace(s) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(out=0), BAD), (dict(lse=0), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(dtype=2), BAD), (dict(q=A + 8), MIS),
    (dict(k=A + T + 2), MIS), (dict(out=A + 4 * T + 4), MIS), (dict(lse=A + 5 * T + 2), MIS), (dict(lens=A + 3 * T + 1), MIS),
    (dict(lse=A + 64), BAD),
])
def test_refused_arguments(lib, kw, code):
    assert _fwd(lib, **kw) == code
    assert _bwd(lib, **kw) == code or kw == dict(lse=A + 64)  # the gradient reads both: no overlap of what is written


@pytest.mark.parametrize("kw,code", [
    (dict(dout=0), BAD), (dict(dq=0), BAD), (dict(dk=0), BAD), (dict(dv=0), BAD), (dict(delta=0), BAD),
    (dict(dq=A + 7 * T + 8), MIS), (dict(dv=A + 9 * T + 2), MIS), (dict(delta=A + 10 * T + 2), MIS),
    (dict(dq=A), BAD), (dict(dk=A + T), BAD), (dict(dv=A + 8 * T), BAD), (dict(delta=A + 5 * T), BAD),
    (dict(dq=A + 6 * T), BAD), (dict(dk=A + 3 * T), BAD), (dict(ws=A + 9 * T, space=4096), BAD),
])
def test_refused_gradients(lib, kw, code):
    assert _bwd(lib, **kw) == code


def test_refused_overlaps_of_the_forward(lib):
    for kw in (dict(out=A), dict(out=A + T), dict(out=A + 2 * T + 4096), dict(lse=A + 4 * T), dict(out=A + 3 * T),
               dict(ws=A + 4 * T, space=64)):
        assert _fwd(lib, **kw) == BAD


def test_binding_refuses_bad_tensors():
    q = torch.zeros(1, 2, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cross.cross_fwd(q, q, q)  # not on the GPU
    with pytest.raises(TypeError):
        cross.cross_fwd(q.float(), q, q)
    with pytest.raises(TypeError):
        cross.cross_fwd(q, q.half(), q)
