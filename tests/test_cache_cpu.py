"""CPU checks of the 8-bit cache: its C ABI is exported and refuses bad
arguments before touching CUDA, the binding refuses bad tensors, and the
oracle's pieces meet independent restatements."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cache as kv
from exact_attention_68_gb300.build import build_library
from oracle import cache as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK_NO_GPU = (binding.ATTN_ERR_CUDA, binding.ATTN_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    return kv.declare(binding.load_library(build_library()))


def test_header_declares_the_bound_symbols(lib):
    with open(os.path.join(ROOT, "include", "attn_cache.h")) as f:
        names = re.findall(r"ATTN_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", f.read())
    assert sorted(names) == sorted(kv.CACHE_SYMBOLS)
    for n in names:
        assert hasattr(lib, n)


# Fake, never dereferenced device addresses, far apart.
A, GB = 0x7F0000000000, 1 << 30


def _cache(**kw):
    d = dict(k=A, v=A + GB, k_scale=A + 2 * GB, v_scale=A + 3 * GB, k_bounds=A + 4 * GB, pages=100, heads=4,
             head_dim=128, page=64)
    d.update(kw)
    return kv._Cache(*[d[f] for f, _ in kv._Cache._fields_])


def _seqs(**kw):
    d = dict(table=A + 5 * GB, lens=A + 6 * GB, fresh=0, batch=3, width=20)
    d.update(kw)
    return kv._Seqs(*[d[f] for f, _ in kv._Seqs._fields_])


def _append(lib, c={}, s={}, k=A + 7 * GB, v=A + 8 * GB, T=2, dtype=0):
    return lib.attn_cache_append(_cache(**c), _seqs(**s), k, v, T, dtype, None)


def _fwd(lib, c={}, s={}, q=A + 7 * GB, pages=0, listed=0, out=A + 8 * GB, lse=A + 9 * GB, mass=0, q_heads=8, T=2,
         scale=0.1, dtype=0, ws=A + 10 * GB, ws_bytes=1 << 28):
    return lib.attn_cache_fwd(_cache(**c), _seqs(**s), q, pages, listed, out, lse, mass, q_heads, T, scale, dtype, ws,
                              ws_bytes, 0, None)


def _select(lib, c={}, s={}, q=A + 7 * GB, q_heads=8, T=2, dtype=0, count=5, pages=A + 8 * GB, scores=A + 9 * GB):
    return lib.attn_cache_select(_cache(**c), _seqs(**s), q, q_heads, T, dtype, count, pages, scores, None)


def _evict(lib, c={}, s={}, mass=A + 7 * GB, dst=A + 8 * GB, dst_width=5, keep=300, recent=10, kept=A + 9 * GB,
           new_lens=A + 10 * GB, mass_out=A + 11 * GB, ws=A + 12 * GB, ws_bytes=1 << 20):
    return lib.attn_cache_evict(_cache(**c), _seqs(**s), mass, dst, dst_width, keep, recent, kept, new_lens, mass_out,
                                ws, ws_bytes, None)


CALLS = [_append, _fwd, _select, _evict]
INV, UNS, MIS = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED, binding.ATTN_ERR_MISALIGNED


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("c,s,code", [
    (dict(k=0), {}, INV), (dict(v=0), {}, INV), (dict(k_scale=0), {}, INV), (dict(v_scale=0), {}, INV),
    (dict(k_bounds=0), {}, INV), (dict(pages=0), {}, INV), (dict(heads=0), {}, INV), (dict(head_dim=0), {}, INV),
    (dict(head_dim=100), {}, UNS), (dict(head_dim=264), {}, UNS), (dict(page=8), {}, UNS), (dict(page=48), {}, UNS),
    (dict(page=128), {}, UNS), (dict(heads=65536), {}, INV), (dict(pages=1 << 31), {}, INV),
    (dict(pages=1 << 24, heads=8), {}, INV),
    ({}, dict(table=0), INV), ({}, dict(lens=0), INV), ({}, dict(batch=0), INV), ({}, dict(batch=65535), INV),
    ({}, dict(width=0), INV), ({}, dict(width=1 << 26), INV),
    (dict(k=A + 8), {}, MIS), (dict(v=A + GB + 1), {}, MIS), (dict(k_bounds=A + 4 * GB + 4), {}, MIS),
    (dict(k_scale=A + 2 * GB + 2), {}, MIS), ({}, dict(table=A + 5 * GB + 1), MIS),
    ({}, dict(lens=A + 6 * GB + 2), MIS), ({}, dict(fresh=A + 6 * GB + 65537), MIS),
])
def test_bad_caches_and_sequences_are_refused(lib, call, c, s, code):
    assert call(lib, c=c, s=s) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), INV), (dict(v=0), INV), (dict(T=0), INV), (dict(T=1 << 31), INV), (dict(dtype=2), INV),
    (dict(k=A + 7 * GB + 8), MIS), (dict(k=A + 64), INV), (dict(v=A + 2 * GB), INV), (dict(T=1 << 30, s=dict(batch=60000)), INV),
    (dict(c=dict(v=A)), INV), (dict(s=dict(lens=A + 16)), INV),
])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INV), (dict(out=0), INV), (dict(lse=0), INV), (dict(dtype=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(scale=-1.0), INV),
    (dict(q_heads=0), INV), (dict(q_heads=6), INV), (dict(T=0), INV), (dict(T=65), INV),
    (dict(listed=4), INV), (dict(pages=A + 11 * GB, listed=0), INV), (dict(pages=A + 11 * GB, listed=-1), INV),
    (dict(pages=A + 11 * GB + 2, listed=4), MIS), (dict(q=A + 7 * GB + 8), MIS), (dict(out=A + 8 * GB + 4), MIS),
    (dict(lse=A + 9 * GB + 1), MIS), (dict(mass=A + 11 * GB + 3), MIS), (dict(ws=A + 10 * GB + 8), MIS),
    (dict(s=dict(width=1 << 24, batch=60000), q_heads=4096, T=64), INV),
])
def test_fwd_refuses(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INV), (dict(pages=0), INV), (dict(scores=0), INV), (dict(count=0), INV), (dict(count=1 << 31), INV),
    (dict(dtype=7), INV), (dict(q_heads=3), INV), (dict(T=65), INV), (dict(q=A + 7 * GB + 2), MIS),
    (dict(pages=A + 8 * GB + 1), MIS), (dict(scores=A + 8 * GB + 16), INV), (dict(scores=A + 4 * GB), INV),
])
def test_select_refuses(lib, kw, code):
    assert _select(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mass=0), INV), (dict(dst=0), INV), (dict(kept=0), INV), (dict(new_lens=0), INV), (dict(mass_out=0), INV),
    (dict(ws=0), INV), (dict(ws_bytes=16), INV), (dict(dst_width=0), INV), (dict(keep=0), INV),
    (dict(keep=321), INV), (dict(recent=-1), INV), (dict(recent=301), INV), (dict(ws=A + 12 * GB + 8), MIS),
    (dict(mass_out=A + 7 * GB), INV), (dict(dst=A + 5 * GB, new_lens=A + 5 * GB), INV), (dict(kept=A), INV),
])
def test_evict_refuses(lib, kw, code):
    assert _evict(lib, **kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("call", CALLS)
def test_good_arguments_get_as_far_as_the_device(lib, call):
    assert call(lib) in OK_NO_GPU


def test_workspace_sizes_refuse_what_the_calls_refuse(lib):
    assert lib.attn_cache_evict_workspace(_cache(), _seqs(), 5) == 2 * 4 * 4 + 64  # 2 bitmaps of 100 pages, 15 entries
    assert lib.attn_cache_evict_workspace(_cache(page=8), _seqs(), 5) == 0
    assert lib.attn_cache_evict_workspace(_cache(), _seqs(), 0) == 0
    assert lib.attn_cache_fwd_workspace(_cache(head_dim=12), _seqs(), 0, 8, 1, 0) == 0


def test_binding_refuses_host_and_misshapen_tensors():
    c = kv.cache_alloc(4, 2, 64, 16, device="cpu")
    with pytest.raises(TypeError, match="CUDA"):
        kv.cache_append(c, None, None, None, None)
    for kw in (dict(page=8), dict(head_dim=12), dict(head_dim=264), dict(pages=0), dict(heads=0)):
        with pytest.raises(ValueError):
            kv.cache_alloc(**{**dict(pages=4, heads=2, head_dim=64, page=16, device="cpu"), **kw})


# ---------------------------------------------------------------- the oracle's pieces
def test_oracle_decodes_and_rounds_e4m3_like_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ours, theirs = oc.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).normal(0, s, 4000) for s in (1e-3, 0.1, 10, 200)])
    edges = np.sort(np.abs(ours[np.isfinite(ours)]))
    x = np.concatenate([x, edges, (edges[1:] + edges[:-1]) / 2, -(edges[1:] + edges[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oc.e4m3_codes(x), want)
    assert np.isnan(oc.e4m3_values()[oc.e4m3_codes(np.nan)])
    assert oc.e4m3_values()[oc.e4m3_codes(np.inf)] == 448


@pytest.mark.parametrize("a", [0.0, 1e-40, 448.0, 448.0001, 1.75, 1.7500001, 3e38, 2.0 ** -100, 0.4375])
def test_oracle_page_scale_is_the_smallest_that_holds(a):
    s = oc.page_scale(np.array([-a, a / 3]))
    assert a <= 448 * s and math.log2(s) == int(math.log2(s))
    assert s == 2.0 ** -100 or a > 448 * s / 2


def test_oracle_attention_meets_the_dense_oracle():
    """A cache whose pages hold exactly representable values: the attention of
    the last tokens equals the dense causal attention's last rows."""
    from oracle import attention_fwd
    rng = np.random.default_rng(3)
    B, H, S, D, P, T = 2, 2, 37, 16, 16, 3
    k, v = (oc.e4m3_values()[rng.integers(0, 127, (B, H, S, D))] * rng.choice([-1, 1], (B, H, S, D)) / 64 for _ in "kv")
    q = rng.normal(size=(B, 2 * H, S, D))
    pool = dict(k=np.zeros((9, H, P, 16), np.uint8), v=np.zeros((9, H, P, 16), np.uint8),
                k_scale=np.ones((9, H), np.float32), v_scale=np.ones((9, H), np.float32),
                k_bounds=np.zeros((9, H, 2, 16), np.int8), head_dim=D)
    table = rng.permutation(9)[:6].reshape(2, 3)
    lens, fresh = np.array([S, S]), np.array([S, S])
    oc.cache_append(pool, table, lens, fresh, k, v)
    out, lse, mass, _, _ = oc.cache_attention(pool, table, lens, np.array([T, T]), q[:, :, -T:], 0.25)
    held = {}
    for n, x in (("k", k), ("v", v)):
        full = oc.e4m3_values()[pool[n][table]] * pool[n + "_scale"][table][..., None, None].astype(float)
        held[n] = full.transpose(0, 2, 1, 3, 4).reshape(B, H, 48, 16)[:, :, :S]
        assert np.abs(held[n] - x).max() <= np.abs(x).max() * 2.0 ** -9  # subnormals under the page's scale
    for h in range(2 * H):
        ro, rl = attention_fwd(q[:, h:h + 1], held["k"][:, h // 2:h // 2 + 1], held["v"][:, h // 2:h // 2 + 1], 0.25, True)
        assert np.allclose(out[:, h], ro[:, 0, -T:], atol=1e-12) and np.allclose(lse[:, h], rl[:, 0, -T:], atol=1e-12)
    assert np.allclose(mass.sum(2), 2 * T)


def test_oracle_bounds_widen_while_the_scale_stays():
    """A channel of NaN codes leaves 0 inside, tokens taken back their bounds, until the scale grows."""
    pool = dict(k=np.zeros((2, 1, 16, 16), np.uint8), v=np.zeros((2, 1, 16, 16), np.uint8),
                k_scale=np.ones((2, 1), np.float32), v_scale=np.ones((2, 1), np.float32),
                k_bounds=np.full((2, 1, 2, 16), 99, np.int8), head_dim=16)
    table = np.array([[1]])

    def append(x, n):
        x = np.asarray(x, float).reshape(1, 1, -1, 1) * np.ones(16)
        x[..., 0] = np.where(np.isnan(x[..., 1]), 448.0, x[..., 1])
        oc.cache_append(pool, table, np.array([n]), np.array([x.shape[2]]), x, x)
        return pool["k_bounds"][1, 0, :, 1].tolist()

    assert append([np.nan, np.nan], 2) == [0, 0]
    assert append([112.0], 3) == [math.ceil(112 * 127 / 448), 0]
    assert append([224.0, 224.0], 5) == [math.ceil(224 * 127 / 448), 0]
    assert append([56.0], 4) == [math.ceil(224 * 127 / 448), 0]  # one of the two taken back, another in its place
    assert append([896.0], 5)[1] == math.floor(28 * 127 / 448)   # a larger scale: found anew, 56 / 2 the least
    assert (pool["k_bounds"][0] == 99).all()


def test_oracle_evicts_nan_weights_first():
    pool = {n: np.zeros((3, 1, 16, 16), np.uint8) for n in "kv"}
    pool.update(k_scale=np.ones((3, 1), np.float32), v_scale=np.ones((3, 1), np.float32),
                k_bounds=np.zeros((3, 1, 2, 16), np.int8), head_dim=16)
    mass = np.full((1, 1, 16), -np.inf, np.float32)
    mass[0, 0, [0, 1, 5]], mass[0, 0, [3, 7]] = np.nan, 1.0
    kept, lens, _ = oc.cache_evict(pool, mass, np.array([[0]]), np.array([10]), np.array([[2]]), 6, 1)
    assert kept[0, 0].tolist() == [2, 3, 4, 6, 7, 9] and lens.tolist() == [6]
