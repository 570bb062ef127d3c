"""GPU tests of what cross-attention and its gradient answer where values are not finite, where a gradient's
sums have few terms or are cut at a near tie, and past 4 GiB (the oracle is oracle/cross.py)."""
import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cross
from oracle import cross as oracle
from test_gpu_o_cross import check, check_bwd, half_step, n64, problem

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# B, Hq, Hkv, Sq, Sk, lens, D: each gradient kernel, a tile or more with keys that are not there beside ones that are
GRADS = [
    ((2, 2, 2, 30, 40, [33, 5]), 64), ((2, 4, 2, 20, 64, [50, 17]), 128), ((2, 2, 1, 7, 60, [3, 59]), 256),
    ((2, 2, 2, 300, 400, [333, 5]), 64), ((2, 4, 2, 70, 900, [800, 130]), 128), ((2, 2, 2, 150, 300, [290, 70]), 256),
]


@pytest.mark.parametrize("shape,D", GRADS, ids=str)
@pytest.mark.parametrize("what", ["q", "dout"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_keys_that_are_not_there_have_no_gradient_whatever_the_queries_are(cuda_device, shape, D, what, value):
    """A query or upstream gradient that is not finite: its own dq and the keys of its head take it, keys behind
    the end get 0 all the same, and other rows and heads what they get without it."""
    B, Hq, Hkv, Sq, Sk, lens = shape
    q, k, v, dout, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, torch.bfloat16, seed=Sq + D)
    out, lse = cross.cross_fwd(q, k, v, ln)
    clean = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    (q if what == "q" else dout)[1, 0, 2, 3] = value
    dq, dk, dv, _ = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    for b, n in enumerate(lens):
        assert (dk[b, :, n:] == 0).all() and (dv[b, :, n:] == 0).all()
    assert not dq[1, 0, 2].isfinite().all() and not (dk[1, 0, :lens[1]].isfinite().all() and dv[1, 0, :lens[1]].isfinite().all())
    for got, want in zip((dk, dv), clean[1:3]):
        got = got.clone()
        got[1, 0] = want[1, 0]
        assert torch.equal(got, want)
    dq = dq.clone()
    dq[1, 0, 2] = clean[0][1, 0, 2]
    assert torch.equal(dq, clean[0])


@pytest.mark.parametrize("steps", [63, 83, 104, 124])
def test_gradient_where_two_numbers_of_runs_cost_nearly_the_same(cuda_device, steps):
    """497 key tiles of 56 channels: cutting the sums over the queries into two runs costs what three do to a part in
    2^24, and the kernels of a call have to settle it alike.  NaN in the workspace shows a run that nobody wrote."""
    H, Sq, Sk, D = 71, 128 * steps, 896, 56
    g = torch.Generator(device="cuda").manual_seed(steps)
    q, dout = (torch.randn(1, H, Sq, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "qd")
    k, v = (torch.randn(1, H, Sk, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    out, lse = cross.cross_fwd(q, k, v)
    space = torch.full((cross.cross_bwd_workspace(q, k),), 0xff, dtype=torch.uint8, device="cuda")
    _, dk, dv, delta = cross.cross_bwd(q, k, v, out, lse, dout, workspace=space)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    h, scale = 2.0 ** -8, D ** -0.5
    for i in range(H):
        p = torch.exp(q[0, i].double() @ k[0, i].double().T * scale - lse[0, i].double()[:, None])
        dp, d = dout[0, i].double() @ v[0, i].double().T, delta[0, i].double()[:, None]
        ds = p * (dp - d)
        refs = (scale * ds.T @ q[0, i].double(), p.T @ dout[0, i].double())
        mags = (scale * ds.abs().T @ q[0, i].double().abs(), p.T @ dout[0, i].double().abs())
        m2 = scale * (p * (dp.abs() + d.abs())).T @ q[0, i].double().abs()
        # P and dS are rounded to bf16, the result is; fp32 for the rest
        assert ((dk[0, i].double() - refs[0]).abs() <= h * mags[0] + 2.0 ** -12 * m2 + h * refs[0].abs()).all()
        assert ((dv[0, i].double() - refs[1]).abs() <= (h + 2.0 ** -12) * mags[1] + h * refs[1].abs()).all()


# B, Hq, Hkv, Sq, Sk, lens, D: a CTA a slice, clusters, clusters and runs; tiles and runs of them, 128 and 64 keys a step
FORWARDS = [
    ((3, 4, 2, 2, 40, [40, 0, 17]), 64), ((2, 2, 2, 5, 700, [650, 300]), 64), ((1, 4, 1, 3, 20000, [19999]), 64),
    ((2, 2, 2, 150, 300, [300, 200]), 64), ((3, 2, 2, 40, 400, [390, 0, 130]), 128), ((1, 4, 2, 64, 6000, [5500]), 128),
    ((2, 2, 2, 150, 300, [300, 200]), 192), ((1, 2, 2, 30, 6000, [5500]), 256), ((2, 2, 1, 20, 100, [90, 70]), 256),
]


def _live_key(lens, b, i):
    """Places of keys that are there: the first, one in the middle, the last."""
    return (0, lens[b] // 2, lens[b] - 1)[i % 3]


@pytest.mark.parametrize("shape,D", FORWARDS, ids=str)
def test_keys_and_values_that_are_not_finite(cuda_device, shape, D):
    """A key of NaN, or of an infinity that gives +inf scores, makes the rows that meet it NaN; with -inf scores it is
    as if it were not there; a NaN value is its channel's.  However the keys are cut, and for no other head."""
    B, Hq, Hkv, Sq, Sk, lens = shape
    q, k, v, _, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, torch.bfloat16, seed=Sk + D)
    q[..., 0] = q[..., 0].abs() + 0.5
    q[..., ::2, 0] *= -1.0  # every other query's score against an infinite key is -inf, the others' +inf
    k[..., 0] = k[..., 0].nan_to_num(0.0)
    G = Hq // Hkv
    want, wantl = cross.cross_fwd(q, k, v, ln)
    for i in range(3):
        at = _live_key(lens, 0, i)
        k2 = k.clone()
        k2[0, 0, at, 1] = NAN
        out, lse = cross.cross_fwd(q, k2, v, ln)
        assert out[0, :G].isnan().all() and lse[0, :G].isnan().all()
        assert torch.equal(out[0, G:], want[0, G:]) and torch.equal(out[1:], want[1:])
        k2 = k.clone()
        k2[0, 0, at, 0] = INF
        out, lse = cross.cross_fwd(q, k2, v, ln)
        assert out[0, :G, 1::2].isnan().all() and lse[0, :G, 1::2].isnan().all()
        k3, v3 = k.clone(), v.clone()
        k3[0, 0, at, 0], v3[0, 0, at] = -1e30, 0.0  # a score far below the others, of the sign that is -inf above
        k3[0, 0, at, 0] *= -1.0
        ref, refl = cross.cross_fwd(q, k3, v3, ln)
        assert torch.equal(out[0, :G, ::2], ref[0, :G, ::2]) and torch.equal(lse[0, :G, ::2], refl[0, :G, ::2])
        v2 = v.clone()
        v2[0, 0, at, 3] = NAN
        out, lse = cross.cross_fwd(q, k, v2, ln)
        assert out[0, :G, :, 3].isnan().all() and torch.equal(lse, wantl)
        out[0, :G, :, 3] = want[0, :G, :, 3]
        assert torch.equal(out, want)
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("shape,D", FORWARDS, ids=str)
def test_no_score_but_minus_infinity_is_not_no_keys(cuda_device, shape, D):
    """All of a head's keys at -inf for some queries: 0 / 0 in out, -inf in lse; a sequence without keys keeps its 0.
    One finite key among them is the result."""
    B, Hq, Hkv, Sq, Sk, lens = shape
    q, k, v, _, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, torch.bfloat16, seed=Sk + D + 1)
    q[..., 0] = q[..., 0].abs() + 0.5
    G, full = Hq // Hkv, k[0, 0].clone()
    want, wantl = cross.cross_fwd(q, k, v, ln)
    k[0, 0, :lens[0], 0] = -INF
    out, lse = cross.cross_fwd(q, k, v, ln)
    assert out[0, :G].isnan().all() and torch.isneginf(lse[0, :G]).all()
    assert torch.equal(out[0, G:], want[0, G:]) and torch.equal(out[1:], want[1:])
    assert torch.equal(lse[0, G:], wantl[0, G:]) and torch.equal(lse[1:], wantl[1:])
    for i in range(3):
        at = _live_key(lens, 0, i)
        k[0, 0, :lens[0], 0], k[0, 0, at] = -INF, full[at]
        out, lse = cross.cross_fwd(q, k, v, ln)
        t = (q[0, :G].double() @ full[at].double()) * D ** -0.5
        assert (out[0, :G] == v[0, 0, at]).all()  # a weight of 1
        assert ((lse[0, :G].double() - t).abs() <= 2.0 ** -13 + t.abs() * 2.0 ** -22).all()
    assert binding.device_status() == binding.ATTN_OK


def test_gradients_past_four_gigabytes(cuda_device):
    """dq, delta, dk and dv of both heads, the second of which lies past 2^32 bytes and 2^31 values of k: dq as the
    sum over all keys, dk and dv at the first, the last and some keys between.  As the bounds of test_gpu_o_cross.py."""
    H, Sk, D, n = 2, 9_000_001, 128, 9_000_001 - 3
    g = torch.Generator(device="cuda").manual_seed(72)
    q, dout = (torch.randn(1, H, 2, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "qd")
    k, v = (torch.empty(1, H, Sk, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for t in (k, v):
        for h in range(H):
            for i in range(0, Sk, 1 << 20):
                part = t[0, h, i:i + (1 << 20)]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    k[0, :, -1000:] += 0.5 * q[0, :, :1]  # what lies far back decides
    v[0, :, -1000:] += 4.0
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    out, lse = cross.cross_fwd(q, k, v, lens)
    dq, dk, dv, delta = cross.cross_bwd(q, k, v, out, lse, dout, lens)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    scale, h_step = D ** -0.5, 2.0 ** -8
    want_delta = (dout.double() * out.double()).sum(-1)
    assert ((delta.double() - want_delta).abs() <= 2.0 ** -16 * (dout.double() * out.double()).abs().sum(-1)).all()
    for h in range(H):
        Q, dO, z, d = q[0, h].double(), dout[0, h].double(), lse[0, h].double()[:, None], delta[0, h].double()[:, None]
        ref, mag, mag2 = (torch.zeros(2, D, dtype=torch.double, device="cuda") for _ in range(3))
        for i in range(0, n, 1 << 20):
            kk, vv = (t[0, h, i:min(n, i + (1 << 20))].double() for t in (k, v))
            p = torch.exp(scale * (Q @ kk.T) - z)
            ds = p * (dO @ vv.T - d)
            ref += scale * ds @ kk
            mag += scale * ds.abs() @ kk.abs()
            mag2 += scale * (p * (dO.abs() @ vv.abs().T + d.abs())) @ kk.abs()
            last = i + (1 << 20) >= n
            at = torch.arange(kk.shape[0] - 1100, kk.shape[0], device="cuda") if last else torch.arange(64, device="cuda")
            w, s = p[:, at], ds[:, at]
            for got, r, m in ((dv[0, h, i + at], w.T @ dO, w.T @ dO.abs()),
                              (dk[0, h, i + at], scale * s.T @ Q, scale * s.abs().T @ Q.abs())):
                m2 = scale * (w * (dO.abs() @ vv[at].abs().T + d.abs())).T @ Q.abs() + w.T @ dO.abs()
                assert ((got.double() - r).abs() <= h_step * m + 2.0 ** -12 * m2 + h_step * r.abs()).all(), (h, i)
        # runs of 1e5 keys and more: their fp32 sums add 2^-10 of the magnitude at most
        assert ((dq[0, h].double() - ref).abs() <= (h_step + 2.0 ** -10) * mag + 2.0 ** -12 * mag2 + h_step * ref.abs()).all(), h
        assert dq[0, h].abs().min() > 0 and (dk[0, h, n:] == 0).all() and (dv[0, h, n:] == 0).all()


@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,lens", [
    (1, 1, 1, 1, 70, None), (2, 2, 2, 1, 700, [699, 130]), (1, 4, 2, 2, 5000, [4801]), (3, 2, 1, 20, 300, [300, 0, 129]),
    (1, 3, 3, 64, 257, None), (2, 6, 1, 20, 400, [257, 400]), (1, 2, 2, 128, 129, [128]), (40, 2, 2, 3, 200, None)])
@pytest.mark.parametrize("D", [64, 72, 128, 200, 256])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_gradients_of_few_queries_round_once(cuda_device, B, Hq, Hkv, Sq, Sk, lens, D, dt):
    """Slices whose queries are one tile: P and dS enter their products in two terms each, so that besides the fp32 sums
    only the results are rounded.  An fp16 term below 2^-14 loses 2^-25 at most.  Of the norm the results' own rounding
    is then all but a tenth: the rest is 2^-12 of the terms and less, against 2^-9 or 2^-12 that a rounding takes
    on average, and adds up as squares do."""
    q, k, v, dout, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, dt, seed=Sq + Sk + D)
    out, lse = cross.cross_fwd(q, k, v, ln)
    dq, dk, dv, delta = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    check_bwd(q, k, v, out, lse, dout, lens, D ** -0.5, (dq, dk, dv, delta))
    full = lens if lens is not None else [Sk] * B
    kk, vv = (np.nan_to_num(n64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (k, v))
    rq, rk, rv, _, (mq, mk, mv, m2q, m2k) = oracle.cross_bwd(n64(q), kk, vv, n64(out), n64(lse), n64(dout), full, D ** -0.5)
    h, tiny, G = half_step(dt), 2.0 ** -25 if dt == torch.float16 else 0.0, Hq // Hkv
    sq = np.stack([[D ** -0.5 * np.abs(kk[b, i // G, :full[b]]).sum(0) + 1 for i in range(Hq)] for b in range(B)])[:, :, None]
    sk = D ** -0.5 * np.abs(n64(q)).reshape(B, Hkv, -1, D).sum(2, keepdims=True) + 1
    sv = np.abs(n64(dout)).reshape(B, Hkv, -1, D).sum(2, keepdims=True) + 1
    for name, got, ref, m2, s in (("dq", dq, rq, m2q, sq), ("dk", dk, rk, m2k, sk), ("dv", dv, rv, mv, sv)):
        check(name, got, ref, h * np.abs(ref) + 2.0 ** -12 * m2 + tiny * s)
        err, own = (np.linalg.norm(n64(x) - ref) for x in (got, torch.from_numpy(ref).to(dt)))
        assert err <= 1.1 * own, (name, err / own)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Sk", [30000, 400000])
def test_fp16_weights_of_very_many_keys(cuda_device, D, Sk):
    """dv where most weights are below fp16's smallest normal value, 2^-14: as far off as with large ones, which is
    P's rounding and dv's own, each h of a value at most and of equal size: 1.42 times dv's own by norm."""
    Sq, dt = 300, torch.float16
    g = torch.Generator(device="cuda").manual_seed(Sk + D)
    q, dout = (torch.randn(1, 1, Sq, D, generator=g, device="cuda").to(dt) for _ in "qd")
    k, v = (torch.randn(1, 1, Sk, D, generator=g, device="cuda").to(dt) for _ in "kv")
    out, lse = cross.cross_fwd(q, k, v)
    dv = cross.cross_bwd(q, k, v, out, lse, dout)[2][0, 0].double()
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    ref = torch.empty_like(dv)
    for i in range(0, Sk, 1 << 16):
        t = q[0, 0].double() @ k[0, 0, i:i + (1 << 16)].double().T * D ** -0.5
        ref[i:i + (1 << 16)] = torch.exp(t - lse[0, 0].double()[:, None]).T @ dout[0, 0].double()
    # dv itself is partly below 2^-14: its own rounding counts that
    own = (ref.to(dt).double() - ref).norm()
    assert (dv - ref).norm() <= 1.5 * own
    h, mag = 2.0 ** -11, torch.zeros_like(ref)
    for i in range(0, Sk, 1 << 16):
        t = q[0, 0].double() @ k[0, 0, i:i + (1 << 16)].double().T * D ** -0.5
        mag[i:i + (1 << 16)] = torch.exp(t - lse[0, 0].double()[:, None]).T @ dout[0, 0].double().abs()
    assert ((dv - ref).abs() <= (h + 2.0 ** -12) * mag + h * ref.abs() + 2.0 ** -25).all()
