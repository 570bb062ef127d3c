"""GPU tests of the heads' norm and rotation and of their gradient, against the fp64
oracle (oracle/rope.py).

Tolerances.  A result is rounded once to its type, by at most half a step, eps/2 of
its value (fp16 below its normal range: 2^-25).  Before that it is computed in fp32:
a row's sum over D channels is off by at most D·2^-24 of the sum of its terms'
magnitudes, a handful of products by 2^-24 each (16 allowed), and an angle by 2^-21.
So with M the magnitude that an element's formula goes over,
|err| <= eps/2·|ref| + ((D + 16)·2^-24 + 2^-21)·M + tiny.  A weight's gradient is a
sum of N terms in fp32, whose chain of additions is at most N long: N·2^-24 of the
terms' magnitudes more.
"""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, rope
from oracle import attention_bwd, attention_fwd
from oracle import rope as oracle

pytestmark = pytest.mark.gpu

SENTINEL, GUARD = 7.0, 4096


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 1e-37


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), SENTINEL, dtype=dtype, device="cuda:0")
    return buf, buf[:n].view(shape)


def close(got, ref, mag, dt, D, chain=0, what=""):
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bound = half_step(dt) * np.abs(ref) + ((D + 16 + chain) * 2.0 ** -24 + 2.0 ** -21) * mag + tiny(dt)
    worst = float((np.abs(got - ref) / bound).max())
    assert worst <= 1.0, (what, worst)


def plan_of(pairs, axes, interleaved):
    freq = [3.0 * 0.7 ** i for i in range(pairs)]
    axis = [(i * 5) % axes for i in range(pairs)]
    return rope.Rope(torch.tensor(freq, dtype=torch.float64), torch.tensor(axis, dtype=torch.uint8), interleaved)


def problem(B, S, heads, D, pairs, axes, dt, weight, seed):
    """A packed projection's views, weights, positions and the upstream gradients."""
    g = torch.Generator().manual_seed(seed)
    packed = torch.randn(B, S, sum(heads) * D, generator=g).mul(1.5).to(dt).cuda()
    xs = packed.view(B, S, sum(heads), D).split(heads, dim=2)
    wt = {"same": dt, "fp32": torch.float32}.get(weight)
    ws = [None if wt is None or i == 2 else torch.randn(D, generator=g).add(1.0).to(wt).cuda() for i in range(len(heads))]
    pos = torch.randint(-500, 500, (B, S, axes), generator=g, dtype=torch.int32).cuda()
    dys = [torch.randn(B, h, S, D, generator=g).to(dt).cuda() for h in heads]
    return packed, xs, ws, pos, dys


def refs(xs, ws, pos, plan, turn, dys=None, eps=1e-6):
    out = []
    for i, x in enumerate(xs):
        kw = {}
        if turn[i]:
            kw = dict(positions=pos.cpu().numpy(), inv_freq=plan.inv_freq.numpy(), axis=plan.axis.numpy(),
                      interleaved=plan.interleaved)
        w = None if ws[i] is None else ws[i].double().cpu().numpy()
        x64 = x.double().cpu().numpy()
        if dys is None:
            y = oracle.rope_fwd(x64, w, eps=eps, **kw)
            kw0 = {k: v for k, v in kw.items() if k != "inv_freq"}
            z = np.abs(oracle.rope_fwd(x64, w, eps=eps))
            mag = z.copy()
            if kw:
                n = len(kw["inv_freq"])
                for p in range(n):
                    u, v = (2 * p, 2 * p + 1) if kw0["interleaved"] else (p, p + n)
                    mag[..., u] = mag[..., v] = z[..., u] + z[..., v]
            out.append((y, mag))
        else:
            out.append(oracle.rope_bwd(dys[i].double().cpu().numpy(), x64, w, eps=eps, **kw))
    return out


SHAPES = [  # B, S, heads, D, pairs, axes
    (2, 37, (4, 2, 2), 64, 32, 1), (1, 5, (3, 1, 1), 72, 36, 3), (2, 9, (5, 5, 5), 80, 40, 2), (1, 1, (2, 1, 1), 8, 4, 1),
    (3, 3, (1, 1, 1), 128, 64, 1), (2, 19, (8, 2, 2), 128, 16, 2), (1, 11, (2, 2, 2), 200, 100, 1),
    (1, 13, (2, 1, 1), 256, 128, 3), (1, 7, (3, 3, 3), 72, 18, 1), (2, 4, (2, 2, 2), 256, 1, 1), (1, 6, (2, 1, 1), 128, 0, 1),
    (1, 300, (7, 1, 1), 96, 17, 2), (1, 3, (2, 2, 2), 256, 126, 2), (1, 2, (40, 8, 8), 176, 88, 1),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("dt,weight", [(torch.bfloat16, "same"), (torch.float16, "fp32"), (torch.bfloat16, None)],
                         ids=["bf16", "fp16w32", "noweight"])
def test_forward_and_gradient(cuda_device, shape, interleaved, dt, weight):
    B, S, heads, D, pairs, axes = shape
    plan = plan_of(pairs, axes, interleaved)
    packed, xs, ws, pos, dys = problem(B, S, heads, D, pairs, axes, dt, weight, seed=D + S + pairs)
    turn = (True, True, False)
    bufs = [guarded((B, h, S, D), dt) for h in heads]
    rope.rope_fwd(xs, plan, pos, ws, 1e-6, turn, ys=[b[1] for b in bufs])
    dbuf, dpacked = guarded(packed.shape, dt)
    dxs = dpacked.view(B, S, sum(heads), D).split(heads, dim=2)
    dwbufs = [None if w is None else guarded((D,), w.dtype) for w in ws]
    _, dws = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn, dxs=dxs, dweights=[b and b[1] for b in dwbufs])
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    for buf, t in bufs + [(dbuf, dpacked)] + [b for b in dwbufs if b]:
        assert (buf[t.numel():] == SENTINEL).all(), "written past the end"
    for i, (y, mag) in enumerate(refs(xs, ws, pos, plan, turn)):
        close(bufs[i][1], y, mag, dt, D, what=f"y{i}")
        if ws[i] is None and not turn[i]:
            assert torch.equal(bufs[i][1], xs[i].transpose(1, 2)), "a part that is only laid out is copied"
    for i, (dx, dw, dx_mag, dw_mag) in enumerate(refs(xs, ws, pos, plan, turn, dys)):
        close(dxs[i], dx, dx_mag, dt, D, what=f"dx{i}")
        if dw is not None:
            close(dws[i], dw, dw_mag, ws[i].dtype, D, chain=B * S * heads[i] + 64, what=f"dw{i}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(cuda_device, interleaved):
    """Angles at the ends of int32, against arithmetic of 60 digits."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    D, at = 64, [2 ** 31 - 1, -2 ** 31, 1234567891, -7, 0, 2 ** 24 + 1]
    plan = rope.rope_plan(D, interleaved=interleaved)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, len(at), 2, D, generator=g).to(torch.float16).cuda()
    pos = torch.tensor([at], dtype=torch.int32).cuda()
    y = rope.rope_fwd((x,), plan, pos)[0].double().cpu().numpy()
    z = x.double().cpu().numpy()
    for s, p in enumerate(at):
        for i, f in enumerate(plan.inv_freq.tolist()):
            a = float((Decimal(p) * Decimal(f)) % two_pi)
            u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + D // 2)
            r0 = z[0, s, :, u] * np.cos(a) - z[0, s, :, v] * np.sin(a)
            r1 = z[0, s, :, u] * np.sin(a) + z[0, s, :, v] * np.cos(a)
            slack = (abs(p) * f * 2.0 ** -52 + 2.0 ** -21 + 4 * 2.0 ** -24) * (np.abs(z[0, s, :, u]) + np.abs(z[0, s, :, v]))
            for got, ref in ((y[0, :, s, u], r0), (y[0, :, s, v], r1)):
                assert (np.abs(got - ref) <= 2.0 ** -11 * np.abs(ref) + slack + 2.0 ** -25).all(), (p, i)


def test_shared_positions_and_layouts(cuda_device):
    """Positions [S], [B, 1] and permuted; x already [B, H, S, D], or with rows apart; the same values as from copies."""
    B, S, H, D = 3, 21, 4, 64
    g = torch.Generator().manual_seed(6)
    x = torch.randn(B, S, H, D, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(D, generator=g).to(torch.bfloat16).cuda()
    plan = rope.rope_plan(D)
    one = torch.arange(S, dtype=torch.int32).cuda()[None] + 100
    want = rope.rope_fwd((x,), plan, one.expand(B, S).contiguous(), (w,))[0]
    assert torch.equal(rope.rope_fwd((x,), plan, one, (w,))[0], want)
    assert torch.equal(rope.rope_fwd((x,), plan, one.expand(B, S), (w,))[0], want)
    wide = torch.zeros(S, 3, dtype=torch.int32).cuda()
    wide[:, 1] = one[0]
    assert torch.equal(rope.rope_fwd((x,), plan, wide[:, 1][None], (w,))[0], want)
    heads_first = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(rope.rope_fwd((heads_first,), plan, one, (w,))[0], want)
    apart = torch.full((B, S, H, D + 24), SENTINEL, dtype=x.dtype, device="cuda")
    apart[..., :D] = x
    assert torch.equal(rope.rope_fwd((apart[..., :D],), plan, one, (w,))[0], want)
    at = torch.tensor([[5], [9], [2]], dtype=torch.int32).cuda()
    assert torch.equal(rope.rope_fwd((x,), plan, at, (w,))[0], rope.rope_fwd((x,), plan, at.expand(B, S).contiguous(), (w,))[0])
    dy = torch.randn(B, H, S, D, generator=g).to(torch.bfloat16).cuda()
    dx, dw = rope.rope_bwd((dy,), (x,), plan, one, (w,))
    into = torch.full((B, S, H, D + 24), SENTINEL, dtype=x.dtype, device="cuda")
    dx2, dw2 = rope.rope_bwd((dy,), (heads_first,), plan, one, (w,), dxs=(into[..., :D],))
    assert torch.equal(dx[0], dx2[0]) and torch.equal(dw[0], dw2[0])
    assert (into[..., D:] == SENTINEL).all()


def test_norm_without_rotation_and_four_parts(cuda_device):
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(2, 10, h, 72, generator=g).to(torch.float16).cuda() for h in (1, 2, 3, 4)]
    ws = [torch.randn(72, generator=g).cuda() if i % 2 == 0 else None for i in range(4)]
    ys = rope.rope_fwd(xs, None, None, ws)
    for i in range(4):
        w = None if ws[i] is None else ws[i].double().cpu().numpy()
        ref = oracle.rope_fwd(xs[i].double().cpu().numpy(), w)
        close(ys[i], ref, np.abs(ref), torch.float16, 72, what=str(i))


def test_gradients_of_four_weights(cuda_device):
    """More weights than one launch adds up."""
    B, S, heads, D, dt = 2, 33, (1, 2, 3, 4), 64, torch.bfloat16
    g = torch.Generator().manual_seed(81)
    xs = [torch.randn(B, S, h, D, generator=g).to(dt).cuda() for h in heads]
    ws = [torch.randn(D, generator=g).add(1).cuda() for _ in heads]
    dys = [torch.randn(B, h, S, D, generator=g).to(dt).cuda() for h in heads]
    plan, pos = plan_of(32, 2, False), torch.randint(-99, 99, (B, S, 2), generator=g, dtype=torch.int32).cuda()
    turn = (True, False, True, True)
    space = rope.rope_bwd_workspace(xs, ws)
    room = torch.full((space + 64,), 0x55, dtype=torch.uint8, device="cuda")
    dxs, dws = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn, workspace=room[:space])
    torch.cuda.synchronize()
    assert (room[space:] == 0x55).all()
    for i, (dx, dw, dx_mag, dw_mag) in enumerate(refs(xs, ws, pos, plan, turn, dys)):
        close(dxs[i], dx, dx_mag, dt, D, what=f"dx{i}")
        close(dws[i], dw, dw_mag, torch.float32, D, chain=B * S * heads[i] + 64, what=f"dw{i}")
    with pytest.raises(binding.AttnError):
        rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn, workspace=room[:1024])


def test_many_tokens_of_few_heads(cuda_device):
    """More units than warps, rows that fill a fraction of one, a batch whose sequences end inside a warp's share."""
    B, S, H, D, dt = 7, 3001, 1, 64, torch.float16
    g = torch.Generator().manual_seed(82)
    x = torch.randn(B, S, H, D, generator=g).to(dt).cuda()
    w = torch.randn(D, generator=g).add(1).cuda()
    plan, pos = rope.rope_plan(D), torch.arange(S, dtype=torch.int32).cuda()[None]
    y = rope.rope_fwd((x,), plan, pos, (w,))[0]
    dy = torch.randn(B, H, S, D, generator=g).to(dt).cuda()
    dx, dw = rope.rope_bwd((dy,), (x,), plan, pos, (w,))
    full = pos.expand(B, S)[..., None]
    r = refs((x,), (w,), full, plan, (True,))[0]
    close(y, r[0], r[1], dt, D, what="y")
    rx, rw, mx, mw = refs((x,), (w,), full, plan, (True,), (dy,))[0]
    close(dx[0], rx, mx, dt, D, what="dx")
    # a lane adds up every so many-th token: at most B·S / 152 / 4 in a chain, then CTAs and warps
    close(dw[0], rw, mw, torch.float32, D, chain=B * S // 600 + 700, what="dw")


def test_gradients_that_overlap(cuda_device):
    """Two launches a call, the second set up while the first ends: on two streams at once, again and again, each
    input written just before and each result read just after."""
    cases = []
    for seed, (D, dt) in enumerate(((64, torch.bfloat16), (128, torch.float16))):
        plan = plan_of(D // 2, 1, False)
        _, xs, ws, pos, dys = problem(2, 301, (4, 2, 2), D, D // 2, 1, dt, "same", 90 + seed)
        cases.append((xs, ws, pos, dys, plan, rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, (True, True, False))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(8):
        got = []
        for (xs, ws, pos, dys, plan, _), st in zip(cases, streams):
            with torch.cuda.stream(st):
                fresh = [d.clone() for d in dys]
                dxs, dws = rope.rope_bwd(fresh, xs, plan, pos, ws, 1e-6, (True, True, False))
                got.append([x.clone() for x in (*dxs, *dws[:2])])
                for x in (*fresh, *dxs, *dws[:2]):
                    x.zero_()
    torch.cuda.synchronize()
    for (*_, (dxs, dws)), g in zip(cases, got):
        assert all(torch.equal(a, b) for a, b in zip((*dxs, *dws[:2]), g))


def test_second_derivatives_are_refused(cuda_device):
    x = torch.randn(1, 4, 2, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    y = rope.norm_rope((x,), rope.rope_plan(64), pos)[0]
    (dx,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.float().sum(), x)


def test_no_finite_rows_stay_by_themselves(cuda_device):
    """Rows with NaN or infinities, and rows of zeros, leave every other row as it is."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(1, 24, 4, 128, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(128, generator=g).to(torch.bfloat16).cuda()
    plan, pos = rope.rope_plan(128), torch.arange(24, dtype=torch.int32).cuda()[None]
    clean = rope.rope_fwd((x,), plan, pos, (w,))[0]
    y = x.clone()
    y[0, 3, 1, 5], y[0, 7, 0, 0], y[0, 8, 2] = float("nan"), float("inf"), 0.0
    got = rope.rope_fwd((y,), plan, pos, (w,))[0]
    assert got[0, 1, 3].isnan().all() and got[0, 0, 7].isnan().any() and (got[0, 2, 8] == 0).all()
    for h, s in ((1, 3), (0, 7), (2, 8)):
        got[0, h, s] = clean[0, h, s]
    assert torch.equal(got, clean)


def test_streams_graphs_and_repeats(cuda_device):
    """On a side stream, captured and replayed with other inputs, and twice: the same bits."""
    B, S, heads, D = 2, 65, (4, 2, 2), 128
    plan = rope.rope_plan((32, 48, 48))
    packed, xs, ws, pos, dys = problem(B, S, heads, D, 64, 3, torch.bfloat16, "fp32", 11)
    turn = (True, True, False)
    want = rope.rope_fwd(xs, plan, pos, ws, 1e-6, turn)
    wdx, wdw = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = rope.rope_fwd(xs, plan, pos, ws, 1e-6, turn, stream=side)
    gdx, gdw = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn, stream=side)
    side.synchronize()
    same = lambda a, b: all((u is None and v is None) or torch.equal(u, v) for u, v in zip(a, b))  # noqa: E731
    assert same(got, want) and same(gdx, wdx) and same(gdw, wdw)
    keep = packed.clone()
    packed.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rope.rope_fwd(xs, plan, pos, ws, 1e-6, turn)
        gdx, gdw = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn)
    packed.copy_(keep)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(got, want) and same(gdx, wdx) and same(gdw, wdw)


def test_autograd_and_rotary_attention(cuda_device):
    """norm_rope's gradients are rope_bwd's; rotary_attention is its parts, forward and backward, and near the oracle."""
    B, S, H, D = 2, 150, 3, 64
    g = torch.Generator().manual_seed(12)
    q, k, v = (torch.randn(B, S, H, D, generator=g).to(torch.bfloat16).cuda().requires_grad_() for _ in "qkv")
    wq, wk = (torch.randn(D, generator=g).mul(0.2).add(1).cuda().requires_grad_() for _ in "qk")
    plan, pos = rope.rope_plan((16, 24, 24)), torch.randint(0, 50, (B, S, 3), generator=g, dtype=torch.int32).cuda()
    dout = torch.randn(B, H, S, D, generator=g).to(torch.bfloat16).cuda()
    out = rope.rotary_attention(q, k, v, plan, pos, wq, wk, causal=True)
    got = torch.autograd.grad(out, (q, k, v, wq, wk), dout)
    qh, kh, vh = rope.norm_rope((q, k, v), plan, pos, (wq, wk, None), turn=(True, True, False))
    out2 = binding.attention(qh, kh, vh, causal=True)
    want = torch.autograd.grad(out2, (q, k, v, wq, wk), dout)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(got, want))
    # the oracle from the same rounded heads on; and the whole chain's gradient, relative
    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    ro, _ = attention_fwd(n(qh), n(kh), n(vh), D ** -0.5, True)
    assert np.abs(n(out) - ro).max() <= 2e-2
    dq, dk, dv = attention_bwd(n(qh), n(kh), n(vh), n(dout), D ** -0.5, True)
    kw = dict(positions=pos.cpu().numpy(), inv_freq=plan.inv_freq.numpy(), axis=plan.axis.numpy(), interleaved=False)
    # each gradient is rounded to bf16 twice (attention's, then this one), attention's own error is at most 2^-7
    # of its size relative (its tests), and the heads' Jacobian is at most as large as its terms
    for a, (gh, x, w, kk) in zip((0, 1, 2), ((dq, q, wq, kw), (dk, k, wk, kw), (dv, v, None, {}))):
        dx, dw = oracle.rope_bwd(gh, n(x), None if w is None else n(w), **kk)[:2]
        assert np.linalg.norm(n(got[a]) - dx) <= 2 ** -6 * np.linalg.norm(dx)
        if w is not None:
            assert np.linalg.norm(n(got[3 + a]) - dw) <= 2 ** -5 * np.linalg.norm(dw)


def test_packed_gradient_into_a_frozen_norm(cuda_device):
    """dweight left out where it is not wanted: dx is the same."""
    B, S, H, D = 1, 33, 2, 64
    g = torch.Generator().manual_seed(13)
    x = torch.randn(B, S, H, D, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(D, generator=g).cuda()
    dy = torch.randn(B, H, S, D, generator=g).to(torch.bfloat16).cuda()
    plan, pos = rope.rope_plan(D), torch.arange(S, dtype=torch.int32).cuda()[None]
    want = rope.rope_bwd((dy,), (x,), plan, pos, (w,))[0][0]
    lib, dx = rope._library(), torch.empty_like(x)
    part = rope._pack_part(x.data_ptr(), *x.stride()[:3], H, w.data_ptr(), 1, 1, dy.data_ptr(), dx.data_ptr(),
                           *dx.stride()[:3], 0)
    r, at = rope._rope(plan, pos, B, S, 0)
    assert lib.attn_rope_bwd(part, 1, r, at, B, S, D, 1e-6, 0, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx, want)


@pytest.mark.parametrize("order", ["bsphd", "sbphd", "bshpd", "sbhpd", "bphsd", "hbspd"])
def test_packed_gradients_of_any_order(cuda_device, order):
    """q, k and v of one packed projection whose dimensions (p: which of the three) lie in any order, forward and back:
    the same bits as from and into tensors of their own."""
    B, S, H, D, dt = 3, 7, 4, 72, torch.bfloat16
    size = dict(b=B, s=S, h=H, d=D, p=3)
    g = torch.Generator().manual_seed(14)
    packed = torch.randn(*(size[c] for c in order), generator=g).to(dt).cuda()
    into = torch.full_like(packed, SENTINEL)
    parts = lambda t: t.permute(*(order.index(c) for c in "pbshd")).unbind(0)  # noqa: E731
    plan, pos = plan_of(36, 2, True), torch.randint(-99, 99, (B, S, 2), generator=g, dtype=torch.int32).cuda()
    ws = [torch.randn(D, generator=g).add(1).cuda() for _ in "qk"] + [None]
    dys = [torch.randn(B, H, S, D, generator=g).to(dt).cuda() for _ in "qkv"]
    turn, own = (True, True, False), [x.contiguous() for x in parts(packed)]
    want = rope.rope_fwd(own, plan, pos, ws, 1e-6, turn)
    assert all(torch.equal(a, b) for a, b in zip(rope.rope_fwd(parts(packed), plan, pos, ws, 1e-6, turn), want))
    wdx, wdw = rope.rope_bwd(dys, own, plan, pos, ws, 1e-6, turn)
    _, dw = rope.rope_bwd(dys, parts(packed), plan, pos, ws, 1e-6, turn, dxs=parts(into))
    assert all(torch.equal(a, b) for a, b in zip(parts(into), wdx))
    assert all(torch.equal(a, b) for a, b in zip(dw[:2], wdw[:2]))
    assert binding.device_status() == binding.ATTN_OK


def test_a_plan_changed_before_the_backward_pass_is_refused(cuda_device):
    """As torch refuses any saved tensor that was changed in place; a plan left alone serves any number of calls."""
    x = torch.randn(1, 4, 2, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for call in (lambda p: rope.norm_rope((x,), p, pos)[0], lambda p: rope.rotary_attention(x, x, x, p, pos)):
        for plan in (rope.rope_plan(64), rope.Rope(rope.rope_plan(64).inv_freq, None, True)):
            a, b = (torch.autograd.grad(call(plan), x, torch.ones(1, 2, 4, 64, device="cuda").to(x.dtype))[0] for _ in "ab")
            assert torch.equal(a, b)
            y = call(plan)
            plan.inv_freq.mul_(2.0)
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward(torch.ones_like(y))


@pytest.mark.parametrize("D,pairs", [(256, 127), (200, 33), (64, 31)])
def test_odd_numbers_of_pairs_in_four_parts(cuda_device, D, pairs):
    """One pair a vector and the most parts of a call, two of them with weights: the most a CTA keeps."""
    B, S, heads, dt = 2, 19, (3, 2, 1, 5), torch.float16
    g = torch.Generator().manual_seed(D)
    xs = [torch.randn(B, S, h, D, generator=g).to(dt).cuda() for h in heads]
    ws = [torch.randn(D, generator=g).add(1).cuda() if i % 2 == 0 else None for i in range(4)]
    dys = [torch.randn(B, h, S, D, generator=g).to(dt).cuda() for h in heads]
    plan, pos = plan_of(pairs, 3, False), torch.randint(-99, 99, (B, S, 3), generator=g, dtype=torch.int32).cuda()
    turn = (True, True, False, True)
    ys = rope.rope_fwd(xs, plan, pos, ws, 1e-6, turn)
    dxs, dws = rope.rope_bwd(dys, xs, plan, pos, ws, 1e-6, turn)
    for i, (y, mag) in enumerate(refs(xs, ws, pos, plan, turn)):
        close(ys[i], y, mag, dt, D, what=f"y{i}")
    for i, (dx, dw, dx_mag, dw_mag) in enumerate(refs(xs, ws, pos, plan, turn, dys)):
        close(dxs[i], dx, dx_mag, dt, D, what=f"dx{i}")
        if dw is not None:
            close(dws[i], dw, dw_mag, torch.float32, D, chain=B * S * heads[i] + 64, what=f"dw{i}")
