"""GPU tests of cross-attention and its gradient against the fp64 oracle (oracle/cross.py).

Tolerances, with h = eps/2 of the 16-bit type (half a step) and M the sum of the
magnitudes that an element adds up.  The weights P are rounded to the type before
their product with V (h·M) and the normaliser allows for that of each tile's largest
only (another h·M); scores are fp32 sums of D products, whose error, with the
exponential's, moves a weight by at most 2^-13 of itself for the sizes used here
(|scale·q·k| summed over the channels below 2^10, times 2^-24); the result is rounded
once (h·|ref|).  fp16 weights below 2^-14 lose at most 2^-25 each.  So
    out   (2h + 2^-13)·M + h·|ref|,  M = Σ P|v|
    dq    h·M1 + 2^-12·M2 + h·|ref|, M1 = scale·Σ|dS||k|, M2 the same of P(|dout||v| + |delta|),
          of which dS, rounded to the type, is the difference; dk likewise
    dv    (h + 2^-12)·M + h·|ref|,   M = Σ P|dout|
and in fp16 2^-25 of the plain sum of the other factor's magnitudes more.
"""
import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cross, rope
from oracle import cross as oracle

pytestmark = pytest.mark.gpu

SENTINEL, GUARD = 7.0, 4096
NAN, INF = float("nan"), float("inf")


def half_step(dt):
    return torch.finfo(dt).eps / 2


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), SENTINEL, dtype=dtype, device="cuda:0")
    return buf, buf[:n].view(shape)


def untouched(*pairs):
    return all((buf[t.numel():] == SENTINEL).all() for buf, t in pairs)


def n64(t):
    return t.detach().double().cpu().numpy()


def problem(B, Hq, Hkv, Sq, Sk, D, lens, dt, seed, poison=True):
    """Inputs on the GPU; behind a sequence's end k and v hold NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, Sq, D, generator=g).mul(1.5).to(dt)
    k, v = (torch.randn(B, Hkv, Sk, D, generator=g).to(dt) for _ in "kv")
    dout = torch.randn(B, Hq, Sq, D, generator=g).to(dt)
    if lens is not None and poison:
        for b, n in enumerate(lens):
            k[b, :, n:], v[b, :, n:] = NAN, -INF
            v[b, :, n::2] = NAN
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    return q.cuda(), k.cuda(), v.cuda(), dout.cuda(), ln


def check(what, got, ref, bound):
    got = n64(got)
    assert np.isfinite(got).all(), what
    worst = float((np.abs(got - ref) / (bound + 1e-30)).max())
    assert worst <= 1.0, (what, worst)


def check_fwd(q, k, v, lens, out, lse, scale):
    dt, h = q.dtype, half_step(q.dtype)
    B, Hq, _, _ = q.shape
    G, full = Hq // k.shape[1], lens if lens is not None else [k.shape[2]] * B
    kk, vv = (np.nan_to_num(n64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (k, v))
    ro, rl = oracle.cross_fwd(n64(q), kk, vv, full, scale)
    mag = oracle.cross_fwd(n64(q), kk, np.abs(vv), full, scale)[0]
    bound = (2 * h + 2.0 ** -13) * mag + h * np.abs(ro)
    if dt == torch.float16:
        for b in range(B):
            for i in range(Hq):
                bound[b, i] += 2.0 ** -25 * (1 + np.abs(vv[b, i // G, :full[b]]).sum(0))
    check("out", out, ro, bound)
    got = n64(lse)
    dead = np.isneginf(rl)
    assert np.array_equal(dead, np.isneginf(got)) and (n64(out)[dead] == 0).all()
    assert (np.abs(got[~dead] - rl[~dead]) <= 2.0 ** -13 + np.abs(rl[~dead]) * 2.0 ** -22).all()
    return ro, rl


def check_bwd(q, k, v, out, lse, dout, lens, scale, grads):
    dt, h = q.dtype, half_step(q.dtype)
    B, Hq = q.shape[:2]
    G, full = Hq // k.shape[1], lens if lens is not None else [k.shape[2]] * B
    kk, vv = (np.nan_to_num(n64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (k, v))
    dq, dk, dv, delta, (mq, mk, mv, m2q, m2k) = oracle.cross_bwd(n64(q), kk, vv, n64(out), n64(lse), n64(dout), full, scale)
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    sq, sk, sv = np.zeros_like(dq), np.zeros_like(dk), np.zeros_like(dv)
    for b in range(B):
        for i in range(Hq):
            sq[b, i] = scale * np.abs(kk[b, i // G, :full[b]]).sum(0) + 1
            sk[b, i // G] += scale * np.abs(n64(q)[b, i]).sum(0) + 1
            sv[b, i // G] += np.abs(n64(dout)[b, i]).sum(0) + 1
    check("dq", grads[0], dq, h * mq + 2.0 ** -12 * m2q + h * np.abs(dq) + tiny * sq)
    check("dk", grads[1], dk, h * mk + 2.0 ** -12 * m2k + h * np.abs(dk) + tiny * sk)
    check("dv", grads[2], dv, (h + 2.0 ** -12) * mv + h * np.abs(dv) + tiny * sv)
    np.testing.assert_allclose(n64(grads[3]), delta, rtol=0, atol=float(2.0 ** -16 * np.abs(n64(dout) * n64(out)).sum(-1).max() + 1e-30))
    for b in range(B):  # keys that are not there
        assert (grads[1][b, :, full[b]:] == 0).all() and (grads[2][b, :, full[b]:] == 0).all()


def run_both(B, Hq, Hkv, Sq, Sk, D, lens, dt, seed):
    q, k, v, dout, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, dt, seed)
    scale = D ** -0.5
    ob, out = guarded(q.shape, dt)
    lb, lse = guarded(q.shape[:3], torch.float32)
    cross.cross_fwd(q, k, v, ln, out=out, lse=lse)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    assert untouched((ob, out), (lb, lse))
    check_fwd(q, k, v, lens, out, lse, scale)
    bufs = [guarded(s, t) for s, t in ((q.shape, dt), (k.shape, dt), (k.shape, dt), (q.shape[:3], torch.float32))]
    grads = [b[1] for b in bufs]
    cross.cross_bwd(q, k, v, out, lse, dout, ln, dq=grads[0], dk=grads[1], dv=grads[2], delta=grads[3])
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    assert untouched(*bufs)
    check_bwd(q, k, v, out, lse, dout, lens, scale, grads)


SHAPES = [  # B, Hq, Hkv, Sq, Sk, lens
    (1, 1, 1, 1, 1, None),
    (2, 2, 2, 1, 40, [40, 0]),
    (3, 4, 2, 5, 130, [128, 1, 129]),
    (2, 2, 1, 129, 77, [77, 13]),
    (1, 3, 3, 300, 300, None),
    (2, 8, 2, 33, 700, [699, 300]),
    (1, 2, 2, 700, 5, [5]),
    (4, 2, 2, 64, 257, [256, 0, 257, 127]),
    (1, 2, 1, 1, 5000, [4097]),
    (1, 1, 1, 3000, 200, [150]),
]
DIMS = [64, 128, 256, 72, 192, 8, 96, 136, 200]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("D", DIMS[:3])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_against_the_oracle(cuda_device, shape, D, dt):
    B, Hq, Hkv, Sq, Sk, lens = shape
    run_both(B, Hq, Hkv, Sq, Sk, D, lens, dt, seed=Sq + Sk + D)


@pytest.mark.parametrize("D", DIMS[3:])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[3], SHAPES[5], SHAPES[8]], ids=str)
def test_other_head_dimensions(cuda_device, shape, D):
    B, Hq, Hkv, Sq, Sk, lens = shape
    run_both(B, Hq, Hkv, Sq, Sk, D, lens, torch.bfloat16, seed=Sq + Sk + D)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1)])
@pytest.mark.parametrize("D", [64, 128, 80, 256])
def test_few_queries(cuda_device, T, heads, D):
    """A decoder's few tokens: every count of rows around the tiles' sizes, ragged keys, a sequence without any."""
    lens = [900, 0, 1, 511, 64]
    q, k, v, _, ln = problem(5, *heads, T, 900, D, lens, torch.bfloat16, seed=T + D)
    ob, out = guarded(q.shape, q.dtype)
    lb, lse = guarded(q.shape[:3], torch.float32)
    cross.cross_fwd(q, k, v, ln, out=out, lse=lse)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK and untouched((ob, out), (lb, lse))
    check_fwd(q, k, v, lens, out, lse, D ** -0.5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Sq", [1, 20, 200])
def test_scores_that_climb(cuda_device, dt, Sq):
    """Scores that rise along the keys by far more than the softmax's reference may lag, and the same falling; peaked rows."""
    D, Sk = 64, 1500
    q, k, v, _, _ = problem(1, 2, 2, Sq, Sk, D, None, dt, seed=4)
    ramp = torch.linspace(-30, 30, Sk, device="cuda")
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[0, 0, :, 0], k[0, 1, :, 0] = ramp.to(dt), -ramp.to(dt)
    out, lse = cross.cross_fwd(q, k, v)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    check_fwd(q, k, v, None, out, lse, D ** -0.5)


@pytest.mark.parametrize("Sq,Sk,lens", [(1, 1, None), (1, 2, [2, 1]), (3, 7, [7, 0]), (16, 17, [17, 16]), (32, 64, [64, 33]),
                                        (30, 5, None)])
@pytest.mark.parametrize("heads", [(2, 2), (4, 2)])
@pytest.mark.parametrize("D", [64, 72, 128, 200, 256])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_small_gradients_round_once(cuda_device, Sq, Sk, lens, heads, D, dt):
    """A slice of few queries and keys: P and dS enter their products in two terms each, so that besides the fp32 sums
    only the results are rounded."""
    q, k, v, dout, ln = problem(2, *heads, Sq, Sk, D, lens, dt, seed=Sq + Sk + D)
    out, lse = cross.cross_fwd(q, k, v, ln)
    bufs = [guarded(s, t) for s, t in ((q.shape, dt), (k.shape, dt), (k.shape, dt), (q.shape[:3], torch.float32))]
    grads = [b[1] for b in bufs]
    cross.cross_bwd(q, k, v, out, lse, dout, ln, dq=grads[0], dk=grads[1], dv=grads[2], delta=grads[3])
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK and untouched(*bufs)
    assert cross.cross_bwd_workspace(q, k) == 16
    check_bwd(q, k, v, out, lse, dout, lens, D ** -0.5, grads)
    kk, vv = (np.nan_to_num(n64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (k, v))
    full = lens if lens is not None else [Sk] * 2
    dq, dk, dv, _, (mq, mk, mv, m2q, m2k) = oracle.cross_bwd(n64(q), kk, vv, n64(out), n64(lse), n64(dout), full, D ** -0.5)
    h = half_step(dt)
    tiny = 2.0 ** -24 * (1 + float(np.abs(n64(q)).max() + np.abs(kk).max() + np.abs(n64(dout)).max()) * Sq * heads[0])
    for name, got, ref, m2 in (("dq", grads[0], dq, m2q), ("dk", grads[1], dk, m2k), ("dv", grads[2], dv, mv)):
        check(name, got, ref, h * np.abs(ref) + 2.0 ** -12 * m2 + tiny)


def test_results_do_not_depend_on_the_padding(cuda_device):
    for shape in ((2, 4, 2, 40, 400, [390, 5]), (2, 2, 2, 600, 300, [129, 0]), (1, 2, 2, 3, 900, [700]),
                  (3, 2, 1, 9, 60, [59, 0, 1])):
        for D in (64, 128, 256):
            q, k, v, dout, ln = problem(*shape[:5], D, shape[5], torch.bfloat16, 21)
            k2, v2 = k.nan_to_num(1.0, 2.0, 3.0), v.nan_to_num(4.0, 5.0, -6.0)
            a, b = cross.cross_fwd(q, k, v, ln), cross.cross_fwd(q, k2, v2, ln)
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            ga, gb = (cross.cross_bwd(q, kk, vv, *a, dout, ln) for kk, vv in ((k, v), (k2, v2)))
            assert all(torch.equal(x, y) for x, y in zip(ga, gb))


@pytest.mark.parametrize("Sq,Sk", [(1, 300), (40, 30), (200, 300), (2000, 300)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nobody_has_keys(cuda_device, Sq, Sk, D):
    q, k, v, dout, ln = problem(2, 2, 2, Sq, Sk, D, [0, 0], torch.bfloat16, 23)
    out, lse = cross.cross_fwd(q, k, v, ln)
    grads = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    assert binding.device_status() == binding.ATTN_OK
    assert (out == 0).all() and torch.isneginf(lse).all() and all((g == 0).all() for g in grads)


def test_many_short_sequences(cuda_device):
    """More sequences than SMs by far, most of them without keys: units are found by counting through the lengths."""
    B, Sq, Sk, D = 700, 70, 140, 64
    lens = [(i * 37) % 141 if i % 3 == 0 else 0 for i in range(B)]
    q, k, v, dout, ln = problem(B, 1, 1, Sq, Sk, D, lens, torch.bfloat16, 24)
    out, lse = cross.cross_fwd(q, k, v, ln)
    grads = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    assert binding.device_status() == binding.ATTN_OK
    check_fwd(q, k, v, lens, out, lse, D ** -0.5)
    check_bwd(q, k, v, out, lse, dout, lens, D ** -0.5, grads)


@pytest.mark.parametrize("D", [64, 128])
def test_gradient_of_a_ragged_batch(cuda_device, D):
    """A few units a CTA, of very different lengths: taken longest first; equal lengths, none and one among them."""
    B, H, Sq, Sk = 6, 20, 400, 700
    lens = [1, 700, 0, 700, 333, 129]
    q, k, v, dout, ln = problem(B, H, H, Sq, Sk, D, lens, torch.float16, 26)
    out, lse = cross.cross_fwd(q, k, v, ln)
    grads = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    again = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    assert binding.device_status() == binding.ATTN_OK
    check_bwd(q, k, v, out, lse, dout, lens, D ** -0.5, grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("D,B", [(64, 1500), (128, 700), (256, 300)])
def test_gradients_of_very_many_sequences(cuda_device, D, B):
    """Several rounds of a unit a CTA, sequences of one tile or none; and a wrong length among them is found."""
    lens = [(i * 53) % 101 if i % 4 else 0 for i in range(B)]
    q, k, v, dout, ln = problem(B, 1, 1, 70, 100, D, lens, torch.float16, 27)
    out, lse = cross.cross_fwd(q, k, v, ln)
    grads = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    assert binding.device_status() == binding.ATTN_OK
    check_bwd(q, k, v, out, lse, dout, lens, D ** -0.5, grads)
    for at, wrong, meant in ((B - 2, 101, 100), (B // 2, -3, 0)):
        bad, good = ln.clone(), ln.clone()
        bad[at], good[at] = wrong, meant
        out, lse = cross.cross_fwd(q, k, v, good)
        want = cross.cross_bwd(q, k, v, out, lse, dout, good)
        assert binding.device_status() == binding.ATTN_OK
        got = cross.cross_bwd(q, k, v, out, lse, dout, bad)
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        # in bits: keys that were behind the end, and with them the gradients, hold NaN
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))


def test_shared_inputs_and_repeated_use(cuda_device):
    """k and v one tensor, q among them; a graph of autograd used for two losses."""
    g = torch.Generator().manual_seed(25)
    x = torch.randn(2, 3, 90, 64, generator=g).to(torch.bfloat16).cuda()
    out, lse = cross.cross_fwd(x, x, x)
    check_fwd(x, x, x, None, out, lse, 0.125)
    grads = cross.cross_bwd(x, x, x, out, lse, x)
    check_bwd(x, x, x, out, lse, x, None, 0.125, grads)
    q, k = x.clone().requires_grad_(), x[:, :, :40].contiguous().requires_grad_()
    o = cross.cross_attention(q, k, k)
    a = torch.autograd.grad(o, (q, k), torch.ones_like(o), retain_graph=True)
    b = torch.autograd.grad(o, (q, k), torch.ones_like(o))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_nan_and_infinite_queries_and_keys(cuda_device):
    """A NaN query makes its own row NaN and no other; a key that gives +inf or NaN scores, the rows that meet it."""
    q, k, v, _, ln = problem(2, 2, 2, 150, 300, 64, [300, 200], torch.bfloat16, 22)
    want, _ = cross.cross_fwd(q, k, v, ln)
    q2 = q.clone()
    q2[0, 1, 7, 3] = NAN
    out, lse = cross.cross_fwd(q2, k, v, ln)
    assert out[0, 1, 7].isnan().all() and lse[0, 1, 7].isnan()
    out[0, 1, 7] = want[0, 1, 7]
    assert torch.equal(out, want)
    k2 = k.clone()
    k2[1, 0, 5, 0] = NAN
    out, lse = cross.cross_fwd(q, k2, v, ln)
    assert out[1, 0].isnan().all() and torch.equal(out[0], want[0]) and torch.equal(out[1, 1], want[1, 1])


def test_streams_graphs_and_repeats(cuda_device):
    """On a side stream, captured and replayed on other inputs with one workspace each, and twice: the same bits."""
    for shape in ((2, 4, 2, 1, 900, [800, 33]), (1, 4, 2, 64, 4000, [3333]), (2, 2, 2, 1000, 100, [100, 3])):
        q, k, v, dout, ln = problem(*shape[:5], 128, shape[5], torch.bfloat16, 31)
        want = cross.cross_fwd(q, k, v, ln)
        wantg = cross.cross_bwd(q, k, v, *want, dout, ln)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = cross.cross_fwd(q, k, v, ln, stream=side)
        gotg = cross.cross_bwd(q, k, v, *got, dout, ln, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + gotg, want + wantg))
        keep = q.clone()
        q.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = cross.cross_fwd(q, k, v, ln)
            gotg = cross.cross_bwd(q, k, v, *got, dout, ln)
        q.copy_(keep)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + gotg, want + wantg))
        assert binding.device_status() == binding.ATTN_OK


def test_calls_that_overlap(cuda_device):
    """Two streams at once, each with its own workspace."""
    a = problem(1, 4, 2, 64, 6000, 128, [5000], torch.bfloat16, 41)
    b = problem(2, 4, 4, 3, 3000, 64, [3000, 100], torch.float16, 42)
    want = [cross.cross_fwd(*x[:3], x[4]) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [cross.cross_fwd(*x[:3], x[4], stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_gradients_that_overlap(cuda_device):
    """Calls of several kernels each, which are set up while one another end, on three streams at once and over and
    over on one; inputs that the kernel before wrote, results that the next one reads."""
    shapes = (((4, 12, 12, 300, 600, [600, 1, 0, 333]), 64), ((2, 8, 2, 100, 900, [900, 400]), 128),
              ((1, 2, 2, 700, 400, [399]), 256))
    calls = [problem(*s[:5], D, s[5], torch.bfloat16, 43 + i) for i, (s, D) in enumerate(shapes)]
    fwd = [cross.cross_fwd(*c[:3], c[4]) for c in calls]
    want = [cross.cross_bwd(*c[:3], *f, c[3], c[4]) for c, f in zip(calls, fwd)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(8):
        got = []
        for c, st in zip(calls, streams):
            with torch.cuda.stream(st):
                dout = c[3].clone()
                f = cross.cross_fwd(*c[:3], c[4])
                g = cross.cross_bwd(*c[:3], *f, dout, c[4])
                got.append([x.clone() for x in g])
                for x in (dout, *f, *g):
                    x.zero_()
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_bad_lengths_are_reported(cuda_device):
    q, k, v, dout, _ = problem(3, 2, 2, 20, 100, 64, None, torch.bfloat16, 51)
    for Sq in (20, 1):
        qq, dd = q[:, :, :Sq].contiguous(), dout[:, :, :Sq].contiguous()
        bad, good = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([101, -1, 50], [100, 0, 50]))
        want = cross.cross_fwd(qq, k, v, good)
        wantg = cross.cross_bwd(qq, k, v, *want, dd, good)
        assert binding.device_status() == binding.ATTN_OK
        got = cross.cross_fwd(qq, k, v, bad)
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        gotg = cross.cross_bwd(qq, k, v, *got, dd, bad)
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        assert all(torch.equal(a, b) for a, b in zip(got + gotg, want + wantg))
    assert binding.device_status() == binding.ATTN_OK


def test_waits_that_run_out_are_reported(cuda_device):
    q, k, v, dout, ln = problem(1, 2, 2, 300, 600, 128, [600], torch.bfloat16, 52)
    out, lse = cross.cross_fwd(q, k, v, ln)
    assert binding.device_status() == binding.ATTN_OK
    cross.cross_fwd(q, k, v, ln, wait_timeout_ns=0)
    assert binding.device_status() == binding.ATTN_ERR_TIMEOUT
    cross.cross_bwd(q, k, v, out, lse, dout, ln, wait_timeout_ns=0)
    assert binding.device_status() == binding.ATTN_ERR_TIMEOUT
    again, _ = cross.cross_fwd(q, k, v, ln)
    assert binding.device_status() == binding.ATTN_OK and torch.equal(again, out)


def test_workspace_is_asked_for(cuda_device):
    q, k, v, dout, _ = problem(1, 2, 2, 64, 6000, 128, None, torch.bfloat16, 53)
    out, lse = cross.cross_fwd(q, k, v)
    need, needg = cross.cross_fwd_workspace(q, k), cross.cross_bwd_workspace(q, k)
    assert need > 16 and needg > 16
    for n, call in ((need, lambda w: cross.cross_fwd(q, k, v, workspace=w)),
                    (needg, lambda w: cross.cross_bwd(q, k, v, out, lse, dout, workspace=w))):
        with pytest.raises(binding.AttnError):
            call(torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
        w = torch.full((n + 64,), 0x7f, dtype=torch.uint8, device="cuda")
        call(w[:n])
        torch.cuda.synchronize()
        assert (w[n:] == 0x7f).all()
    with pytest.raises(TypeError):
        cross.cross_fwd(q, k, v, workspace=torch.empty(need, device="cuda"))


def test_autograd_through_a_block(cuda_device):
    """Projections, norm and rotation, self-attention, then cross-attention over a prompt with normed heads: the
    operators run together, and the gradients are those of an fp64 composition."""
    B, S, P, H, D, dt = 2, 200, 70, 2, 64, torch.bfloat16
    g = torch.Generator().manual_seed(61)
    x = [torch.randn(B, S, H, D, generator=g).to(dt).cuda().requires_grad_() for _ in "qkv"]
    c = [torch.randn(B, P, H, D, generator=g).to(dt).cuda().requires_grad_() for _ in "kv"]
    w = [torch.randn(D, generator=g).mul(0.1).add(1).cuda().requires_grad_() for _ in range(3)]
    lens = torch.tensor([70, 41], dtype=torch.int32).cuda()
    plan, pos = rope.rope_plan((24, 40)), torch.randint(0, 60, (B, S, 2), generator=g, dtype=torch.int32).cuda()
    a = rope.rotary_attention(*x, plan, pos, w[0], w[1], causal=False)
    (kc, vc) = rope.norm_rope(c, None, None, (w[2], None))
    out = cross.cross_attention(a, kc, vc, lens)
    dout = torch.randn(out.shape, generator=g).to(dt).cuda()
    got = torch.autograd.grad(out, x + c + w, dout)
    assert binding.device_status() == binding.ATTN_OK

    def ref(x, c, w):
        norm = lambda z, ww: z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * ww  # noqa: E731
        at = pos.double()[:, :, plan.axis.long().cuda()] * plan.inv_freq.cuda()
        cos, sin = at.cos()[:, :, None], at.sin()[:, :, None]
        rot = lambda z: torch.cat([z[..., :32] * cos - z[..., 32:] * sin, z[..., :32] * sin + z[..., 32:] * cos], -1)  # noqa: E731
        q, k, v = rot(norm(x[0], w[0])).transpose(1, 2), rot(norm(x[1], w[1])).transpose(1, 2), x[2].transpose(1, 2)
        a = torch.softmax(q @ k.transpose(2, 3) * D ** -0.5, -1) @ v
        kc, vc = norm(c[0], w[2]).transpose(1, 2), c[1].transpose(1, 2)
        t = (a @ kc.transpose(2, 3) * D ** -0.5).masked_fill(torch.arange(P, device="cuda")[None, None, None] >= lens[:, None, None, None], -INF)
        return torch.softmax(t, -1) @ vc

    leaves = [t.detach().double().requires_grad_() for t in x + c + w]
    want_out = ref(leaves[:3], leaves[3:5], leaves[5:])
    want = torch.autograd.grad(want_out, leaves, dout.double())
    # each of the four stages rounds what it passes on, and the heads it takes in, to bf16 (2^-8 of a value each);
    # relative to the whole, 2^-8 a stage forward and back: 2^-5 in all
    assert (out.double() - want_out).norm() <= 2 ** -6 * want_out.norm()
    for name, u, r in zip("q k v kc vc wq wk wc".split(), got, want):
        assert (u.double() - r).norm() <= 2 ** -5 * r.norm(), name


def test_more_than_four_gigabytes(cuda_device):
    """Keys whose last head lies past 2^32 bytes and 2^31 values, for one query and for its gradient."""
    H, Sk, D = 2, 9_000_001, 128
    g = torch.Generator(device="cuda").manual_seed(71)
    q = torch.randn(1, H, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.empty(1, H, Sk, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for t in (k, v):
        for h in range(H):
            for i in range(0, Sk, 1 << 20):
                part = t[0, h, i:i + (1 << 20)]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    v[0, 1, -1000:] += 40.0  # what lies past the 32-bit offsets decides
    k[0, 1, -1000:] += 0.5 * q[0, 1]
    lens = torch.tensor([Sk - 3], dtype=torch.int32).cuda()
    out, lse = cross.cross_fwd(q, k, v, lens)
    for h in range(H):
        t = torch.cat([(q[0, h].double() @ k[0, h, i:i + (1 << 20)].double().T) for i in range(0, Sk, 1 << 20)], 1)[0] * D ** -0.5
        t[Sk - 3:] = -INF
        z = torch.logsumexp(t, 0)
        p = torch.exp(t - z)
        ref, mag = torch.zeros(D, dtype=torch.double, device="cuda"), torch.zeros(D, dtype=torch.double, device="cuda")
        for i in range(0, Sk, 1 << 20):
            vv = v[0, h, i:i + (1 << 20)].double()
            ref += p[i:i + (1 << 20)] @ vv
            mag += p[i:i + (1 << 20)] @ vv.abs()
        assert abs(float(lse[0, h, 0]) - float(z)) < 1e-3
        # runs of 1e5 keys and more: their fp32 sums add 2^-10 of the magnitude at most
        assert ((out[0, h, 0].double() - ref).abs() <= (2 ** -7 + 2 ** -10) * mag + 2 ** -8 * ref.abs()).all()
    dout = torch.randn(out.shape, generator=g, device="cuda").to(torch.bfloat16)
    dq, dk, dv, delta = cross.cross_bwd(q, k, v, out, lse, dout, lens)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    h, rows = 1, torch.arange(Sk - 1100, Sk, device="cuda")
    p = torch.exp(q[0, h].double() @ k[0, h, rows].double().T * D ** -0.5 - lse[0, h].double()[:, None])[0]
    p[-3:] = 0
    ref = p[:, None] * dout[0, h].double()
    assert ((dv[0, h, rows].double() - ref).abs() <= (2 ** -7 + 2 ** -12) * ref.abs() + 1e-30).all()
    assert (dk[0, h, -3:] == 0).all() and (dv[0, h, -3:] == 0).all() and dk[0, h, -1000:-3].abs().max() > 0
