"""GPU checks of the 8-bit key/value cache against the fp64 oracle (oracle/cache.py)."""
import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cache as kv
from exact_attention_68_gb300.build import build_debug_library
from oracle import cache as oc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def clean_status(cuda_device):
    assert binding.device_status() == binding.ATTN_OK
    yield
    torch.cuda.synchronize()
    binding.device_status()


def pool(pages, heads, D, P, seed, stale=True):
    """An empty pool whose slots hold anything (NaN codes among it)."""
    c = kv.cache_alloc(pages, heads, D, P, device=DEV)
    if stale:
        g = torch.Generator().manual_seed(seed)
        for t in (c.k, c.v):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.exp2(torch.randint(-20, 20, t.shape, generator=g).float()))
    return c


def to_np(c):
    d = {n: getattr(c, n).cpu().numpy().copy() for n in ("k", "v", "k_scale", "v_scale", "k_bounds")}
    return {**d, "head_dim": c.head_dim}


def table_for(lens, P, pages, seed, width=None):
    need = [-(-n // P) for n in lens]
    perm = np.random.default_rng(seed).permutation(pages)
    t = np.full((len(lens), width or max(max(need), 1)), -7, np.int32)  # entries behind the end are not read
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    assert at <= pages
    return t, perm[at:]


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rows(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def same_cache(c, ref):
    """Codes by value (any NaN code is NaN), scales and bounds by bits."""
    val = oc.e4m3_values()
    for n in "kv":
        assert np.array_equal(val[getattr(c, n).cpu().numpy()], val[ref[n]], equal_nan=True), n
        assert np.array_equal(getattr(c, n + "_scale").cpu().numpy(), ref[n + "_scale"]), n + "_scale"
    assert np.array_equal(c.k_bounds.cpu().numpy(), ref["k_bounds"])


def append_both(c, ref, table, lens, fresh, T, dtype, seed, std=1.0):
    H, D = c.k.shape[1], c.head_dim
    k, v = (rows((len(lens), H, T, D), dtype, seed + i, std) for i in range(2))
    kv.cache_append(c, k.to(DEV), v.to(DEV), ints(table), ints(lens), None if fresh is None else ints(fresh))
    f = np.full(len(lens), T) if fresh is None else np.asarray(fresh)
    oc.cache_append(ref, table, np.asarray(lens), f, k.double().numpy(), v.double().numpy())


def filled(lens, H, D, P, dtype, seed, extra=2, width=None):
    """A pool with these sequences appended in one go, its oracle copy, the table and free pages."""
    pages = sum(-(-n // P) for n in lens) + extra
    c = pool(pages, H, D, P, seed)
    ref = to_np(c)
    table, free = table_for(lens, P, pages, seed, width)
    T = max(max(lens), 1)
    append_both(c, ref, table, lens, lens, T, dtype, seed + 10)
    return c, ref, table, free


# |out - ref| and |lse - ref|: q and the codes reach the tensor cores exactly and
# S sums D products in fp32, each step at most 2^-23 of the products' magnitude
# (the unit may truncate), the two scale factors and t itself are rounded:
# dt = (D + 16)·2^-23·absqk in ln units.  A weight is off by 2·dt relative (its
# own and the sum's), P is rounded to fp16 (2^-11, and 2^-38 of the largest term
# where it is subnormal), ex2 and the fp32 sums of out add 2^-18.  The output's
# rounding is half a step of its type.
def check_fwd(out, lse, ref_out, ref_lse, absv, absqk, D, dtype, fresh):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    half = torch.finfo(dtype).eps / 2
    dt = (D + 16) * 2.0 ** -23 * absqk
    worst = 0.0
    for b, n in enumerate(fresh):
        o, r, a, d = out[b, :, :n], ref_out[b, :, :n], absv[b, :, :n], dt[b, :, :n, None]
        top = np.abs(r).max(initial=0.0) + a.max(initial=0.0)
        tol = half * np.abs(r) + (2.0 ** -11 + 2 * d + 2.0 ** -18) * (1 + half) * a + 2.0 ** -36 * top + 2.0 ** -25
        assert np.isfinite(o).all()
        if o.size:
            worst = max(worst, float((np.abs(o - r) / tol).max()))
        z, w = lse[b, :, :n], ref_lse[b, :, :n]
        assert np.array_equal(np.isneginf(z), np.isneginf(w))
        live = ~np.isneginf(w)
        z, w = z[live], w[live]
        assert (np.abs(z - w) <= dt[b, :, :n][live] + 2.0 ** -20 + 2.0 ** -22 * np.abs(w)).all()
    assert worst <= 1.0, worst


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("D,P,H,dtype", [(128, 64, 2, BF), (64, 16, 3, FP), (72, 32, 1, BF), (256, 64, 1, FP),
                                         (8, 16, 2, BF), (200, 32, 2, FP), (136, 64, 5, BF)])
def test_append_writes_the_oracles_pages(D, P, H, dtype):
    lens0 = [P + 3, 1, 2 * P, P - 1, 0]
    pages = 24
    c = pool(pages, H, D, P, 1)
    ref = to_np(c)
    table, _ = table_for([4 * P] * 5, P, pages, 2)
    append_both(c, ref, table, lens0, lens0, max(lens0), dtype, 3)
    same_cache(c, ref)
    lens = np.array(lens0)
    # single tokens, larger ones (scales grow), smaller ones, several; some sequences idle
    for step, (T, std, fresh) in enumerate([(1, 1.0, None), (1, 40.0, None), (1, 0.01, None), (5, 3.0, [5, 0, 2, 1, 3]),
                                            (P + 2, 500.0, [P + 2, 1, 0, P, 4])]):
        f = np.full(5, T) if fresh is None else np.array(fresh)
        lens = lens + f
        append_both(c, ref, table, lens, fresh, T, dtype, 20 + 2 * step, std)
        same_cache(c, ref)
    assert binding.device_status() == binding.ATTN_OK


def test_append_of_infinities_nans_zeros_and_extremes():
    P, D = 16, 64
    c = pool(4, 1, D, P, 5)
    ref = to_np(c)
    table = np.array([[2, 0]], np.int32)
    k, v = (rows((1, 1, 20, D), BF, s) for s in (6, 7))
    k[0, 0, 3, 5], k[0, 0, 4, 6], k[0, 0, 5, 7] = np.inf, -np.inf, np.nan
    k[0, 0, :16, 9] = np.nan  # a channel of nothing else
    v[0, 0, :16] = 0.0
    v[0, 0, 16:, 0], v[0, 0, 16:, 1] = 3e38, 1e-30
    for n in (13, 20):
        f = 13 if n == 13 else 7
        a, b = (x[:, :, n - f:n].contiguous() for x in (k, v))
        kv.cache_append(c, a.to(DEV), b.to(DEV), ints(table), ints([n]))
        oc.cache_append(ref, table, np.array([n]), np.array([f]), a.double().numpy(), b.double().numpy())
        same_cache(c, ref)


# ---------------------------------------------------------------- attention
FWD = [  # D, P, Hq, H, T, dtype, lens
    (128, 64, 8, 2, 1, BF, [1, 63, 64, 65, 1000]),
    (128, 64, 4, 4, 1, FP, [300, 17]),
    (64, 16, 12, 4, 3, FP, [3, 16, 33, 200]),
    (72, 32, 5, 1, 2, BF, [2, 129, 700]),
    (256, 64, 4, 2, 1, BF, [5, 321]),
    (136, 16, 6, 2, 4, FP, [4, 100]),
    (200, 32, 1, 1, 1, BF, [1]),
    (8, 16, 2, 1, 1, FP, [40]),
    (96, 64, 32, 2, 5, BF, [640, 77]),      # five row tiles
    (128, 32, 20, 1, 64, FP, [64, 150]),    # the most tokens, 80 row tiles
    (128, 64, 2, 1, 1, BF, [9000]),         # one segment over many workers
]


@pytest.mark.parametrize("D,P,Hq,H,T,dtype,lens", FWD)
def test_fwd_meets_the_oracle(D, P, Hq, H, T, dtype, lens):
    c, ref, table, _ = filled(lens, H, D, P, dtype, 31, width=-(-max(lens) // P) + 3)
    q = rows((len(lens), Hq, T, D), dtype, 32, 2.0)
    scale = D ** -0.5
    mass = torch.ones((len(lens), H, table.shape[1] * P), device=DEV)
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens))
    out2, lse2 = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), mass=mass)
    fresh = [T] * len(lens)
    ro, rl, rm, av, aq = oc.cache_attention(ref, table, np.array(lens), fresh, q.double().numpy(), scale)
    check_fwd(out, lse, ro, rl, av, aq, D, dtype, fresh)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # a weight is off by 2·dt and 2^-19 (ex2, the stored logsumexp), sums of rows fp32
    dt = (D + 16) * 2.0 ** -23 * aq.max() + 2.0 ** -21 * np.abs(rl).max()
    got = mass.double().cpu().numpy() - 1.0
    assert (np.abs(got - rm) <= (2 * dt + 2.0 ** -19) * rm + 2.0 ** -23 * (1 + rm)).all()
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (256, 16)])
def test_many_sequences_one_warp_each(D, P):
    """Enough segments that every warp is a worker of its own; ragged, some empty of new tokens."""
    rng = np.random.default_rng(41)
    B, H, T = 160, 4, 2
    lens = rng.integers(0, 150, B)
    fresh = np.minimum(rng.integers(0, T + 1, B), lens)
    c, ref, table, _ = filled([int(n) for n in lens], H, D, P, BF, 42)
    q = rows((B, H, T, D), BF, 43)
    out = torch.full((B, H, T, D), 7.0, dtype=BF, device=DEV)
    lse = torch.full((B, H, T), 7.0, device=DEV)
    kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh), out=out, lse=lse)
    ro, rl, _, av, aq = oc.cache_attention(ref, table, lens, fresh, q.double().numpy(), D ** -0.5)
    check_fwd(out, lse, ro, rl, av, aq, D, BF, fresh)
    for b in range(B):  # rows of tokens that are not there stay as they were
        assert (out[b, :, fresh[b]:] == 7.0).all() and (lse[b, :, fresh[b]:] == 7.0).all()
    assert binding.device_status() == binding.ATTN_OK


def test_batches_wider_than_a_warp_share_workers():
    """More sequences than lanes, most without work: the deal's scan over the batch."""
    B = 300
    lens = np.zeros(B, int)
    lens[[5, 37, 64, 255, 299]] = [200, 1, 77, 3000, 64]
    fresh = (lens > 0).astype(int)
    c, ref, table, _ = filled([int(n) for n in lens], 1, 64, 16, BF, 45)
    q = rows((B, 1, 1, 64), BF, 46)
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh))
    ro, rl, _, av, aq = oc.cache_attention(ref, table, lens, fresh, q.double().numpy(), 0.125)
    check_fwd(out, lse, ro, rl, av, aq, 64, BF, fresh)


@pytest.mark.parametrize("B,width", [(3, 4), (3, 20000), (200, 4)])
def test_a_step_without_tokens_does_nothing(B, width):
    c = pool(8, 4, 64, 16, 47)
    before = to_np(c)
    table, lens, fresh = ints(np.zeros((B, width))), ints([40] + [0] * (B - 1)), ints([0] * B)
    table[0, :3] = ints([1, 2, 3])
    q, k = rows((B, 8, 2, 64), BF, 48).to(DEV), rows((B, 4, 2, 64), BF, 49).to(DEV)
    out, lse = torch.full_like(q, 5.0), torch.full((B, 8, 2), 5.0, device=DEV)
    mass = torch.full((B, 4, width * 16), 5.0, device=DEV) if width == 4 else None
    kv.cache_append(c, k, k, table, lens, fresh=fresh)
    kv.cache_fwd(q, c, table, lens, fresh=fresh, out=out, lse=lse, mass=mass)
    pages, scores = kv.cache_select(q, c, table, lens, 3, fresh=fresh)
    torch.cuda.synchronize()
    assert (out == 5.0).all() and (lse == 5.0).all() and (mass is None or (mass == 5.0).all())
    assert (pages == -1).all() and torch.isneginf(scores).all()
    after = to_np(c)
    assert all(np.array_equal(before[n], after[n]) for n in ("k", "v", "k_scale", "v_scale", "k_bounds"))
    assert binding.device_status() == binding.ATTN_OK


def test_calls_at_the_same_time_on_two_streams():
    lens = [3000, 700]
    c, ref, table, _ = filled(lens, 2, 128, 64, BF, 55, width=400)
    tb, ln = ints(table), ints(lens)
    qs = [rows((2, 8, 1, 128), BF, 56 + i).to(DEV) for i in range(2)]
    want = [kv.cache_fwd(q, c, tb, ln) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(kv.cache_fwd(qs[i], c, tb, ln, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(z, want[i][1]) for o, z in got[i])


def test_v_scales_far_apart_and_other_than_powers_of_two():
    lens, P, D = [256], 16, 64
    c, ref, table, _ = filled(lens, 2, D, P, BF, 51)
    s = np.exp2(np.random.default_rng(52).uniform(-40, 40, c.v_scale.shape)).astype(np.float32)
    c.v_scale.copy_(torch.from_numpy(s))
    ks = ref["k_scale"] * np.float32(1.3)
    c.k_scale.copy_(torch.from_numpy(ks))
    ref["v_scale"], ref["k_scale"] = s, ks
    q = rows((1, 4, 1, D), BF, 53)
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens))
    ro, rl, _, av, aq = oc.cache_attention(ref, table, np.array(lens), [1], q.double().numpy(), 0.125)
    check_fwd(out, lse, ro, rl, av, aq, D, BF, [1])
    # and where the pages with the weight hold values 2^60 below the others'
    k = torch.zeros_like(c.k[table[0, 3]])
    k.fill_(0x38)  # 1.0
    c.k[int(table[0, 3])] = k
    ref["k"][table[0, 3]] = 0x38
    c.k_scale[int(table[0, 3])] = 8.0
    ref["k_scale"][table[0, 3]] = 8.0
    s[:] = 1.0
    s[table[0, 3]] = 2.0 ** -60
    c.v_scale.copy_(torch.from_numpy(s))
    ref["v_scale"] = s
    q = torch.full((1, 4, 1, D), 4.0).to(BF)
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), scale=1.0)
    ro, rl, _, av, aq = oc.cache_attention(ref, table, np.array(lens), [1], q.double().numpy(), 1.0)
    assert (np.abs(ro) < 2.0 ** -50).any()
    o = out.double().cpu().numpy()
    assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * av).all()


def test_a_nan_reaches_only_the_rows_that_may_see_it():
    P, D, T = 32, 128, 3
    lens = [70]
    c, ref, table, _ = filled(lens, 1, D, P, FP, 61)
    q = rows((1, 2, T, D), FP, 62)
    base, _ = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens))
    g, slot = int(table[0, 2]), 68 % P
    c.v[g, 0, slot, 17] = 0x7f      # the second new token's value: rows 1 and 2 see it
    c.k[int(table[0, 2]), 0, 69 % P, 3] = 0xff  # the last token's key: row 2 only
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens))
    o, z = out.cpu(), lse.cpu()
    assert torch.equal(o[:, :, 0], base[:, :, 0].cpu()) and torch.isfinite(z[:, :, :2]).all()
    assert torch.isnan(o[:, :, 1, 17]).all() and torch.isnan(o[:, :, 1]).sum() == 2
    assert torch.equal(o[:, :, 1, :17], base[:, :, 1, :17].cpu())
    assert torch.isnan(o[:, :, 2]).all() and torch.isnan(z[:, :, 2]).all()


@pytest.mark.parametrize("P,T", [(16, 1), (32, 3), (64, 70 // 2)])
def test_listed_pages(P, T):
    D, Hq, H = 128, 6, 3
    lens = [20 * P + 5, 3 * P, T]
    c, ref, table, _ = filled(lens, H, D, P, BF, 71, width=24)
    rng = np.random.default_rng(72)
    N = 9
    pages = np.full((3, H, N), -1, np.int32)
    for b in range(3):
        for h in range(H):
            n = -(-lens[b] // P)
            pick = np.sort(rng.choice(n, min(n, [N, 2, 1][h]), replace=False))
            pages[b, h, :len(pick)] = pick
    pages[0, 1, :2] = [2, 23]  # a page behind the sequence's end: no token there
    pages[1, 2] = -1  # nothing at all
    q = rows((3, Hq, T, D), BF, 73)
    mass = torch.zeros((3, H, 24 * P), device=DEV)
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), pages=ints(pages), mass=mass)
    fresh = [T] * 3
    ro, rl, rm, av, aq = oc.cache_attention(ref, table, np.array(lens), fresh, q.double().numpy(), D ** -0.5,
                                            ListOf(pages, lens, P))
    check_fwd(out, lse, ro, rl, av, aq, D, BF, fresh)
    assert np.isneginf(lse.cpu().numpy()[1, 4:]).all() and (out[1, 4:] == 0).all()
    dt = (D + 16) * 2.0 ** -23 * aq.max() + 2.0 ** -21 * np.abs(rl[np.isfinite(rl)]).max()
    assert (np.abs(mass.double().cpu().numpy() - rm) <= (2 * dt + 2.0 ** -19) * rm + 2.0 ** -23 * rm).all()
    assert binding.device_status() == binding.ATTN_OK


class ListOf:
    """pages[b, h]: the listed pages that hold tokens."""

    def __init__(self, pages, lens, P):
        self.pages, self.lens, self.P = pages, lens, P

    def __getitem__(self, bh):
        return [int(i) for i in self.pages[bh] if 0 <= i * self.P < self.lens[bh[0]]]


def test_bad_entries_are_left_out_and_reported():
    D, P, H = 64, 16, 2
    lens = [100, 50, 40, 33]
    c, ref, table, _ = filled(lens, H, D, P, BF, 81, width=8)
    q = rows((4, 2, 1, D), BF, 82).to(DEV)
    good, _ = kv.cache_fwd(q, c, ints(table), ints(lens))
    def run(t=table, n=lens, **kw):
        out = torch.full_like(q, 3.0)
        kv.cache_fwd(q, c, ints(t), ints(n), out=out, **kw)
        torch.cuda.synchronize()
        return out, binding.device_status()
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 2] = bad
        out, st = run(t)
        assert st == binding.ATTN_ERR_DEVICE_CHECK
        assert torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
        # the page counts as not there
        pages = np.array([[[0, 1, 3, -1, -1, -1, -1]] * H for _ in range(4)], np.int32)
        want, _ = kv.cache_fwd(q, c, ints(table), ints(lens), pages=ints(pages))
        assert torch.allclose(out[1].float(), want[1].float(), rtol=2.0 ** -7, atol=2.0 ** -9)
        assert binding.device_status() == binding.ATTN_OK
        k = rows((4, H, 1, D), BF, 83).to(DEV)
        before = to_np(c)
        t = table.copy()
        t[1, 3] = bad  # where sequence 1's last token goes
        kv.cache_append(c, k, k, ints(t), ints([100, 50, 40, 33]))
        torch.cuda.synchronize()
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        after = to_np(c)
        changed = np.unique(np.nonzero((before["k"] != after["k"]).any(axis=(1, 2, 3)))[0])
        assert set(changed) <= {table[0, 6], table[2, 2], table[3, 2]}
        for n in ("k", "v", "k_scale", "v_scale", "k_bounds"):
            getattr(c, n).copy_(torch.from_numpy(before[n]))
    for bad in (-1, 8 * P + 1, 2 ** 31 - 1):
        n = list(lens)
        n[2] = bad
        out, st = run(n=n)
        assert st == binding.ATTN_ERR_DEVICE_CHECK
        assert torch.equal(out[[0, 1, 3]], good[[0, 1, 3]]) and (out[2] == 3.0).all()
        pages, scores = kv.cache_select(q, c, ints(table), ints(n), 3)
        torch.cuda.synchronize()
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        assert (pages[2] == -1).all() and torch.isneginf(scores[2]).all()
    t = table.copy()
    t[1, 0] = 10 ** 9
    pages, scores = kv.cache_select(q, c, ints(t), ints(lens), 2)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
    assert torch.isneginf(scores[1, :, 0]).all() and torch.isfinite(scores[1, :, 1:4]).all()
    for bad in (-1, 2):
        out, st = run(fresh=ints([1, 1, bad, 1]))
        assert st == binding.ATTN_ERR_DEVICE_CHECK and (out[2] == 3.0).all()
        assert torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])
    for entries in ([0, 2, 2, -1], [3, 1, -1, -1], [0, 8, -1, -1], [1, 2 ** 31 - 1, -1, -1], [-1, 2, -1, -1]):
        pages = np.array([[entries] * H for _ in range(4)], np.int32)
        out, st = run(pages=ints(pages))
        assert st == binding.ATTN_ERR_DEVICE_CHECK
        keep = [e for i, e in enumerate(entries) if 0 <= e < 8 and (i == 0 or 0 <= entries[i - 1] < e)]
        fine = np.array([[keep + [-1] * (4 - len(keep))] * H for _ in range(4)], np.int32)
        want, st = run(pages=ints(fine))
        assert st == binding.ATTN_OK
        assert torch.allclose(out.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -9)


def test_workspace_too_small_is_refused():
    c, _, table, _ = filled([30], 1, 64, 16, BF, 91, width=20000)
    q = rows((1, 1, 1, 64), BF, 92).to(DEV)
    # a short table: one CTA has each segment and nothing is joined
    assert kv.cache_fwd_workspace(c, ints(table[:, :2]), ints([30]), 1, 1) == 16
    need = kv.cache_fwd_workspace(c, ints(table), ints([30]), 1, 1)
    assert 16 < need < kv.cache_fwd_workspace(c, ints(table), ints([30]), 1, 1, with_mass=True)
    tb, ln = ints(table), ints([30])  # kept: the structures hold their addresses only
    lib, (cc, ss) = kv._library(), kv._views(c, tb, ln, None)[:2]
    out, lse = torch.empty_like(q), torch.empty((1, 1, 1), device=DEV)
    assert lib.attn_cache_fwd(cc, ss, q.data_ptr(), None, 0, out.data_ptr(), lse.data_ptr(), None, 1, 1, 0.1, 0, None,
                              need, 0, None) == binding.ATTN_ERR_INVALID_ARG
    with pytest.raises(binding.AttnError) as e:
        kv.cache_fwd(q, c, ints(table), ints([30]), workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.code == binding.ATTN_ERR_INVALID_ARG
    kv.cache_fwd(q, c, ints(table), ints([30]), workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        kv.cache_fwd(q.transpose(0, 1).expand(2, 1, 1, 64), c, ints(table), ints([30]))
    with pytest.raises(TypeError):
        kv.cache_fwd(q.float(), c, ints(table), ints([30]))
    with pytest.raises(ValueError):
        kv.cache_select(q, c, ints(table), ints([30]), 0)


def test_a_wait_that_runs_out_is_reported_and_recovers():
    # enough to read that the copies do not keep ahead of every wait
    B, H, S, P = 8, 8, 12000, 64
    n = -(-S // P)
    c = pool(B * n, H, 128, P, 95, stale=False)
    table, lens = torch.arange(B * n, dtype=torch.int32, device=DEV).view(B, n), ints([S] * B)
    k = torch.randn((B, H, S, 128), device=DEV).to(BF)
    kv.cache_append(c, k, k, table, lens)
    q = rows((B, 2 * H, 1, 128), BF, 96).to(DEV)
    good, _ = kv.cache_fwd(q, c, table, lens)
    assert torch.isfinite(good.float()).all()
    kv.cache_fwd(q, c, table, lens, wait_timeout_ns=0)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_ERR_TIMEOUT
    assert binding.device_status() == binding.ATTN_OK
    again, _ = kv.cache_fwd(q, c, table, lens)
    assert torch.equal(good, again)


# ---------------------------------------------------------------- select, evict
@pytest.mark.parametrize("D,P,Hq,H,T,dtype,lens,count", [
    (128, 64, 8, 2, 1, BF, [1000, 64, 1], 5),
    (64, 16, 4, 4, 3, FP, [300, 17, 3], 4),
    (72, 32, 5, 1, 2, BF, [700, 129], 30),
    (256, 16, 12, 1, 4, BF, [2100], 1),
    (128, 16, 66, 1, 1, FP, [5000], 100),
    (128, 16, 2, 1, 64, FP, [64, 100], 2),   # the new tokens alone are more pages than asked for
])
def test_select_meets_the_oracle(D, P, Hq, H, T, dtype, lens, count):
    c, ref, table, _ = filled(lens, H, D, P, dtype, 101, width=-(-max(lens) // P) + 2)
    q = rows((len(lens), Hq, T, D), dtype, 102)
    q[0, 0, 0, 0], q[0, Hq - 1, 0, 1] = float("inf"), float("nan")
    fresh = [min(T, n) for n in lens]
    fresh[-1] = fresh[-1] - 1 if T > 1 else fresh[-1]
    pages, scores = kv.cache_select(q.to(DEV), c, ints(table), ints(lens), count, fresh=ints(fresh))
    rp, rs = oc.cache_select(ref, table, np.array(lens), fresh, q.float().numpy(), count)
    assert np.array_equal(scores.cpu().numpy(), rs)
    assert np.array_equal(pages.cpu().numpy(), rp)
    assert binding.device_status() == binding.ATTN_OK


def test_select_among_more_pages_than_one_tile_of_registers_holds():
    P, D, n = 16, 16, 9001
    c = pool(n, 1, D, P, 107, stale=False)
    g = torch.Generator().manual_seed(108)
    hi = torch.randint(-20, 128, (n, 1, 1, 16), generator=g)
    lo = torch.minimum(hi, torch.randint(-127, 30, (n, 1, 1, 16), generator=g))
    c.k_bounds.copy_(torch.cat([hi, lo], dim=2).to(torch.int8))
    c.k_scale.copy_(torch.exp2(torch.randint(-3, 3, (n, 1), generator=g).float()))
    table = np.random.default_rng(109).permutation(n).reshape(1, n).astype(np.int32)
    lens = [P * (n - 1) + 3]
    q = rows((1, 3, 1, D), FP, 110)
    for count in (700, 1, 9000):
        pages, scores = kv.cache_select(q.to(DEV), c, ints(table), ints(lens), count)
        rp, rs = oc.cache_select(to_np(c), table, np.array(lens), [1], q.float().numpy(), count)
        assert np.array_equal(scores.cpu().numpy(), rs) and np.array_equal(pages.cpu().numpy(), rp)


def test_select_equal_scores_take_the_lowest_pages():
    c, ref, table, _ = filled([640], 1, 64, 16, BF, 105)
    c.k_bounds.fill_(3), c.k_scale.fill_(1.0)
    q = rows((1, 2, 1, 64), BF, 106).to(DEV)
    pages, _ = kv.cache_select(q, c, ints(table), ints([640]), 6)
    assert pages[0, 0].tolist() == [0, 1, 2, 3, 4, 39]
    q.zero_()
    pages, scores = kv.cache_select(q, c, ints(table), ints([640]), 60)
    assert pages[0, 0].tolist() == list(range(40)) + [-1] * 20 and (scores == 0).all()
    empty, none = kv.cache_select(q, c, ints(table), ints([640]), 2, fresh=ints([0]))
    assert (empty == -1).all() and torch.isneginf(none).all()


@pytest.mark.parametrize("D,P,H,lens,keep,recent", [
    (128, 64, 2, [1000, 300, 64, 0], 200, 50),
    (64, 16, 3, [333, 40], 40, 0),
    (72, 32, 1, [129], 33, 33),
    (256, 16, 2, [77, 500], 1, 1),
    (136, 64, 1, [2500], 1100, 100),
    (64, 16, 1, [5000], 4999, 4000),
    (8, 64, 1, [40000], 2000, 100),  # more weights than one tile of registers holds
])
def test_evict_meets_the_oracle(D, P, H, lens, keep, recent):
    dst_width = -(-keep // P) + 1
    c, ref, table, free = filled(lens, H, D, P, BF, 111, extra=len(lens) * dst_width + 1,
                                 width=-(-max(lens) // P) + 1)
    dst = free[:len(lens) * dst_width].reshape(len(lens), dst_width).astype(np.int32)
    rng = np.random.default_rng(112)
    mass = rng.integers(0, 40, (len(lens), H, table.shape[1] * P)).astype(np.float32) / 8  # many equal weights
    mass[:, :, 5::17] = np.nan
    mass[:, :, 3::29] = np.inf
    mass[:, :, 4::31] = -0.0
    want = oc.cache_evict(ref, mass, table, np.array(lens), dst, keep, recent)
    got = kv.cache_evict(c, torch.from_numpy(mass).to(DEV), ints(table), ints(lens), ints(dst), keep, recent)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=True)
    same_cache(c, ref)
    assert binding.device_status() == binding.ATTN_OK


def test_evict_does_not_write_pages_in_use_named_twice_or_out_of_range():
    P, D = 16, 64
    lens = [64, 48]
    c, ref, table, free = filled(lens, 1, D, P, BF, 121, extra=8)
    dst = free[:6].reshape(2, 3).astype(np.int32)
    mass = torch.rand((2, 1, table.shape[1] * P), device=DEV)
    before = to_np(c)
    for b, i, page in ((0, 0, table[1, 1]), (0, 1, dst[1, 2]), (1, 0, -1), (1, 1, c.k.shape[0]), (0, 2, table[0, 0])):
        d = dst.copy()
        d[b, i] = page
        kept, new_lens, _ = kv.cache_evict(c, mass, ints(table), ints(lens), ints(d), 40, 8)
        torch.cuda.synchronize()
        assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
        assert new_lens.tolist() == [40, 40] and (kept >= 0).all()
        after = to_np(c)
        for n in ("k", "v", "k_scale", "v_scale", "k_bounds"):
            for g in set(table.flatten()) - {-7}:
                assert np.array_equal(before[n][g], after[n][g])
        for n in ("k", "v", "k_scale", "v_scale", "k_bounds"):
            getattr(c, n).copy_(torch.from_numpy(before[n]))


# ---------------------------------------------------------------- together
def test_a_generation_as_it_would_run():
    """Prompts, drafted tokens with weights, an eviction, and sparse single steps."""
    P, D, H, Hq, dtype = 16, 128, 2, 6, BF
    pages = 200
    c = pool(pages, H, D, P, 131)
    ref = to_np(c)
    lens = np.array([150, 90])
    width = 12
    table, free = table_for([width * P] * 2, P, pages, 132)
    append_both(c, ref, table, lens, lens, 150, dtype, 133)
    mass = torch.zeros((2, H, width * P), device=DEV)
    rmass = np.zeros((2, H, width * P))
    T = 3
    for step in range(3):
        fresh = np.array([3, 1 + step % 2])
        lens = lens + fresh
        append_both(c, ref, table, lens, fresh, T, dtype, 140 + 2 * step)
        q = rows((2, Hq, T, D), dtype, 150 + step)
        out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh), mass=mass)
        ro, rl, rm, av, aq = oc.cache_attention(ref, table, lens, fresh, q.double().numpy(), D ** -0.5)
        check_fwd(out, lse, ro, rl, av, aq, D, dtype, fresh)
        rmass += rm
    assert np.allclose(mass.cpu().numpy(), rmass, rtol=1e-4, atol=1e-6)
    keep, recent = 64, 16
    dst = free[:16].reshape(2, 8).astype(np.int32)
    kept, new_lens, new_mass = kv.cache_evict(c, mass, ints(table), ints(lens), ints(dst), keep, recent)
    want = oc.cache_evict(ref, mass.cpu().numpy(), table, lens, dst, keep, recent)
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(new_mass.cpu().numpy(), want[2])
    same_cache(c, ref)
    lens = want[1].astype(int)
    for step in range(4):
        lens = lens + 1
        append_both(c, ref, dst, lens, None, 1, dtype, 160 + 2 * step)
        q = rows((2, Hq, 1, D), dtype, 170 + step)
        pages_t, _ = kv.cache_select(q.to(DEV), c, ints(dst), ints(lens), 3)
        rp, _ = oc.cache_select(ref, dst, lens, [1, 1], q.float().numpy(), 3)
        assert np.array_equal(pages_t.cpu().numpy(), rp)
        out, lse = kv.cache_fwd(q.to(DEV), c, ints(dst), ints(lens), pages=pages_t)
        ro, rl, _, av, aq = oc.cache_attention(ref, dst, lens, [1, 1], q.double().numpy(), D ** -0.5,
                                               ListOf(rp, lens, P))
        check_fwd(out, lse, ro, rl, av, aq, D, dtype, [1, 1])
    assert binding.device_status() == binding.ATTN_OK


def test_a_captured_step_replays_on_new_lengths_and_on_another_stream():
    P, D, H, Hq = 32, 128, 4, 8
    lens0 = [200, 31, 64]
    c, ref, table, _ = filled([260] * 3, H, D, P, FP, 181)
    tb, lens = ints(table), ints(lens0)
    k, v = (rows((3, H, 1, D), FP, s).to(DEV) for s in (182, 183))
    q = rows((3, Hq, 1, D), FP, 184).to(DEV)
    mass = torch.zeros((3, H, table.shape[1] * P), device=DEV)
    out, lse = torch.empty_like(q), torch.empty((3, Hq, 1), device=DEV)
    pages = torch.empty((3, H, 4), dtype=torch.int32, device=DEV)
    scores = torch.empty((3, H, table.shape[1]), device=DEV)
    ws = torch.empty(kv.cache_fwd_workspace(c, tb, lens, Hq, 1, 4, True), dtype=torch.uint8, device=DEV)

    def step():
        lens.add_(1)
        kv.cache_append(c, k, v, tb, lens)
        kv.cache_select(q, c, tb, lens, 4, pages=pages, scores=scores)
        kv.cache_fwd(q, c, tb, lens, pages=pages, mass=mass, out=out, lse=lse, workspace=ws)

    start = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale, c.k_bounds)]
    step()
    torch.cuda.synchronize()
    def reset():
        for t, s in zip((c.k, c.v, c.k_scale, c.v_scale, c.k_bounds), start):
            t.copy_(s)
        lens.copy_(ints(lens0)), mass.zero_()
    reset()
    eager = []
    for _ in range(3):
        step()
        eager.append((out.clone(), lse.clone(), pages.clone(), mass.clone()))
    reset()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for want in eager:
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((out, lse, pages, mass), want))
    # the same steps enqueued on another stream by name
    reset()
    torch.cuda.synchronize()
    for want in eager:
        with torch.cuda.stream(side):
            lens.add_(1)
        kv.cache_append(c, k, v, tb, lens, stream=side)
        p2, _ = kv.cache_select(q, c, tb, lens, 4, stream=side)
        o2, l2 = kv.cache_fwd(q, c, tb, lens, pages=p2, mass=mass, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((o2, l2, p2, mass), want))
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("D,P,Hq,H,T,lens", [
    (128, 64, 4, 2, 1, [700, 64, 1]),
    (64, 16, 2, 2, 3, [300] * 80),
    (8, 32, 2, 1, 2, [100, 33]),
    (136, 32, 3, 1, 20, [200, 20]),
    (256, 16, 2, 1, 1, [50] * 400),
])
def test_the_debug_build_finds_no_copy_out_of_its_bounds(monkeypatch, D, P, Hq, H, T, lens):
    c, _, table, _ = filled(lens, H, D, P, BF, 141)
    q = rows((len(lens), Hq, T, D), BF, 142, 2.0).to(DEV)
    want = kv.cache_fwd(q, c, ints(table), ints(lens))
    lib = kv.declare(binding.load_library(build_debug_library()))
    monkeypatch.setattr(kv, "_lib", lib)
    got = kv.cache_fwd(q, c, ints(table), ints(lens))
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.attn_device_status(stream) == binding.ATTN_OK
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("D,P,Hq,H,T,lens", [
    (128, 64, 2, 2, 1, [1, 64, 65, 1500, 17, 0, 300] * 12),   # dealt to CTAs, many segments of one chunk
    (80, 16, 8, 4, 3, [3, 1100, 64, 66, 129] * 9),
    (200, 32, 2, 2, 8, [8, 1100, 64, 66, 129] * 16),
    (64, 16, 32, 16, 1, [1, 900, 64, 17, 130, 2] * 10),       # dealt to warps
    (48, 16, 16, 16, 2, [2, 900, 64, 17, 130, 3] * 10),
    (112, 64, 6, 2, 3, [4, 2500]),                            # a cluster each
])
def test_segments_of_one_chunk_beside_long_ones(D, P, Hq, H, T, lens):
    """What a segment costs by itself is counted when the chunks are dealt: every chunk is still read once."""
    c, ref, table, _ = filled(lens, H, D, P, FP, 151)
    q = rows((len(lens), Hq, T, D), FP, 152)
    fresh = np.minimum(T, np.array(lens))
    out = torch.full((len(lens), Hq, T, D), 7.0, dtype=FP, device=DEV)
    lse = torch.full((len(lens), Hq, T), 7.0, device=DEV)
    kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh), out=out, lse=lse)
    ro, rl, _, av, aq = oc.cache_attention(ref, table, np.array(lens), fresh, q.double().numpy(), D ** -0.5)
    check_fwd(out, lse, ro, rl, av, aq, D, FP, fresh)
    for b, n in enumerate(fresh):
        assert (out[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("D", [8, 40, 72, 136, 200, 248])
@pytest.mark.parametrize("P", [16, 64])
def test_padding_channels_may_hold_anything(D, P):
    lens = [200, 31]
    c, _, table, _ = filled(lens, 2, D, P, BF, 161)
    q = rows((2, 4, 2, D), BF, 162).to(DEV)
    want = kv.cache_fwd(q, c, ints(table), ints(lens))
    c.k[..., D:] = 0x7f  # NaN codes
    c.v[..., D:] = 0xff
    got = kv.cache_fwd(q, c, ints(table), ints(lens))
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert torch.isfinite(got[0].float()).all()


def test_weights_and_scores_off_a_16_byte_boundary():
    """Weights and scores need 4-byte alignment only; the selection loads vectors where it can."""
    lens, H, D, P, keep = [3000, 5500], 2, 64, 16, 900
    dst_width = -(-keep // P)
    c, ref, table, free = filled(lens, H, D, P, BF, 171, extra=2 * dst_width)
    q = rows((2, 4, 1, D), BF, 172)
    off = lambda shape: torch.empty(int(np.prod(shape)) + 1, device=DEV)[1:].view(shape)
    scores = off((2, H, table.shape[1]))
    pages, _ = kv.cache_select(q.to(DEV), c, ints(table), ints(lens), 40, scores=scores)
    rp, rs = oc.cache_select(ref, table, np.array(lens), [1, 1], q.float().numpy(), 40)
    assert np.array_equal(scores.cpu().numpy(), rs) and np.array_equal(pages.cpu().numpy(), rp)
    dst = free[:2 * dst_width].reshape(2, dst_width).astype(np.int32)
    mass = np.random.default_rng(173).random((2, H, table.shape[1] * P)).astype(np.float32)
    want = oc.cache_evict(ref, mass, table, np.array(lens), dst, keep, 100)
    given, new_mass = off(mass.shape).copy_(torch.from_numpy(mass)), off((2, H, dst_width * P))
    got = kv.cache_evict(c, given, ints(table), ints(lens), ints(dst), keep, 100, new_mass=new_mass)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    same_cache(c, ref)
    assert binding.device_status() == binding.ATTN_OK
