"""GPU checks of the 8-bit cache on unusual values: NaN and infinities in queries
and keys, padding rows that hold anything, bounds of NaN-only channels, and every
kernel of the attention by width, rows of a pass and route."""
import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cache as kv
from oracle import cache as oc
from test_gpu_l_cache import BF, DEV, FP, check_fwd, clean_status, filled, ints, pool, rows, same_cache, to_np  # noqa: F401

pytestmark = pytest.mark.gpu

# The ways the attention's work is cut (152 SMs): lengths, heads and the table's
# width in pages of 64 tokens.  2817 = 44 chunks and one token, whose chunk is a
# worker's only one where chunks are dealt to CTAs (20 units a worker, 16 of them
# the segment's lead) and alone in its warp everywhere.
ROUTES = {
    "one CTA": ([65, 129, 1], 3),
    "cluster": ([2817, 65, 1], 45),
    "dealt to CTAs": ([2817, 65, 1], 2000),
    "dealt to warps": ([65, 129, 1] * 60, 3),
}


def call(c, q, table, lens, fresh, mass=True, fill=7.0):
    B, Hq, T, D = q.shape
    out = torch.full(q.shape, fill, dtype=q.dtype, device=DEV)
    lse = torch.full((B, Hq, T), fill, device=DEV)
    m = torch.zeros((B, c.k.shape[1], table.shape[1] * c.k.shape[2]), device=DEV) if mass else None
    kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh), mass=m, out=out, lse=lse)
    torch.cuda.synchronize()
    return out, lse, m


# ---------------------------------------------------------------- padding rows
@pytest.mark.parametrize("G", [2, 16])  # one pass of 6 rows, three of 16
@pytest.mark.parametrize("route", ROUTES)
def test_rows_behind_the_fresh_tokens_may_hold_anything(route, G):
    """Queries of tokens from fresh[b] on are not part of the step: no output or weight depends on them."""
    lens, width = ROUTES[route]
    T, D = 3, 128
    c, _, table, _ = filled(lens, 1, D, 64, BF, 11, width=width)
    fresh = np.minimum([[1, 3, 1][b % 3] for b in range(len(lens))], lens)
    q = rows((len(lens), G, T, D), BF, 12)
    want = call(c, q, table, lens, fresh)
    bad = q.clone()
    for b, n in enumerate(fresh):
        bad[b, :, n:] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38]).to(BF).repeat(D // 4)
        bad[b, ::2, n:, 5:] = q[b, ::2, n:, 5:]
    got = call(c, bad, table, lens, fresh)
    assert all(torch.isfinite(w).all() for w in (want[0].float(), want[1], want[2]))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert binding.device_status() == binding.ATTN_OK


# ---------------------------------------------------------------- NaN and infinities
def meets(out, lse, mass, ref, D, dtype, fresh):
    """check_fwd where the oracle is finite; where it is NaN, NaN."""
    ro, rl, rm, av, aq = (np.array(x) for x in ref)
    live = np.zeros(rl.shape, bool)
    for b, n in enumerate(fresh):
        live[b, :, :n] = True
    lost = np.isnan(rl) & live
    o, z, m = out.clone(), lse.clone(), mass.double().cpu().numpy()
    none = torch.from_numpy(np.isnan(ro) & live[..., None]).to(DEV)
    gone = torch.from_numpy(lost).to(DEV)
    assert torch.equal(torch.isnan(z) & torch.from_numpy(live).to(DEV), gone)
    assert torch.equal(torch.isnan(o) & torch.from_numpy(live[..., None]).to(DEV), none)
    assert np.array_equal(np.isnan(m), np.isnan(rm))
    for x in (ro, rl, av, aq):
        x[~np.isfinite(x) & ~np.isneginf(x)] = 0.0
    aq[lost] = 0.0
    check_fwd(o.masked_fill(none, 0.0), z.masked_fill(gone, 0.0), ro, rl, av, aq, D, dtype, fresh)
    fine = ~np.isnan(rm)
    # a weight is off by 2·dt and 2^-19 (ex2, the stored logsumexp), sums of rows fp32; ex2
    # gives 0 below 2^-126, for at most 64 rows of a key here
    dt = (D + 16) * 2.0 ** -23 * aq.max() + 2.0 ** -21 * np.abs(rl[np.isfinite(rl)]).max(initial=0.0)
    assert (np.abs(m[fine] - rm[fine]) <= (2 * dt + 2.0 ** -19) * rm[fine] + 2.0 ** -23 * rm[fine] + 2.0 ** -120).all()


def attend(c, ref, q, table, lens, fresh, dtype):
    D = c.head_dim
    with np.errstate(invalid="ignore", over="ignore"):
        want = oc.cache_attention(ref, table, np.array(lens), fresh, q.double().numpy(), D ** -0.5)
    meets(*call(c, q, table, lens, fresh), want, D, dtype, fresh)
    # without weights the same
    assert all(torch.equal(torch.nan_to_num(a, 5.0), torch.nan_to_num(b, 5.0))
               for a, b in zip(call(c, q, table, lens, fresh)[:2], call(c, q, table, lens, fresh, mass=False)[:2]))
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("G", [2, 18])  # one pass, two
@pytest.mark.parametrize("route", ROUTES)
def test_nan_and_infinite_queries(route, G, dtype):
    """A row's NaN stays in that row: out and lse NaN, and the weights of the keys it may see."""
    lens, width = ROUTES[route]
    T, D = 2, 128
    c, ref, table, _ = filled(lens, 1, D, 64, dtype, 21, width=width)
    fresh = np.minimum(T, lens)
    q = rows((len(lens), G, T, D), dtype, 22)
    q[0, 0, 0, 7] = float("nan")   # the first of two tokens: the last key keeps a finite weight
    q[1, 1, 1] = float("nan")
    q[1, 0, 0, 3] = float("inf")
    q[2, G - 1, 0, 100] = float("-inf")
    attend(c, ref, q, table, lens, fresh, dtype)


@pytest.mark.parametrize("route", ROUTES)
def test_a_nan_key_alone_in_its_chunk(route):
    """The last key's chunk holds no other key: its NaN is not taken for a chunk without keys."""
    lens, width = ROUTES[route]
    D = 128
    c, ref, table, _ = filled(lens, 1, D, 64, BF, 31, width=width)
    for b, n in enumerate(lens[:3]):
        g, slot = int(table[b, (n - 1) // 64]), (n - 1) % 64
        c.k[g, 0, slot, 5] = 0x7f
        ref["k"][g, 0, slot, 5] = 0x7f
    attend(c, ref, rows((len(lens), 2, 1, D), BF, 32), table, lens, [1] * len(lens), BF)


@pytest.mark.parametrize("route", ROUTES)
def test_a_nan_value_far_below_the_rest_still_counts(route):
    """A NaN value code makes its channel NaN, however small its weight and wherever the work is cut."""
    lens, width = ROUTES[route]
    D = 128
    c, ref, table, _ = filled(lens, 1, D, 64, BF, 41, width=width)
    q = rows((len(lens), 2, 1, D), BF, 42)
    for b, n in enumerate(lens[:2]):
        g, slot = int(table[b, (n - 1) // 64]), (n - 1) % 64
        for d in (c, ref):
            k, v = (d.k, d.v) if d is c else (d["k"], d["v"])
            k[g, 0, slot] = 0x78  # 256 in every channel: 256·scale, against q of one sign far below the others
            v[g, 0, slot, 9] = 0xff
        q[b] = -8.0
    attend(c, ref, q, table, lens, [1] * len(lens), BF)


@pytest.mark.parametrize("route", ROUTES)
def test_scores_of_minus_infinity(route):
    """Beside finite scores a weight of 0; a row of nothing else is NaN, unlike one that sees no key."""
    lens, width = ROUTES[route]
    D = 128
    c, ref, table, _ = filled(lens, 1, D, 64, BF, 51, width=width)
    for b, n in enumerate(lens[:3]):
        for i in range(-(-n // 64)):
            held = 0x38 if b != 1 or i == 0 else 0xb8  # 1, and -1 behind the first page of sequence 1
            c.k[int(table[b, i])], ref["k"][table[b, i]] = held, held
    q = rows((len(lens), 2, 1, D), BF, 52)
    q[0, 0, 0, 3] = float("-inf")
    q[1, 0, 0, 3] = float("inf")
    q[2, 1, 0, 3] = float("-inf")
    attend(c, ref, q, table, lens, [1] * len(lens), BF)
    # finite queries whose scores pass fp32's range behind a first page of zero keys
    for b, n in enumerate(lens[:2]):
        c.k[int(table[b, 0])], ref["k"][table[b, 0]] = 0, 0
        c.k_scale[table[b, 0]], ref["k_scale"][table[b, 0]] = 1.0, 1.0
        for i in range(1, -(-n // 64)):
            c.k_scale[int(table[b, i])], ref["k_scale"][table[b, i]] = 2.0 ** 90, 2.0 ** 90
    q = torch.full((len(lens), 2, 1, D), -(2.0 ** 60)).to(BF)
    q[2:] = 1.0
    out, lse, mass = call(c, q, table, lens, [1] * len(lens))
    # sequence 0: the zero keys of its first page have all the weight, evenly
    g = int(table[0, 0])
    v = oc.e4m3_values()[ref["v"][g, 0]] * float(ref["v_scale"][g, 0])
    assert np.abs(out[0].double().cpu().numpy() - v.mean(0)).max() <= 2.0 ** -8 * np.abs(v).max()
    assert torch.allclose(mass[0, 0, :64], torch.full((64,), 2.0 / 64, device=DEV), rtol=2.0 ** -18)
    assert (mass[0, 0, 64:] == 0).all() and torch.isfinite(lse[0]).all()


@pytest.mark.parametrize("width", [12, 2000])
def test_rows_of_a_list_without_keys_beside_nan_rows(width):
    """No key listed: 0 and -inf. NaN query over an empty list: still no key."""
    lens, D, H = [700, 130], 128, 2
    c, ref, table, _ = filled(lens, H, D, 64, BF, 61, width=width)
    pages = np.array([[[0, 10, -1], [-1, -1, -1]], [[2, -1, -1], [0, 1, 2]]], np.int32)
    q = rows((2, 4, 1, D), BF, 62)
    q[0, 0], q[0, 2], q[1, 1], q[1, 3, 0, 5] = [float("nan")] * 4
    out, lse = kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), pages=ints(pages))
    o, z = out.cpu().float(), lse.cpu()
    assert torch.isnan(o[0, 0]).all() and torch.isnan(z[0, 0]).all()
    assert (o[0, 2:] == 0).all() and torch.isneginf(z[0, 2:]).all()
    assert torch.isnan(o[1, [1, 3]]).all() and torch.isnan(z[1, [1, 3]]).all()
    assert torch.isfinite(o[[0, 1, 1], [1, 0, 2]]).all() and torch.isfinite(z[[0, 1, 1], [1, 0, 2]]).all()


# ---------------------------------------------------------------- one call behind another
@pytest.mark.parametrize("route", ROUTES)
def test_weights_are_those_of_their_own_call(route):
    """The weights' pass begins while the attention still writes the scores it reads: calls on
    one workspace, one right behind the other, get what each gets by itself."""
    lens, width = ROUTES[route]
    c, _, table, _ = filled(lens, 2, 128, 64, BF, 71, width=width)
    tb, ln = ints(table), ints(lens)
    qs = [rows((len(lens), 8, 1, 128), BF, 72 + i, 3.0).to(DEV) for i in range(3)]
    ws = torch.empty(kv.cache_fwd_workspace(c, tb, ln, 8, 1, with_mass=True), dtype=torch.uint8, device=DEV)
    mass = [torch.zeros((len(lens), 2, width * 64), device=DEV) for _ in range(33)]
    want = []
    for i, q in enumerate(qs):
        kv.cache_fwd(q, c, tb, ln, mass=mass[i], workspace=ws)
        torch.cuda.synchronize()
        want.append(mass[i].clone())
    for i in range(3, 33):
        kv.cache_fwd(qs[i % 3], c, tb, ln, mass=mass[i], workspace=ws)
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    for i in range(3, 33):
        assert torch.equal(mass[i], want[i % 3])


# ---------------------------------------------------------------- bounds
@pytest.mark.parametrize("grow", [False, True])
@pytest.mark.parametrize("D,P", [(64, 16), (72, 32), (128, 64)])
def test_bounds_behind_a_channel_of_nan_codes_and_behind_tokens_taken_back(D, P, grow):
    """While a page's scale stays its bounds are widened; where it grows they are found anew."""
    c = pool(4, 2, D, P, 81)
    ref = to_np(c)
    table = np.array([[2, 0]], np.int32)

    def append(k, v, n):
        kv.cache_append(c, k.to(DEV), v.to(DEV), ints(table), ints([n]))
        oc.cache_append(ref, table, np.array([n]), np.array([k.shape[2]]), k.double().numpy(), v.double().numpy())
        same_cache(c, ref)

    k, v = rows((1, 2, 6, D), BF, 82), rows((1, 2, 6, D), BF, 83)
    k[..., 0] = 4.0  # the first tokens hold the largest
    k[:, :, :, 3], k[:, 1, :, D - 1] = float("nan"), float("nan")
    append(k, v, 6)
    assert (c.k_bounds[2, :, :, 3] == 0).all() and (c.k_bounds[2, 1, :, D - 1] == 0).all()
    # all positive behind it: the 0 stays the lower bound where the scale stays
    k2, v2 = rows((1, 2, 3, D), BF, 84).abs() + 0.5, rows((1, 2, 3, D), BF, 85)
    k2 = (k2 * (60.0 if grow else 0.5)).to(BF)
    append(k2, v2, 9)
    lower = c.k_bounds[2, :, 1, 3]
    assert (lower > 0).all() if grow else (lower == 0).all()
    # the last two are taken back and others take their places
    k3, v3 = (rows((1, 2, 4, D), BF, 86 + i, 0.01) for i in range(2))
    append(k3, v3, 11)
    assert (c.k_bounds[2, :, 0, 3] > 0).all()
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("n,keep", [(300, 100), (3000, 1200), (20000, 9000)])
def test_evict_takes_nan_weights_last_of_all(n, keep):
    """NaN counts as less than every other weight, -inf among them."""
    D, P = 64, 16
    dw = -(-keep // P)
    c, ref, table, free = filled([n], 1, D, P, BF, 91, extra=dw)
    mass = np.random.default_rng(92).choice([-np.inf, np.nan, 1.0, 2.0, np.inf], (1, 1, table.shape[1] * P),
                                            p=[0.5, 0.35, 0.05, 0.05, 0.05]).astype(np.float32)
    dst = free[:dw].reshape(1, dw).astype(np.int32)
    want = oc.cache_evict(ref, mass, table, np.array([n]), dst, keep, 10)
    got = kv.cache_evict(c, torch.from_numpy(mass).to(DEV), ints(table), ints([n]), ints(dst), keep, 10)
    assert not np.isnan(mass[0, 0, want[0][0, 0, :-10]]).any()
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=True)
    same_cache(c, ref)


# ---------------------------------------------------------------- scales
@pytest.mark.parametrize("lo,hi", [(-100, -97), (-30, -20), (100, 119)])
def test_scales_over_the_whole_range(lo, hi):
    """Scales from 2^-100, the least that append writes, up to fp32's end; not powers of two."""
    lens, D = [700, 65], 64
    for width in (12, 2000):
        c, ref, table, _ = filled(lens, 2, D, 64, BF, 101, width=width)
        s = np.exp2(np.random.default_rng(102).uniform(lo, hi, c.v_scale.shape)).astype(np.float32)
        c.v_scale.copy_(torch.from_numpy(s))
        ref["v_scale"] = s
        q = rows((2, 4, 1, D), BF, 103)
        out, lse, _ = call(c, q, table, lens, [1, 1])
        ro, rl, _, av, aq = oc.cache_attention(ref, table, np.array(lens), [1, 1], q.double().numpy(), D ** -0.5)
        o = out.double().cpu().numpy()
        # the output's half step, P's 2^-11 and what check_fwd allows the scores, ex2 and sums
        dt = (D + 16) * 2.0 ** -23 * aq.max()
        assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * dt + 2.0 ** -18) * 1.01 * av).all()
        assert np.abs(lse.cpu().numpy() - rl).max() <= dt + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl).max()
    assert binding.device_status() == binding.ATTN_OK


# ---------------------------------------------------------------- workspaces
def test_the_workspace_query_refuses_what_the_attention_refuses():
    c, _, table, _ = filled([30], 1, 64, 16, BF, 111)
    tb, ln = ints(table), ints([30])
    assert kv.cache_fwd_workspace(c, tb, ln, 1, 1, listed=(2 ** 31 - 1) // 64) >= 16
    for kw in (dict(listed=(2 ** 31 - 1) // 64 + 1), dict(listed=2 ** 40), dict(listed=-1), dict(q_heads=0),
               dict(T=0), dict(T=65)):
        with pytest.raises(binding.AttnError) as e:
            kv.cache_fwd_workspace(c, tb, ln, **{**dict(q_heads=1, T=1), **kw})
        assert e.value.code == binding.ATTN_ERR_INVALID_ARG


# ---------------------------------------------------------------- select
@pytest.mark.parametrize("B,H,G,D,width", [(40, 16, 1, 64, 100), (10, 64, 2, 128, 70), (3, 2, 12, 128, 40000)])
def test_select_where_a_group_takes_several_pages(B, H, G, D, width):
    """More heads and pages than one wave of CTAs takes one page a group of."""
    P = 16
    lens = [int(n) for n in np.random.default_rng(121).integers(1, 60 * P, B)]
    c, ref, table, _ = filled(lens, H, D, P, FP, 122, width=width)
    q = rows((B, H * G, 1, D), FP, 123)
    pages, scores = kv.cache_select(q.to(DEV), c, ints(table), ints(lens), 7)
    rp, rs = oc.cache_select(ref, table, np.array(lens), [1] * B, q.float().numpy(), 7)
    assert np.array_equal(scores.cpu().numpy(), rs)
    assert np.array_equal(pages.cpu().numpy(), rp)
    assert binding.device_status() == binding.ATTN_OK


# ---------------------------------------------------------------- every kernel of the attention
ROWS = {8: (4, 2), 16: (8, 2), 24: (8, 3), 32: (16, 2), 40: (8, 5)}  # query rows of a head: heads of a group, tokens


@pytest.mark.parametrize("D,n", [(D, n) for D in (64, 48) for n in ROWS] +
                         [(D, n) for D in (128, 112, 256, 208) for n in (8, 16, 24)])
@pytest.mark.parametrize("route", ROUTES)
def test_every_width_and_number_of_rows_on_every_route(route, D, n):
    """Rows of whole 32 bytes and of odd 16-byte units; up to 32 rows a pass at 64 channels, 16 at more, and two
    or three passes."""
    lens, width = ROUTES[route]
    G, T = ROWS[n]
    c, ref, table, _ = filled(lens, 1, D, 64, FP, 131, width=width)
    q = rows((len(lens), G, T, D), FP, 132)
    attend(c, ref, q, table, lens, np.minimum(T, lens), FP)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("P,D", [(16, 64), (32, 80), (64, 256)])
def test_drafted_tokens_of_which_some_see_no_key_of_the_last_chunk(P, D, wide):
    """Tokens at 61 .. 65: the first three see none of the chunk of 64 and 65, where keys hold NaN."""
    lens, T = [66, 130, 5], 5
    c, ref, table, _ = filled(lens, 2, D, P, BF, 141, width=-(-130 // P) + (120000 // P if wide else 0))
    for b, n in enumerate(lens):
        at = n - 1 if b < 2 else 3  # the last token's key; of five tokens the fourth's
        for held in (c.k, ref["k"]):
            held[int(table[b, at // P]), 1, at % P, 2] = 0x7f
    q = rows((3, 6, T, D), BF, 142)
    q[1, 0, 1] = float("inf")
    q[0, 3, 4, 1], q[0, 1, 2, 1] = float("nan"), float("-inf")
    attend(c, ref, q, table, lens, [T, T - 2, T], BF)


# ---------------------------------------------------------------- what evict moves
@pytest.mark.parametrize("D,P", [(64, 16), (72, 32), (128, 64), (256, 16)])
def test_evict_moves_zeros_and_nans_of_pages_of_any_scale(D, P):
    """Kept tokens that are all zero stay zero whatever the scale of the page they come from."""
    n, keep, H = 6 * P, 3 * P - 1, 2
    c, ref, table, free = filled([n], H, D, P, BF, 151, extra=3)
    codes = np.random.default_rng(152).integers(0, 256, ref["k"].shape).astype(np.uint8)  # NaN codes among them
    for name in "kv":
        for i in range(4):  # zeros of both signs; in the second and fourth page NaN beside them
            codes[table[0, i]] = np.where(codes[table[0, i]] & 1, 0x80, 0)
            if i % 2:
                codes[table[0, i], :, ::3, 1::5] = 0x7f
        codes[..., D:] = 0
        ref[name][:] = codes
        getattr(c, name).copy_(torch.from_numpy(codes))
        s = np.exp2(np.random.default_rng(153).integers(-90, 119, ref[name + "_scale"].shape)).astype(np.float32)
        s[table[0, :4]] = 2.0 ** np.array([119, 100, 28, 27])[:, None]
        s[table[0, 4:]] = 2.0 ** np.array([3, -20])[:, None]
        ref[name + "_scale"][:] = s
        getattr(c, name + "_scale").copy_(torch.from_numpy(s))
    dst = free[:3].reshape(1, 3).astype(np.int32)
    mass = np.zeros((1, H, n), np.float32)
    mass[0, 0, :2 * P] = 1.0     # head 0 keeps the first pages and the last tokens
    mass[0, 1, P:4 * P:2] = 1.0  # head 1 parts of three
    want = oc.cache_evict(ref, mass, table, np.array([n]), dst, keep, P // 2)
    got = kv.cache_evict(c, torch.from_numpy(mass).to(DEV), ints(table), ints([n]), ints(dst), keep, P // 2)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    same_cache(c, ref)
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,P", [(64, 16), (72, 32), (256, 64)])
def test_append_of_extremes_in_both_types(D, P, dtype):
    """Largest and smallest values, infinities, NaN and zeros of both signs, in pages fresh and in use."""
    c = pool(4, 2, D, P, 161)
    ref = to_np(c)
    table = np.array([[2, 0, 1]], np.int32)
    big, least = torch.finfo(dtype).max, 2.0 ** (-24 if dtype is FP else -133)
    rng = np.random.default_rng(162)
    n = 0
    for step, T in enumerate([P // 2, 3, P // 2, 1, P // 4]):
        pick = [[0.0, -0.0, least, -3 * least], [1.0, -2.5, np.nan, 0.0], [big, -big, 1e-3, np.inf], [-np.inf, 1.0, 5.0, -0.0],
                [np.nan, np.inf, -np.inf, 0.0]][step]
        k, v = (torch.from_numpy(rng.choice(pick, (1, 2, T, D))).to(dtype) for _ in range(2))
        n += T
        kv.cache_append(c, k.to(DEV), v.to(DEV), ints(table), ints([n]))
        oc.cache_append(ref, table, np.array([n]), np.array([T]), k.double().numpy(), v.double().numpy())
        same_cache(c, ref)
    assert binding.device_status() == binding.ATTN_OK


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("D", [256, 208])  # tiled copies, runs of bytes
def test_a_pool_beyond_4_gib(D):
    """Pages whose offset passes 32 bits hold what the same pages of a small pool do."""
    H, P, n, T = 2, 64, 500, 70
    M, keep = -(-n // P), 200
    kx, vx = (rows((2, H, n, D), BF, 171 + i).to(DEV) for i in range(2))
    q = rows((2, 8, 3, D), BF, 173).to(DEV)
    got = []
    for total in (163840, 2 * M + 8):
        c = kv.cache_alloc(total, H, D, P, device=DEV)
        assert total < 1000 or c.k.numel() > 2 ** 32
        table = ints(np.random.default_rng(174).permutation(2 * M).reshape(2, M) + total - 2 * M - 8)
        dst = ints(np.arange(8).reshape(2, 4) + total - 8)
        mass = torch.zeros((2, H, M * P), device=DEV)
        kv.cache_append(c, kx[:, :, :n - T].contiguous(), vx[:, :, :n - T].contiguous(), table, ints([n - T] * 2))
        kv.cache_append(c, kx[:, :, n - T:].contiguous(), vx[:, :, n - T:].contiguous(), table, ints([n] * 2))
        out, lse = kv.cache_fwd(q, c, table, ints([n] * 2), mass=mass)
        pages, scores = kv.cache_select(q, c, table, ints([n] * 2), 4)
        out2, lse2 = kv.cache_fwd(q, c, table, ints([n] * 2), pages=pages)
        kept, lens, mass2 = kv.cache_evict(c, mass, table, ints([n] * 2), dst, keep, 20)
        out3, lse3 = kv.cache_fwd(q, c, dst, lens)
        got.append((out, lse, mass, pages, scores, out2, lse2, kept, lens, mass2, out3, lse3))
    assert all(torch.isfinite(x).all() for x in (got[0][0].float(), got[0][1], got[0][10].float()))
    assert got[0][0].float().abs().max() > 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert binding.device_status() == binding.ATTN_OK


def test_thousands_of_sequences_of_which_many_have_nothing_to_do():
    B, D, P = 5000, 64, 16
    rng = np.random.default_rng(181)
    lens = rng.integers(0, 40, B)
    fresh = np.minimum(rng.integers(0, 2, B), lens)
    c, ref, table, _ = filled([int(x) for x in lens], 1, D, P, BF, 182)
    q = rows((B, 2, 1, D), BF, 183)
    out, lse, _ = call(c, q, table, lens, fresh, mass=False)
    ro, rl, _, av, aq = oc.cache_attention(ref, table, lens, fresh, q.double().numpy(), 0.125)
    check_fwd(out, lse, ro, rl, av, aq, D, BF, fresh)
    idle = torch.from_numpy(fresh == 0).to(DEV)
    assert (out[idle] == 7.0).all() and (lse[idle] == 7.0).all()
    pages, scores = kv.cache_select(q.to(DEV), c, ints(table), ints(lens), 2, fresh=ints(fresh))
    rp, rs = oc.cache_select(ref, table, lens, fresh, q.float().numpy(), 2)
    assert np.array_equal(scores.cpu().numpy(), rs) and np.array_equal(pages.cpu().numpy(), rp)
    assert binding.device_status() == binding.ATTN_OK


# ---------------------------------------------------------------- eviction in a graph, and of what is left out
def test_a_captured_eviction_replays_on_new_lengths_and_weights():
    D, P, H, keep, recent = 128, 16, 2, 60, 10
    dw = -(-keep // P)
    c, ref, table, free = filled([200, 130], H, D, P, BF, 191, extra=2 * dw)
    dst = free[:2 * dw].reshape(2, dw).astype(np.int32)
    tb, ds, lens = ints(table), ints(dst), ints([200, 130])
    mass = torch.zeros((2, H, table.shape[1] * P), device=DEV)
    kept, new_lens = torch.empty((2, H, keep), dtype=torch.int32, device=DEV), ints([0, 0])
    new_mass = torch.empty((2, H, dw * P), device=DEV)
    ws = torch.empty(kv.cache_evict_workspace(c, tb, lens, dw), dtype=torch.uint8, device=DEV)

    def evict():
        kv.cache_evict(c, mass, tb, lens, ds, keep, recent, kept=kept, new_lens=new_lens, new_mass=new_mass,
                       workspace=ws)

    evict()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            evict()
    torch.cuda.current_stream().wait_stream(side)
    for i, n in enumerate([[200, 130], [61, 60], [5, 0], [199, 64]]):
        m = np.random.default_rng(192 + i).random(tuple(mass.shape)).astype(np.float32)
        mass.copy_(torch.from_numpy(m)), lens.copy_(ints(n))
        before = to_np(c)
        g.replay()
        torch.cuda.synchronize()
        want = oc.cache_evict(before, m, table, np.array(n), dst, keep, recent)
        for a, w in zip((kept, new_lens, new_mass), want):
            assert np.array_equal(a.cpu().numpy(), w)
        same_cache(c, before)
    assert binding.device_status() == binding.ATTN_OK


@pytest.mark.parametrize("bad", [-1, 200, 2 ** 31 - 1])
def test_evict_counts_a_sequence_left_out_as_empty_and_tokens_without_a_page_as_zeros(bad):
    D, P, keep = 64, 16, 20
    c, ref, table, free = filled([60, 50, 40], 1, D, P, BF, 201, extra=6)
    dst = free[:6].reshape(3, 2).astype(np.int32)
    m = np.random.default_rng(202).random((3, 1, table.shape[1] * P)).astype(np.float32)
    t = table.copy()
    t[2, 0] = bad  # no page of the pool (for 200: of 19)
    n = np.array([60, bad, 40])
    kept, lens, mass = kv.cache_evict(c, torch.from_numpy(m).to(DEV), ints(t), ints(n), ints(dst), keep, 4)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_ERR_DEVICE_CHECK
    assert lens.tolist() == [20, 0, 20] and (kept[1] == -1).all() and (mass[1] == 0).all()
    # as if the tokens of that page were zeros, and the sequence empty
    for name in "kv":
        ref[name][table[2, 0]] = 0
    want = oc.cache_evict(ref, m, table, np.array([60, 0, 40]), dst, keep, 4)
    for a, w in zip((kept, lens, mass), want):
        assert np.array_equal(a.cpu().numpy(), w)
    for name in "kv":
        ref[name][table[2, 0]] = getattr(c, name)[int(table[2, 0])].cpu().numpy()
    same_cache(c, ref)
