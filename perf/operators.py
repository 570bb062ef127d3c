"""Measured workloads of the 8-bit key/value cache operators, with their plain forms.

A cache is a pool of pages of P tokens.  For page g, key/value head h, token
slot s and channel d, ``k[g, h, s, d]`` and ``v[g, h, s, d]`` are e4m3 codes
(bytes), ``k_scale[g, h]`` and ``v_scale[g, h]`` their fp32 scales, and
``k_bounds[g, h, 0 / 1, d]`` the int8 upper / lower bound of the page's key
codes in steps of 448/127.  Rows are padded to a multiple of 16 channels.
Token j of sequence b lives in page ``table[b, j // P]``, slot ``j % P``;
``lens[b]`` tokens are in the cache, the last T of them this step's.

Operators: append (quantise new keys and values into the pages), fwd (attention
of the new tokens' queries over the cache, over all pages or over listed ones,
with the keys' attention weights accumulated on request), select (the pages a
cheap score picks for each sequence and head) and evict (the tokens with the
largest accumulated weight and the latest ones, moved into other pages).
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # smallest exponent of a page scale


# ------------------------------------------------------------------ the cases
def _case(op, B, Hq, Hkv, D, P, T, lo, hi, dtype="bf16", count=0, mass=False, keep=0, recent=0, name=None):
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, T=T, lo=lo, hi=hi, dtype=dtype, count=count, mass=mass, keep=keep,
             recent=recent)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one user's next token over a short context: launch and memory latency are all of it
        _case("fwd", 1, 32, 8, 128, 64, 1, 1000, 1000, name="fwd one sequence"),
        # a server's step over a mixed batch: ragged lengths, none a multiple of the page
        _case("fwd", 16, 32, 8, 128, 64, 1, 500, 8192, name="fwd ragged batch"),
        # a full server: many long sequences, bound by the memory
        _case("fwd", 64, 32, 8, 128, 64, 1, 8000, 16384, name="fwd large batch"),
        # one query head to each key head, small pages and heads, half precision
        _case("fwd", 8, 16, 16, 64, 16, 1, 100, 2048, "fp16", name="fwd heads apart"),
        # five drafted tokens checked at once, with the weights accumulated for a later eviction
        _case("fwd", 4, 32, 4, 128, 32, 5, 2000, 16384, mass=True, name="fwd drafts with mass"),
        # a very long context of which each head reads 64 pages
        _case("fwd", 4, 32, 8, 128, 64, 1, 100000, 131072, count=64, name="fwd listed pages"),
        # the choice of pages for one user
        _case("select", 1, 32, 8, 128, 64, 1, 16384, 16384, count=32, name="select one sequence"),
        # the choice among many small pages for a batch of long contexts
        _case("select", 8, 32, 8, 128, 16, 1, 50001, 65536, count=256, name="select small pages"),
        # the step's one token of each of 64 sequences
        _case("append", 64, 32, 8, 128, 64, 1, 1, 2048, name="append one token"),
        # two long prompts behind a shared beginning
        _case("append", 2, 32, 8, 128, 64, 8192, 8292, 8500, name="append prompts"),
        # one small sequence pair cut to 300 tokens a head
        _case("evict", 2, 16, 4, 64, 16, 1, 250, 1000, "fp16", keep=300, recent=64, name="evict small"),
        # a batch of long contexts cut to a fourth
        _case("evict", 8, 32, 8, 128, 64, 1, 4000, 16384, keep=4096, recent=256, name="evict batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "select", "append", "evict"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    D = rng.choice([64, 64, 72, 80, 96, 128, 128, 128, 192, 200, 256])
    P = rng.choice([16, 32, 64, 64])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    dtype = rng.choice(["bf16", "fp16"])
    B = _log(rng, 1, 64)
    token = 2 * Hkv * D * B  # bytes that one more token of every sequence takes
    T = rng.choice([1, 1, 1, 2, 3, 5, 8])
    rows = G * T if op in ("fwd", "select") else 1
    hi = _log(rng, 16, max(32, min(131072, (1 << 30) // (token * max(1, rows // 8)))))
    if op == "append":
        T = rng.choice([1, 1, 2, _log(rng, 1, 8192)])
        T = max(1, min(T, (1 << 27) // token))
        lo = T + _log(rng, 1, 1000) - 1
        return _case(op, B, Hkv, Hkv, D, P, T, lo, lo + _log(rng, 1, 1000) - 1, dtype)
    lo = rng.randint(T, hi)
    if op == "select":
        return _case(op, B, G * Hkv, Hkv, D, P, T, lo, hi, dtype, count=_log(rng, 1, max(1, hi // P)))
    if op == "evict":
        keep = _log(rng, 1, hi)
        return _case(op, B, Hkv, Hkv, D, P, 1, lo, hi, dtype, keep=keep, recent=rng.randint(0, keep))
    kind = rng.choice(["all", "all", "listed", "mass"])
    count = _log(rng, 1, max(1, min(hi // P, 256))) if kind == "listed" else 0
    return _case(op, B, G * Hkv, Hkv, D, P, T, lo, hi, dtype, count=count, mass=kind == "mass")


def _lens(c):
    """The sequences' lengths: spread over lo .. hi, the first the longest."""
    return [c["hi"] - int((c["hi"] - c["lo"]) * ((i * 0.6180339887) % 1.0)) for i in range(c["B"])]


def _pad(D):
    return -(-D // 16) * 16


def work(c):
    B, Hq, Hkv, D, P, T = (c[k] for k in ("B", "Hq", "Hkv", "D", "P", "T"))
    lens = _lens(c)
    if c["op"] == "append":
        return {"bytes": 2 * Hkv * D * 3 * B * T, "flops": 4 * Hkv * D * B * T}
    if c["op"] == "select":
        pages = sum(-(-n // P) for n in lens)
        return {"bytes": pages * Hkv * (2 * D + 4) + 2 * B * Hq * T * D + 4 * B * Hkv * c["count"],
                "flops": 4 * pages * Hq * T * D}
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens)
        return {"bytes": Hkv * (4 * sum(lens) + kept * (4 * D + 8)), "flops": Hkv * (sum(lens) + 4 * kept * D)}
    keys = sum(min(n, c["count"] * P) if c["count"] else n for n in lens)
    return {"bytes": 2 * Hkv * D * keys + 4 * B * Hq * T * D + 4 * B * Hq * T + (8 * Hkv * keys if c["mass"] else 0),
            "flops": 4 * D * Hq * T * keys}


# ------------------------------------------------------------------ the inputs
def _quantised(x, live):
    """e4m3 codes and page scales of x [pages, H, P, Dp]; live [pages, P]: the slots in use."""
    a = (x.abs() * live[:, None, :, None]).amax(dim=(2, 3)).float()
    f, e = torch.frexp(a)
    e = (e - 9 + (f > 0.875).int()).clamp(min=MIN_EXP)
    scale = torch.where(a > 0, torch.ldexp(torch.ones_like(a), e), torch.full_like(a, 2.0 ** MIN_EXP))
    return (x / scale[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _bounds(codes, live):
    """int8 bounds [pages, H, 2, Dp] of the codes in use."""
    x, m = codes.to(torch.float16), live[:, None, :, None]
    hi = x.masked_fill(~m, -math.inf).amax(dim=2).float()
    lo = x.masked_fill(~m, math.inf).amin(dim=2).float()
    some, one = live.any(1)[:, None, None], torch.full_like(hi, E4M3_MAX)
    # a division by a tensor: one rounding, exact where the quotient is whole
    hi = torch.where(some, torch.ceil(torch.div(hi * 127.0, one)), torch.zeros_like(hi))
    lo = torch.where(some, torch.floor(torch.div(lo * 127.0, one)), torch.zeros_like(lo))
    return torch.stack([hi, lo], dim=2).to(torch.int8)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    B, Hq, Hkv, D, P, T = (c[k] for k in ("B", "Hq", "Hkv", "D", "P", "T"))
    Dp, dt = _pad(D), torch.float16 if c["dtype"] == "fp16" else torch.bfloat16
    lens = _lens(c)
    M = -(-max(lens) // P)
    need = [-(-n // P) for n in lens]
    Md = -(-min(max(lens), c["keep"]) // P) if c["op"] == "evict" else 0
    n_pages = sum(need) + B * Md + 3
    perm = torch.randperm(n_pages, generator=g, **dev).int()
    table, at = torch.zeros(B, M, dtype=torch.int32, **dev), 0
    filled = torch.full((n_pages,), 0, dtype=torch.int64, **dev)
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        held = lens[b] - (T if c["op"] == "append" else 0)
        filled[perm[at:at + n].long()] = (held - torch.arange(n, **dev) * P).clamp(0, P)
        at += n
    live = torch.arange(P, **dev)[None, :] < filled[:, None]

    # keys with a few strong channels, values around zero: what projections give
    strong = 1.0 + 4.0 * (torch.rand(Hkv, 1, Dp, generator=g, **dev) > 0.95)
    real = (torch.arange(Dp, **dev) < D).half()
    cache = {}
    for name, weight in (("k", strong.half()), ("v", 1.0)):
        x = torch.randn(n_pages, Hkv, P, Dp, generator=g, dtype=torch.float16, **dev) * weight * real
        codes, scale = _quantised(x, live)
        cache[name], cache[name + "_scale"] = codes.view(torch.uint8), scale
    del x
    cache["k_bounds"] = _bounds(cache["k"].view(torch.float8_e4m3fn), live)
    s = dict(case=c, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, **dev))
    if c["op"] == "append":
        for name in "kv":
            x = torch.randn(B, Hkv, T, D, generator=g, **dev)
            s[name] = (x * strong[:, :, :D] if name == "k" else x).to(dt)
    if c["op"] in ("fwd", "select"):
        s["q"] = torch.randn(B, Hq, T, D, generator=g, **dev).to(dt)
    if c["mass"] or c["op"] == "evict":
        live_keys = torch.arange(M * P, **dev)[None, None] < s["lens"][:, None, None]
        s["mass"] = torch.randn(B, Hkv, M * P, generator=g, **dev).mul(2).exp() * live_keys
    if c["op"] == "fwd" and c["count"]:
        # listed pages: the first, those of the new tokens, and others by chance
        u = torch.rand(B, Hkv, M, generator=g, **dev)
        i, n = torch.arange(M, **dev), ((s["lens"] + P - 1) // P)[:, None, None]
        u = torch.where(i >= (s["lens"][:, None, None] - T) // P, 2.0, u)
        u = torch.where(i < n, torch.where(i == 0, 1.5, u), -1.0)
        top, idx = u.topk(min(c["count"], M), dim=2)
        idx = torch.where(top >= 0, idx, M).sort(dim=2).values
        idx = torch.where(idx < M, idx, -1).int()
        s["pages"] = torch.full((B, Hkv, c["count"]), -1, dtype=torch.int32, **dev)
        s["pages"][:, :, :idx.shape[2]] = idx
    if c["op"] == "evict":
        s["dst_table"] = perm[at:at + B * Md].view(B, Md).clone()
    return s


# ------------------------------------------------------------------ the plain forms
def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None, None]


def _plain_append(s):
    c, cache = s["case"], s["cache"]
    P, T, D = c["P"], c["T"], c["D"]
    start = s["lens"].long() - T
    first = start // P
    n = (T + P - 2) // P + 1  # pages that T tokens can touch
    i = first[:, None] + torch.arange(n, device="cuda")  # [B, n]
    used = i * P < s["lens"][:, None]
    b, j = torch.nonzero(used, as_tuple=True)
    i, page = i[b, j], s["table"].long()[b, i[b, j]]
    pos = i[:, None] * P + torch.arange(P, device="cuda")  # [N, P]
    rel = pos - start[b][:, None]
    fresh, old = (rel >= 0) & (rel < T), rel < 0
    for name in "kv":
        x = s[name].float()[b[:, None], :, rel.clamp(0, T - 1)].transpose(1, 2)  # [N, H, P, D]
        x = torch.nn.functional.pad(x, (0, _pad(D) - D))
        fine = torch.isfinite(x) & fresh[:, None, :, None]
        a = torch.where(fine, x.abs(), 0.0).amax(dim=(2, 3))
        f, e = torch.frexp(a)
        e = (e - 9 + (f > 0.875).int()).clamp(min=MIN_EXP)
        scale = torch.where(a > 0, torch.ldexp(torch.ones_like(a), e), torch.full_like(a, 2.0 ** MIN_EXP))
        was = cache[name + "_scale"][page]
        scale = torch.where(old.any(1)[:, None], torch.maximum(was, scale), scale)
        codes = cache[name][page].view(torch.float8_e4m3fn).float()
        codes = torch.where(old[:, None, :, None], codes * (was / scale)[..., None, None], codes)
        new = (x / scale[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
        codes = torch.where(fresh[:, None, :, None], new, codes).to(torch.float8_e4m3fn)
        cache[name][page] = codes.view(torch.uint8)
        cache[name + "_scale"][page] = scale
        if name == "k":
            cache["k_bounds"][page] = _bounds(codes, fresh | old)


def _plain_fwd(s):
    c, cache = s["case"], s["cache"]
    B, Hq, Hkv, D, P, T = (c[k] for k in ("B", "Hq", "Hkv", "D", "P", "T"))
    M = s["table"].shape[1]
    lens = s["lens"].long()
    if c["count"]:
        at = s["pages"].long()  # [B, H, N]
        page = torch.gather(s["table"].long()[:, None].expand(B, Hkv, M), 2, at.clamp(min=0))
        there = (at >= 0)[..., None].expand(-1, -1, -1, P)
    else:
        at = torch.arange(M, device="cuda").expand(B, Hkv, M)
        page = s["table"].long()[:, None].expand(B, Hkv, M)
        there = torch.ones(1, 1, 1, 1, dtype=torch.bool, device="cuda").expand(B, Hkv, M, P)
    N = at.shape[2]
    pos = (at[..., None] * P + torch.arange(P, device="cuda")).view(B, Hkv, 1, N * P)
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k = _values(cache["k"][page, head], cache["k_scale"][page, head])[..., :D].reshape(B, Hkv, N * P, D)
    q = s["q"].float().view(B, Hkv, Hq // Hkv * T, D)
    t = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    token = torch.arange(Hq // Hkv * T, device="cuda") % T
    last = (lens[:, None] - T + token)[:, None, :, None]
    t = t.masked_fill(~((pos <= last) & there.reshape(B, Hkv, 1, N * P)), -math.inf)
    m = t.amax(dim=3, keepdim=True).clamp(min=-3e38)
    p = torch.exp(t - m)
    l = p.sum(dim=3, keepdim=True)
    p = p / l.clamp(min=1e-38)
    v = _values(cache["v"][page, head], cache["v_scale"][page, head])[..., :D].reshape(B, Hkv, N * P, D)
    # slots behind the sequence's end hold anything
    v = torch.where((pos < lens[:, None, None, None]).transpose(2, 3), v, 0.0)
    out = torch.matmul(p, v).view(B, Hq, T, D).to(s["q"].dtype)
    r = {"out": out, "lse": (m + torch.log(l)).view(B, Hq, T)}
    if c["mass"]:
        at = torch.where(there.reshape(B, Hkv, N * P), pos[:, :, 0], 0)
        s["mass"].scatter_add_(2, at, p.sum(dim=2))
        r["mass"] = s["mass"]
    return r


def _plain_select(s):
    c, cache = s["case"], s["cache"]
    B, Hq, Hkv, D, P, T = (c[k] for k in ("B", "Hq", "Hkv", "D", "P", "T"))
    M, lens = s["table"].shape[1], s["lens"].long()
    q = s["q"].float().view(B, Hkv, Hq // Hkv * T, D)
    a = q.abs().amax(dim=3, keepdim=True)
    steps = torch.div(torch.full_like(a, 127.0), a)
    qi = torch.round(q * torch.where(a > 0, steps, 0.0)).clamp(-127, 127)
    page = s["table"].long()
    bounds = cache["k_bounds"][page].float()[..., :D].transpose(1, 2)  # [B, H, M, 2, D]
    # whole numbers below 2^24: exact in 32 bits in any order
    up = torch.matmul(qi.clamp(min=0), bounds[:, :, :, 0].transpose(2, 3))
    up += torch.matmul(qi.clamp(max=0), bounds[:, :, :, 1].transpose(2, 3))
    score = (up * cache["k_scale"][page].transpose(1, 2)[:, :, None]) * a
    i, n = torch.arange(M, device="cuda"), ((lens + P - 1) // P)[:, None, None]
    score = torch.where(i < n, score.amax(dim=2), -math.inf)  # [B, H, M]
    # the pages of the new tokens first, the latest of them before the others
    recent = ((lens - T) // P)[:, None, None]
    order = torch.where((i >= recent) & (i < n), 1e300 * (1.0 + i / (2.0 * M)), score.double())
    top, idx = order.sort(dim=2, descending=True, stable=True)
    N = min(c["count"], M)
    idx = torch.where(top[:, :, :N] > -math.inf, idx[:, :, :N], M).sort(dim=2).values
    pages = torch.full((B, Hkv, c["count"]), -1, dtype=torch.int32, device="cuda")
    pages[:, :, :N] = torch.where(idx < M, idx, -1).int()
    return {"pages": pages, "scores": score}


def _plain_evict(s):
    c, cache = s["case"], s["cache"]
    B, Hkv, D, P, keep, recent = (c[k] for k in ("B", "Hkv", "D", "P", "keep", "recent"))
    lens, cap = s["lens"].long(), s["mass"].shape[2]
    i = torch.arange(cap, device="cuda")
    rank = torch.where(i < (lens - recent)[:, None, None], s["mass"], math.inf)
    rank = torch.where(i < lens[:, None, None], rank, -1.0)
    N = min(keep, cap)
    # the latest first, then by weight; equal ones by the lowest index
    order = torch.where(torch.isinf(rank), 1e300 * (1.0 + i / (2.0 * cap)), rank.double())
    idx = order.sort(dim=2, descending=True, stable=True).indices[:, :, :N]
    left = lens.clamp(max=keep)
    idx = torch.where(torch.arange(N, device="cuda") < left[:, None, None], idx, cap).sort(dim=2).values
    # sorting by weight put the chosen `left` first: behind them nothing is kept
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    kept[:, :, :N] = torch.where(idx < cap, idx, -1).int()
    Md = s["dst_table"].shape[1]
    take = torch.full((B, Hkv, Md * P), -1, dtype=torch.int64, device="cuda")
    take[:, :, :N] = kept[:, :, :N].long()
    have = take >= 0
    src = take.clamp(min=0)
    page = torch.gather(s["table"].long()[:, None].expand(-1, Hkv, -1), 2, src // P)
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    dst = s["dst_table"].long()
    full = (torch.arange(Md, device="cuda") * P < left[:, None])  # destination pages in use
    for name in "kv":
        x = cache[name][page, head, src % P].view(torch.float8_e4m3fn).float()
        x = x * cache[name + "_scale"][page, head][..., None]
        x = x.view(B, Hkv, Md, P, -1).transpose(1, 2)[full]  # [N, H, P, Dp]
        there = have[:, 0].view(B, Md, P)[full]
        codes, scale = _quantised(x, there)
        was = cache[name][dst[full]].view(torch.float8_e4m3fn)
        codes = torch.where(there[:, None, :, None], codes.view(torch.uint8), was.view(torch.uint8))
        cache[name][dst[full]] = codes
        cache[name + "_scale"][dst[full]] = scale
        if name == "k":
            cache["k_bounds"][dst[full]] = _bounds(codes.view(torch.float8_e4m3fn), there)
    mass = torch.where(have, torch.gather(s["mass"], 2, src), 0.0)
    return {"kept": kept, "lens": left.int(), "mass": mass}


def _cache_out(s):
    """The cache as numbers: e4m3 values beside their scales, int8 bounds."""
    c = s["cache"]
    return {"k": c["k"].view(torch.float8_e4m3fn), "v": c["v"].view(torch.float8_e4m3fn), "k_scale": c["k_scale"],
            "v_scale": c["v_scale"], "k_bounds": c["k_bounds"]}


def run(s):
    op = s["case"]["op"]
    if own:
        from exact_attention_68_gb300 import cache as kv
        c = s["cache"]
        cache = kv.KVCache8(c["k"], c["v"], c["k_scale"], c["v_scale"], c["k_bounds"], s["case"]["D"])
        if op == "append":
            kv.cache_append(cache, s["k"], s["v"], s["table"], s["lens"])
            return _cache_out(s)
        if op == "fwd":
            out, lse = kv.cache_fwd(s["q"], cache, s["table"], s["lens"], pages=s.get("pages"), mass=s.get("mass"))
            return {"out": out, "lse": lse, **({"mass": s["mass"]} if "mass" in s else {})}
        if op == "select":
            pages, scores = kv.cache_select(s["q"], cache, s["table"], s["lens"], s["case"]["count"])
            return {"pages": pages, "scores": scores}
        kept, lens, mass = kv.cache_evict(cache, s["mass"], s["table"], s["lens"], s["dst_table"], s["case"]["keep"],
                                          s["case"]["recent"])
        return {"kept": kept, "lens": lens, "mass": mass, **_cache_out(s)}
    if op == "append":
        _plain_append(s)
        return _cache_out(s)
    if op == "fwd":
        return _plain_fwd(s)
    if op == "select":
        return _plain_select(s)
    return {**_plain_evict(s), **_cache_out(s)}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_64(x):
    """x rounded to the nearest e4m3 value (ties to even), saturating, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _decoded(codes):
    """e4m3 bytes as 64-bit values, by their bits: sign, 4 bits of exponent, 3 of fraction."""
    b = codes.long()
    e, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e > 0, (8 + f) * torch.exp2((e - 10).double()), f * 2.0 ** -9)
    x = torch.where((b & 127) == 127, math.nan, x)
    return torch.where(b > 127, -x, x)


def _scale64(x):
    """The page scale for values x: the smallest power of two (at least 2^MIN_EXP) with |x| <= 448 scales."""
    a = float(x.abs().max()) if x.numel() else 0.0
    e = MIN_EXP
    if a > 0:
        e = max(MIN_EXP, math.floor(math.log2(a)) - 9)
        while a > E4M3_MAX * 2.0 ** e:
            e += 1
    return 2.0 ** e


def _exact_pages(s, todo):
    """Rewrites pages in 64 bits.  todo: (page, head, slots kept, first new slot, new k, new v)."""
    out = {n: _decoded(s["cache"][n]) for n in "kv"}
    scales = {n: s["cache"][n + "_scale"].double().cpu().numpy().copy() for n in "kv"}
    for page, h, held, xk, xv in todo:
        for n, x in (("k", xk), ("v", xv)):
            sc = _scale64(x)
            if held:
                was = scales[n][page, h]
                sc = max(sc, was)
                if sc != was:
                    out[n][page, h, :held] = _e4m3_64(out[n][page, h, :held] * (was / sc))
            out[n][page, h, held:held + x.shape[0], :x.shape[1]] = _e4m3_64(x / sc)
            scales[n][page, h] = sc
    return {"k": out["k"], "v": out["v"], "k_scale": torch.from_numpy(scales["k"]).cuda(),
            "v_scale": torch.from_numpy(scales["v"]).cuda(), "k_bounds": None}


def exact(c, seed):
    s = prepare(c, seed)
    B, Hq, Hkv, D, P, T = (c[k] for k in ("B", "Hq", "Hkv", "D", "P", "T"))
    lens, table = _lens(c), s["table"].cpu().numpy()
    if c["op"] == "select":
        scores = torch.full((B, Hkv, table.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            at = s["table"][b, :-(-lens[b] // P)].long()
            for h in range(Hkv):
                q = s["q"][b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].reshape(-1, D)
                a = q.abs().amax(dim=1, keepdim=True).float()
                # the rounded queries are by definition those of 32-bit arithmetic
                steps = torch.div(torch.full_like(a, 127.0), a)
                qi = torch.round(q.float() * torch.where(a > 0, steps, 0.0)).double()
                w = s["cache"]["k_bounds"][at, h, :, :D].double()  # [pages, 2, D]
                best = torch.maximum(qi[:, None] * w[None, :, 0], qi[:, None] * w[None, :, 1]).sum(dim=2)
                scores[b, h, :len(at)] = (best * a.double() * s["cache"]["k_scale"][at, h].double()).amax(dim=0)
        return {"pages": None, "scores": scores}
    if c["op"] == "append":
        if B * Hkv * (T // P + 2) > 4000:
            return None
        todo = []
        for b in range(B):
            start = lens[b] - T
            for i in range(start // P, -(-lens[b] // P)):
                u, w = max(i * P, start), min((i + 1) * P, lens[b])
                for h in range(Hkv):
                    todo.append((int(table[b, i]), h, u - i * P, s["k"][b, h, u - start:w - start].double(),
                                 s["v"][b, h, u - start:w - start].double()))
        return _exact_pages(s, todo)
    if c["op"] == "evict":
        if B * Hkv * (min(max(lens), c["keep"]) // P + 1) > 5000:
            return None
        mass, dst = s["mass"].cpu().numpy(), s["dst_table"].cpu().numpy()
        todo, moved = [], np.zeros((B, Hkv, dst.shape[1] * P))
        old = {n: _decoded(s["cache"][n]) * s["cache"][n + "_scale"].double()[..., None, None] for n in "kv"}
        for b in range(B):
            n = lens[b]
            for h in range(Hkv):
                w = mass[b, h, :n]
                tail = min(c["recent"], n)
                best = np.argsort(-w[:n - tail], kind="stable")[:max(0, c["keep"] - tail)]
                kept = np.sort(np.concatenate([best, np.arange(n - tail, n)])) if n > c["keep"] else np.arange(n)
                moved[b, h, :len(kept)] = w[kept]
                for i in range(-(-len(kept) // P)):
                    at = kept[i * P:(i + 1) * P]
                    pg = torch.from_numpy(table[b, at // P].astype(np.int64)).cuda()
                    sl = torch.from_numpy(at % P).cuda()
                    todo.append((int(dst[b, i]), h, 0, old["k"][pg, h, sl], old["v"][pg, h, sl]))
        return {"kept": None, "lens": None, "mass": torch.from_numpy(moved), **_exact_pages(s, todo)}
    outs, lses = [], []
    mass = s["mass"].double() if c["mass"] else None
    for b in range(B):
        n = lens[b]
        for h in range(Hkv):
            pages = s["pages"][b, h][s["pages"][b, h] >= 0].long() if c["count"] else torch.arange(-(-n // P), device="cuda")
            pos = (pages[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
            keep = pos < n
            at = s["table"][b].long()[pages]
            k, v = ((_decoded(s["cache"][x][at, h]) * s["cache"][x + "_scale"][at, h].double()[:, None, None]).reshape(-1, _pad(D))[keep][:, :D]
                    for x in "kv")
            G = Hq // Hkv
            t = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)  # [G, T, keys]
            last = n - T + torch.arange(T, device="cuda")
            t = t.masked_fill(pos[keep][None, None] > last[None, :, None], -math.inf)
            z = torch.logsumexp(t, dim=2)
            p = torch.exp(t - z.clamp(min=-1e300)[..., None])
            outs.append(p @ v)
            lses.append(z)
            if c["mass"]:
                mass[b, h].index_add_(0, pos[keep], p.sum(dim=(0, 1)))
    r = {"out": torch.cat(outs).view(B, Hq, T, D), "lse": torch.cat(lses).view(B, Hq, T)}
    return {**r, "mass": mass} if c["mass"] else r
