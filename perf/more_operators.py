"""Measured workloads of cross attention and of the heads' norm and rotation, with their plain forms.

cross, cross_bwd: queries q [B, Hq, Sq, D] attend to another sequence's keys and
values k, v [B, Hkv, Sk, D] of which sequence b has lens[b]; query heads
h·G .. h·G+G-1 share key/value head h.  With t = scale·q·kᵀ over j < lens[b],
lse = ln Σ exp(t) and out = exp(t - lse)·v; a sequence without keys gives out 0
and lse -inf.  The gradient takes out, lse and dout, and gives dq, dk, dv and
delta = rowsum(dout ⊙ out).

rope, rope_bwd: what stands between a block's packed projection
[B, S, (Hq + 2·Hkv)·D] and its attention.  Each head of q and k is divided by its
root mean square and weighted, z = w·x / sqrt(mean(x²) + eps), and its first R
channels are turned in pairs, pair i by positions[b, s, axis[i]]·inv_freq[i]; v
passes; all three leave as [B, H, S, D].  The pairs are (i, i + R/2), or (2i, 2i+1)
where `interleaved`.  The gradient gives that of the projection and of both weights.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _cross(op, B, Hq, Hkv, Sq, Sk, D, dtype="bf16", lo=None, name=None):
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, dtype=dtype, lo=Sk if lo is None else lo)
    return c if name is None else dict(c, name=name)


def _rope(op, B, S, Hq, Hkv, D, R, axes=1, interleaved=False, dtype="bf16", weight="same", name=None):
    c = dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, R=R, axes=axes, interleaved=interleaved, dtype=dtype, weight=weight)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # the next token of 16 users: launch latency is all of it
        _rope("rope", 16, 1, 32, 8, 128, 128, name="rope one token"),
        # a training step's tokens, shared key heads
        _rope("rope", 2, 4096, 32, 8, 128, 128, name="rope training batch"),
        # 8 x 30 x 53 video patches: three axes, an odd head size
        _rope("rope", 1, 12720, 16, 16, 72, 72, 3, True, "fp16", name="rope video patches"),
        # the same two on the way back
        _rope("rope_bwd", 2, 4096, 32, 8, 128, 128, name="rope gradient training"),
        _rope("rope_bwd", 1, 12720, 16, 16, 72, 72, 3, True, "fp16", "fp32", name="rope gradient video"),
        # a decoder's next token over its encoder's states: memory and latency
        _cross("cross", 8, 16, 16, 1, 1500, 64, "fp16", 300, name="cross decoder step"),
        # a few learned queries that read a long input: few tiles, long keys
        _cross("cross", 1, 16, 4, 64, 16384, 128, name="cross latents"),
        # image patches over a prompt, one of the two prompts empty: memory
        _cross("cross", 2, 16, 16, 4096, 300, 128, lo=0, name="cross image patches"),
        # long on both sides: the tensor cores' rate
        _cross("cross", 1, 32, 8, 8192, 16384, 128, name="cross long"),
        # image patches on the way back: few keys, many queries
        _cross("cross_bwd", 2, 16, 16, 4096, 300, 128, lo=100, name="cross gradient image"),
        # an encoder-decoder's training step, ragged
        _cross("cross_bwd", 8, 16, 16, 500, 1500, 64, "fp16", 300, name="cross gradient decoder"),
        # long on both sides, shared key heads
        _cross("cross_bwd", 2, 16, 4, 4000, 6000, 128, name="cross gradient long"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_bwd", "cross_bwd", "rope", "rope_bwd"])
    Hkv, G = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4, 7])
    D = rng.choice([64, 64, 72, 80, 96, 128, 128, 128, 192, 200, 256])
    B = _log(rng, 1, 32)
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("rope", "rope_bwd"):
        S = _log(rng, 1, max(2, min(30000, (1 << 25) // (B * (G + 2) * Hkv * D))))
        axes = rng.choice([1, 1, 2, 3])
        R = rng.choice([D, D, D // 2, 32])
        return _rope(op, B, S, G * Hkv, Hkv, D, R, axes, rng.random() < 0.4, dtype, rng.choice(["same", "fp32", "none"]))
    rows = (1 << 25) // (B * Hkv * D)  # of q, and of k and v
    Sq = _log(rng, 1, max(2, min(20000, rows // G)))
    pairs = (1 << 30 if op == "cross" else 1 << 29) // (B * G * Hkv) * 128 // max(128, D)
    Sk = _log(rng, 1, max(2, min(30000, rows, pairs // Sq)))
    return _cross(op, B, G * Hkv, Hkv, Sq, Sk, D, dtype, rng.choice([None, rng.randint(0, Sk)]))


def _lens(c):
    """The sequences' lengths: spread from Sk down to lo, which the last has."""
    n = [c["Sk"] - int((c["Sk"] - c["lo"]) * ((i * 0.6180339887) % 1.0)) for i in range(c["B"])]
    if c["B"] > 1:
        n[-1] = c["lo"]
    return n


def work(c):
    B, Hq, Hkv, D = (c[k] for k in ("B", "Hq", "Hkv", "D"))
    if c["op"] in ("rope", "rope_bwd"):
        n, turned = B * c["S"] * D, Hq + Hkv
        if c["op"] == "rope":
            return {"bytes": 4 * n * (turned + Hkv) + 4 * B * c["S"] * c["axes"], "flops": 8 * n * turned}
        reads = turned if c["weight"] != "none" else 0
        return {"bytes": 4 * n * (turned + Hkv) + 2 * n * reads + 4 * B * c["S"] * c["axes"], "flops": 16 * n * turned}
    keys, rows = sum(_lens(c)), B * Hq * c["Sq"]
    if c["op"] == "cross":
        return {"bytes": 4 * rows * D + 4 * Hkv * D * keys + 4 * rows, "flops": 4 * D * Hq * c["Sq"] * keys}
    return {"bytes": 8 * rows * D + 4 * Hkv * D * (keys + B * c["Sk"]) + 8 * rows, "flops": 10 * D * Hq * c["Sq"] * keys}


# ------------------------------------------------------------------ the inputs
def _dtype(c):
    return torch.float16 if c["dtype"] == "fp16" else torch.bfloat16


def _plan(c):
    """inv_freq and axis of each pair: R/2 pairs dealt to the axes, the last ones taking one more, each axis with
    its own falling frequencies."""
    freq, axis, pairs, left = [], [], c["R"] // 2, c["axes"]
    for a in range(c["axes"]):
        n = (pairs - len(freq)) // left
        left -= 1
        freq += [10000.0 ** (-i / n) for i in range(n)]
        axis += [a] * n
    return torch.tensor(freq, dtype=torch.float64), torch.tensor(axis, dtype=torch.uint8)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    dt, s = _dtype(c), dict(case=c)
    B, Hq, Hkv, D = (c[k] for k in ("B", "Hq", "Hkv", "D"))
    if c["op"] in ("rope", "rope_bwd"):
        S, A = c["S"], c["axes"]
        s["x"] = torch.randn(B, S, (Hq + 2 * Hkv) * D, **dev).mul(1.5).to(dt)
        s["inv_freq"], s["axis"] = _plan(c)
        # a sequence's tokens follow one another from somewhere on; further axes wrap, as rows and columns of frames do
        first = torch.randint(0, 30000, (B, 1, 1), **dev)
        at = first * (torch.arange(A, device="cuda") == 0) + torch.arange(S, device="cuda")[None, :, None]
        s["positions"] = torch.stack([at[:, :, a] if a == 0 else at[:, :, a] // (53 if a == 1 else 1) % (30 + 23 * (a - 1))
                                      for a in range(A)], dim=2).int().contiguous()
        if c["weight"] != "none":
            wt = torch.float32 if c["weight"] == "fp32" else dt
            s["wq"], s["wk"] = (torch.randn(D, **dev).mul(0.1).add(1.0).to(wt) for _ in "qk")
        if c["op"] == "rope_bwd":
            for name, H in (("dq", Hq), ("dk", Hkv), ("dv", Hkv)):
                s[name] = torch.randn(B, H, S, D, **dev).to(dt)
        return s
    s["q"] = torch.randn(B, Hq, c["Sq"], D, **dev).mul(1.5).to(dt)
    s["k"], s["v"] = (torch.randn(B, Hkv, c["Sk"], D, **dev).to(dt) for _ in "kv")
    lens = _lens(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if min(lens) < c["Sk"] else None
    if c["op"] == "cross_bwd":
        r = _plain_cross(s)
        s["out"], s["lse"] = r["out"], r["lse"]
        s["dout"] = torch.randn(B, Hq, c["Sq"], D, **dev).to(dt)
    return s


# ------------------------------------------------------------------ the plain forms
def _scores(s):
    """scale·q·kᵀ [B, Hkv, G·Sq, Sk] and which keys are there (None: all)."""
    c = s["case"]
    B, Hkv, D, Sk = c["B"], c["Hkv"], c["D"], c["Sk"]
    q = s["q"].float().view(B, Hkv, -1, D)
    t = torch.matmul(q, s["k"].float().transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    if s["lens"] is None:
        return q, t, None
    return q, t, torch.arange(Sk, device="cuda")[None, None, None] < s["lens"][:, None, None, None]


def _values(s, name, there):
    """k or v in 32 bits; what lies behind a sequence's end counts as zero."""
    x = s[name].float()
    return x if there is None else torch.where(there.transpose(2, 3), x, 0.0)


def _plain_cross(s):
    _, t, there = _scores(s)
    if there is not None:
        t = t.masked_fill_(~there, -math.inf)
    m = t.amax(dim=3, keepdim=True).clamp(min=-3e38)
    p = t.sub_(m).exp_()
    l = p.sum(dim=3, keepdim=True)
    out = torch.matmul(p, _values(s, "v", there)) / l.clamp(min=1e-38)
    return {"out": out.view(s["q"].shape).to(s["q"].dtype), "lse": (m + torch.log(l)).view(s["q"].shape[:3])}


def _plain_cross_bwd(s):
    c, dt = s["case"], s["q"].dtype
    scale = 1.0 / math.sqrt(c["D"])
    q, t, there = _scores(s)
    p = t.sub_(s["lse"].view(*t.shape[:3], 1)).exp_()
    if there is not None:
        p = p.masked_fill_(~there, 0.0)
    dout = s["dout"].float().view(q.shape)
    delta = (dout * s["out"].float().view(q.shape)).sum(dim=3, keepdim=True)
    dv = torch.matmul(p.transpose(2, 3), dout)
    ds = torch.matmul(dout, _values(s, "v", there).transpose(2, 3)).sub_(delta).mul_(p)
    dq = torch.matmul(ds, _values(s, "k", there)) * scale
    dk = torch.matmul(ds.transpose(2, 3), q) * scale
    return {"dq": dq.view(s["q"].shape).to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "delta": delta.view(s["q"].shape[:3])}


def _heads(s, x):
    """q, k and v [B, S, H, D] of a packed projection."""
    c = s["case"]
    return x.view(c["B"], c["S"], -1, c["D"]).split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)


def _turns(s):
    """cos and sin [B, S, 1, R/2] in 32 bits of angles in 64."""
    at = s["positions"].double()[:, :, s["axis"].long().cuda()] * s["inv_freq"].cuda()
    return torch.cos(at).float()[:, :, None], torch.sin(at).float()[:, :, None]


def _turned(s, z, cos, sin):
    c = s["case"]
    R = c["R"]
    a, b = (z[..., 0:R:2], z[..., 1:R:2]) if c["interleaved"] else (z[..., :R // 2], z[..., R // 2:R])
    x, y = a * cos - b * sin, a * sin + b * cos
    pair = torch.stack([x, y], dim=-1).flatten(-2) if c["interleaved"] else torch.cat([x, y], dim=-1)
    return torch.cat([pair, z[..., R:]], dim=-1)


def _plain_rope(s):
    dt, (cos, sin) = s["x"].dtype, _turns(s)
    q, k, v = _heads(s, s["x"])
    r = {"v": v.transpose(1, 2).contiguous()}
    for name, x in (("q", q), ("k", k)):
        z = x.float()
        if "wq" in s:
            z = z * torch.rsqrt((z * z).mean(dim=3, keepdim=True) + EPS) * s["w" + name].float()
        r[name] = _turned(s, z, cos, sin).transpose(1, 2).to(dt).contiguous()
    return r


def _plain_rope_bwd(s):
    dt, (cos, sin) = s["x"].dtype, _turns(s)
    dx = torch.empty_like(s["x"])
    to, r = _heads(s, dx), {"dx": dx}
    to[2].copy_(s["dv"].transpose(1, 2))
    for i, name in enumerate("qk"):
        dz = _turned(s, s["d" + name].float().transpose(1, 2), cos, -sin)
        if "wq" in s:
            x = _heads(s, s["x"])[i].float()
            f = torch.rsqrt((x * x).mean(dim=3, keepdim=True) + EPS)
            x = x * f
            w = s["w" + name]
            r["dw" + name] = (dz * x).sum(dim=(0, 1, 2)).to(w.dtype)
            dz = dz * w.float()
            dz = (dz - x * (dz * x).mean(dim=3, keepdim=True)) * f
        to[i].copy_(dz.to(dt))
    return r


def run(s):
    op = s["case"]["op"]
    if own and op == "cross":
        from exact_attention_68_gb300 import cross
        out, lse = cross.cross_fwd(s["q"], s["k"], s["v"], s["lens"])
        return {"out": out, "lse": lse}
    if own and op == "cross_bwd":
        from exact_attention_68_gb300 import cross
        dq, dk, dv, delta = cross.cross_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["lens"])
        return {"dq": dq, "dk": dk, "dv": dv, "delta": delta}
    if own:
        from exact_attention_68_gb300 import rope
        plan = rope.Rope(s["inv_freq"], s["axis"], s["case"]["interleaved"])
        weights = (s.get("wq"), s.get("wk"), None)
        xs = _heads(s, s["x"])
        if op == "rope":
            q, k, v = rope.rope_fwd(xs, plan, s["positions"], weights, EPS, turn=(True, True, False))
            return {"q": q, "k": k, "v": v}
        dx = torch.empty_like(s["x"])
        _, dw = rope.rope_bwd((s["dq"], s["dk"], s["dv"]), xs, plan, s["positions"], weights, EPS,
                              turn=(True, True, False), dxs=_heads(s, dx))
        return {"dx": dx} if dw[0] is None else {"dx": dx, "dwq": dw[0], "dwk": dw[1]}
    return {"cross": _plain_cross, "cross_bwd": _plain_cross_bwd, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd}[op](s)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_head(q, k, v, scale):
    """out and lse of one head's rows over its keys."""
    if not k.shape[0]:
        return torch.zeros_like(q), torch.full_like(q[:, 0], -math.inf)
    outs, lses = [], []
    for rows in q.split(max(1, (1 << 27) // k.shape[0])):
        t = (rows @ k.T) * scale
        z = torch.logsumexp(t, dim=1)
        outs.append(torch.softmax(t, dim=1) @ v)
        lses.append(z)
    return torch.cat(outs), torch.cat(lses)


def _exact_head_bwd(q, k, v, out, lse, dout, scale):
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    delta = torch.einsum("id,id->i", dout, out)
    step = max(1, (1 << 27) // max(1, k.shape[0]))
    for i in range(0, q.shape[0] if k.shape[0] else 0, step):
        at = slice(i, i + step)
        p = torch.exp(scale * (q[at] @ k.T) - lse[at, None])
        ds = p * (dout[at] @ v.T - delta[at, None])
        dq[at] = scale * (ds @ k)
        dk += scale * (ds.T @ q[at])
        dv += p.T @ dout[at]
    return dq, dk, dv, delta


def _exact_turn(x, positions, freq, axis, interleaved, back):
    """The rotation of rows x [B, S, H, D], pair by pair, in place."""
    n = freq.numel()
    for i in range(n):
        a = positions[:, :, int(axis[i])].double() * float(freq[i])
        a = (-a if back else a)[:, :, None]
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        z = torch.complex(x[..., u], x[..., w]) * torch.polar(torch.ones_like(a), a)
        x[..., u], x[..., w] = z.real, z.imag
    return x


def _exact_rope(s):
    c = s["case"]
    B, S, D, H = c["B"], c["S"], c["D"], (c["Hq"], c["Hkv"], c["Hkv"])
    turn = (s["positions"], s["inv_freq"], s["axis"], c["interleaved"])
    x = s["x"].double().view(B, S, sum(H), D)
    parts = {"q": x[:, :, :H[0]], "k": x[:, :, H[0]:H[0] + H[1]], "v": x[:, :, H[0] + H[1]:]}
    norm = {n: 1.0 / (parts[n].square().sum(-1, keepdim=True) / D + EPS).sqrt() for n in "qk"}
    if c["op"] == "rope":
        r = {"v": parts["v"]}
        for n in "qk":
            z = parts[n] * norm[n] * s["w" + n].double() if "wq" in s else parts[n].clone()
            r[n] = _exact_turn(z, *turn, False)
        return {n: r[n].permute(0, 2, 1, 3) for n in ("v", "q", "k")}
    r, dx = {}, [None, None, s["dv"].double().permute(0, 2, 1, 3)]
    for i, n in enumerate("qk"):
        dz = _exact_turn(s["d" + n].double().permute(0, 2, 1, 3).clone(), *turn, True)
        if "wq" in s:
            unit = parts[n] * norm[n]
            r["dw" + n] = torch.einsum("bshd,bshd->d", dz, unit)
            g = dz * s["w" + n].double()
            dz = norm[n] * (g - unit * torch.einsum("bshd,bshd->bsh", g, unit)[..., None] / D)
        dx[i] = dz
    return {"dx": torch.cat(dx, dim=2).reshape(s["x"].shape), **r}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("rope", "rope_bwd"):
        return _exact_rope(s)
    if work(c)["flops"] > 1e13:
        return None
    B, Hkv, Sk, D, scale = c["B"], c["Hkv"], c["Sk"], c["D"], 1.0 / math.sqrt(c["D"])
    lens, rows = _lens(c), c["Hq"] // c["Hkv"] * c["Sq"]
    names = ("dq", "dk", "dv", "delta") if c["op"] == "cross_bwd" else ("out", "lse")
    got = {n: [] for n in names}
    of = lambda n, b, h: s[n].view(B, Hkv, rows, -1)[b, h].double()  # noqa: E731
    for b in range(B):
        for h in range(Hkv):
            k, v = (s[n][b, h, :lens[b]].double() for n in "kv")
            if c["op"] == "cross":
                r = _exact_head(of("q", b, h), k, v, scale)
            else:
                r = list(_exact_head_bwd(of("q", b, h), k, v, of("out", b, h), of("lse", b, h)[:, 0], of("dout", b, h), scale))
                for i in (1, 2):  # keys behind the sequence's end have no gradient
                    r[i] = torch.cat([r[i], r[i].new_zeros(Sk - lens[b], D)])
            for n, x in zip(names, r):
                got[n].append(x)
    shape = {"dk": s["k"].shape, "dv": s["v"].shape, "lse": s["q"].shape[:3], "delta": s["q"].shape[:3]}
    return {n: torch.cat(x).reshape(shape.get(n, s["q"].shape)) for n, x in got.items()}
