"""Plain fp64 CPU oracle of the 8-bit key/value cache and the operators on it.

TEST INFRASTRUCTURE, like the rest of this package: it restates the definitions
(page scales, e4m3 rounding, masked softmax over the pages, page scores,
eviction) with numpy, one page, row or token at a time, and shares no code with
the library.  A cache is a dict of numpy arrays: k, v uint8 [pages, heads, page,
pitch], k_scale, v_scale float32 [pages, heads], k_bounds int8 [pages, heads, 2,
pitch], and head_dim.
"""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_values", "e4m3_codes", "page_scale", "code_bounds", "cache_append", "cache_attention",
           "cache_select", "cache_evict"]


def e4m3_values() -> np.ndarray:
    """The 256 e4m3 values: sign, 4 exponent bits (bias 7), 3 fraction bits, NaN at S.1111.111."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            x = np.nan
        out[c] = -x if c & 128 else x
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # 0 .. 448, ascending; the index is the code


def e4m3_codes(x) -> np.ndarray:
    """Nearest e4m3 code (ties to the even code), saturating; NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.minimum(np.searchsorted(_POSITIVE, a), 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0))
    return code.astype(np.uint8)


def page_scale(x) -> float:
    """2^e, e the smallest integer >= -100 with |x| <= 448·2^e for the finite x."""
    x = np.abs(np.asarray(x, np.float64))
    x = x[np.isfinite(x)]
    a = x.max() if x.size else 0.0
    e = -100
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def code_bounds(codes) -> np.ndarray:
    """int8 [2, channels]: upper and lower bound of codes [tokens, channels] in steps of 448/127."""
    v = _VALUES[codes]
    out = np.zeros((2, codes.shape[1]), np.int8)
    for d in range(codes.shape[1]):
        w = v[~np.isnan(v[:, d]), d]
        if w.size:
            out[0, d] = np.ceil(w.max() * 127 / 448)
            out[1, d] = np.floor(w.min() * 127 / 448)
    return out


def cache_append(cache, table, lens, fresh, k, v) -> None:
    """In place.  k, v float [batch, heads, T, head_dim]; fresh [batch]."""
    P, D = cache["k"].shape[2], cache["head_dim"]
    pitch = cache["k"].shape[3]
    for b in range(len(lens)):
        start = lens[b] - fresh[b]
        for i in range(start // P, -(-lens[b] // P) if fresh[b] else 0):
            g, u, w = table[b, i], max(i * P, start), min((i + 1) * P, lens[b])
            held = u - i * P
            for h in range(cache["k"].shape[1]):
                for name, src in (("k", k), ("v", v)):
                    x = np.zeros((w - u, pitch))
                    x[:, :D] = src[b, h, u - start:w - start]
                    s = page_scale(x)
                    page = cache[name][g, h]
                    if held:
                        was = float(cache[name + "_scale"][g, h])
                        s = max(s, was)
                        if s != was:
                            page[:held] = e4m3_codes(_VALUES[page[:held]] * (was / s))
                    page[held:held + w - u] = e4m3_codes(x / s)
                    cache[name + "_scale"][g, h] = s
                    if name != "k":
                        continue
                    if held and s == was:  # bounds are widened, by channels that have a code to widen by
                        new, at = code_bounds(page[held:held + w - u]), cache["k_bounds"][g, h]
                        some = ~np.isnan(_VALUES[page[held:held + w - u]]).all(0)
                        at[0] = np.where(some, np.maximum(at[0], new[0]), at[0])
                        at[1] = np.where(some, np.minimum(at[1], new[1]), at[1])
                    else:
                        cache["k_bounds"][g, h] = code_bounds(page[:held + w - u])


def _held(cache, name, g, h):
    return _VALUES[cache[name][g, h]][:, :cache["head_dim"]] * float(cache[name + "_scale"][g, h])


def cache_attention(cache, table, lens, fresh, q, scale, pages=None):
    """q float [batch, q_heads, T, head_dim]; pages int [batch, heads, n] or None.

    Returns out and lse float64 (rows of tokens from fresh[b] on are NaN), the
    keys' weights mass [batch, heads, width·page], and for error bounds absv
    (Σ weight·|v|, like out) and absqk (the largest scale·Σ|q·k| of a row, like lse).
    """
    B, Hq, T, D = q.shape
    H, P = cache["k"].shape[1], cache["k"].shape[2]
    G = Hq // H
    out, absv = np.full((B, Hq, T, D), np.nan), np.zeros((B, Hq, T, D))
    lse, absqk = np.full((B, Hq, T), np.nan), np.zeros((B, Hq, T))
    mass = np.zeros((B, H, table.shape[1] * P))
    for b in range(B):
        for h in range(H):
            which = range(-(-lens[b] // P)) if pages is None else [i for i in pages[b, h] if 0 <= i * P < lens[b]]
            k = np.concatenate([_held(cache, "k", table[b, i], h) for i in which] or [np.zeros((0, D))])
            v = np.concatenate([_held(cache, "v", table[b, i], h) for i in which] or [np.zeros((0, D))])
            pos = np.concatenate([np.arange(i * P, i * P + P) for i in which] or [np.zeros(0, int)]).astype(int)
            for hq in range(h * G, h * G + G):
                for i in range(fresh[b]):
                    see = pos <= lens[b] - fresh[b] + i
                    out[b, hq, i], lse[b, hq, i] = 0.0, -np.inf
                    if not see.any():
                        continue
                    qi = q[b, hq, i].astype(np.float64)
                    t = scale * (k[see] @ qi)
                    absqk[b, hq, i] = scale * (np.abs(k[see]) @ np.abs(qi)).max()
                    m = t.max()
                    e = np.exp(t - m)
                    p = e / e.sum()
                    out[b, hq, i], absv[b, hq, i] = p @ v[see], p @ np.abs(v[see])
                    lse[b, hq, i] = m + np.log(e.sum())
                    mass[b, h, pos[see]] += p
    return out, lse, mass, absv, absqk


def cache_select(cache, table, lens, fresh, q, count):
    """(pages int32 [batch, heads, count], scores float32 [batch, heads, width])."""
    B, Hq, T, D = q.shape
    H, P = cache["k"].shape[1], cache["k"].shape[2]
    G, f = Hq // H, np.float32
    pages = np.full((B, H, count), -1, np.int32)
    scores = np.full((B, H, table.shape[1]), -np.inf, np.float32)
    for b in range(B):
        n = -(-lens[b] // P)
        if fresh[b] == 0:
            continue
        first = (lens[b] - fresh[b]) // P
        for h in range(H):
            for hq in range(h * G, h * G + G):
                for i in range(fresh[b]):
                    x = q[b, hq, i].astype(f)
                    a = f(np.abs(np.where(np.isfinite(x), x, 0)).max())
                    with np.errstate(invalid="ignore", over="ignore"):
                        y = np.rint(x * (f(127) / a if a > 0 else f(0)))
                    qi = np.clip(np.where(np.isnan(y), 0, y), -127, 127).astype(np.int64)
                    for g in range(n):
                        w = cache["k_bounds"][table[b, g], h, :, :D].astype(np.int64)
                        s = int(np.maximum(qi * w[0], qi * w[1]).sum())
                        s = f(f(s) * f(cache["k_scale"][table[b, g], h])) * a
                        scores[b, h, g] = max(scores[b, h, g], s)
            new = list(range(first, n))[-count:]
            order = sorted(range(first), key=lambda g: (-scores[b, h, g], g))
            take = sorted(order[:count - len(new)] + new)
            pages[b, h, :len(take)] = take
    return pages, scores


def cache_evict(cache, mass, table, lens, dst_table, keep, recent):
    """In place on the cache; returns (kept, new_lens, new_mass)."""
    B, H, P = table.shape[0], cache["k"].shape[1], cache["k"].shape[2]
    kept = np.full((B, H, keep), -1, np.int32)
    moved = np.zeros((B, H, dst_table.shape[1] * P), np.float32)
    pitch, D = cache["k"].shape[3], cache["head_dim"]
    old = {n: cache[n].copy() for n in "kv"}
    old_scale = {n: cache[n + "_scale"].copy() for n in "kv"}
    for b in range(B):
        n = lens[b]
        for h in range(H):
            at = list(range(n))
            if n > keep:
                tail = min(recent, n)
                w = mass[b, h, :n - tail]
                best = sorted(range(n - tail), key=lambda j: (np.isnan(w[j]), 0.0 if np.isnan(w[j]) else -w[j], j))
                best = best[:keep - tail]
                at = sorted(best) + list(range(n - tail, n))
            kept[b, h, :len(at)] = at
            moved[b, h, :len(at)] = mass[b, h, at]
            for i in range(-(-len(at) // P)):
                g, part = dst_table[b, i], at[i * P:(i + 1) * P]
                for name in "kv":
                    x = np.zeros((len(part), pitch))
                    for r, j in enumerate(part):
                        src = table[b, j // P]
                        x[r, :D] = _VALUES[old[name][src, h, j % P, :D]] * float(old_scale[name][src, h])
                    s = page_scale(x)
                    cache[name][g, h, :len(part)] = e4m3_codes(x / s)
                    cache[name + "_scale"][g, h] = s
                    if name == "k":
                        cache["k_bounds"][g, h] = code_bounds(cache["k"][g, h, :len(part)])
    return kept, np.minimum(lens, keep).astype(np.int32), moved
