"""fp64 statement of the 8-bit cache operators and the attention over the
cache.  Test infrastructure: plain numpy, one sequence and one head at a
time, sharing no code with the library.

A cache here is dict(k, v: uint8 [pages, kv_heads, page, dim], k_scale,
v_scale: float64 [pages, kv_heads])."""
from __future__ import annotations

import math

import numpy as np


def _values() -> np.ndarray:
    """What each of the 256 codes stands for (sign, 4 exponent bits with bias
    7, 3 mantissa bits; all ones is NaN)."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if (c & 0x7f) == 0x7f else (-x if c & 0x80 else x)
    return t


VALUE = _values()
_POSITIVE = VALUE[:0x7f]  # ascending


def encode(x) -> np.ndarray:
    """Codes of the nearest values, ties to the even code; NaN -> 0, beyond
    448 -> 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    hi = np.searchsorted(_POSITIVE, a)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    c = np.where(take_lo, lo, hi).astype(np.uint8)
    return c | (np.signbit(np.where(np.isnan(x), 0.0, x)).astype(np.uint8) << 7)


def need(a: float) -> float:
    """The smallest power of two s >= 2^-100 with a <= 448 s."""
    s = 2.0 ** -100
    while a > 448 * s:
        s *= 2
    return s


def _put(cache, name, table, page, ctx, x):
    """x [n, kv_heads, dim] becomes tokens ctx.. of the sequence with pages
    ``table``; returns whether something was not finite."""
    codes, scale = cache[name], cache[name + "_scale"]
    n, heads, _ = x.shape
    odd = False
    for g in range(ctx // page, -(-(ctx + n) // page)):
        lo, hi = max(ctx, g * page), min(ctx + n, (g + 1) * page)
        p = int(table[g])
        if not 0 <= p < codes.shape[0]:
            continue
        for h in range(heads):
            part = x[lo - ctx:hi - ctx, h].astype(np.float64)
            fine = np.isfinite(part)
            odd |= not fine.all()
            s = need(np.abs(part[fine]).max(initial=0.0))
            held = lo - g * page
            if held:
                old = scale[p, h]
                s = max(s, old)
                if s > old:
                    codes[p, h, :held] = encode(VALUE[codes[p, h, :held]] * (old / s))
            codes[p, h, lo - g * page:hi - g * page] = encode(part / s)
            scale[p, h] = s
    return odd


def append(cache, k, v, table, page, ctx) -> bool:
    """Append one sequence's k, v [n, kv_heads, dim]."""
    a = _put(cache, "k", table, page, ctx, k)
    return _put(cache, "v", table, page, ctx, v) or a


def read(cache, name, table, page, first, n) -> np.ndarray:
    """Tokens first.. of one sequence: [n, kv_heads, dim]; 0 on a bad page."""
    heads, dim = cache[name].shape[1], cache[name].shape[3]
    out = np.zeros((n, heads, dim))
    for t in range(n):
        p = int(table[(first + t) // page])
        if 0 <= p < cache[name].shape[0]:
            out[t] = VALUE[cache[name][p, :, (first + t) % page]] * cache[name + "_scale"][p][:, None]
    return out


def commit(cache, table, page, ctx, path) -> int:
    """The nodes ``path`` of the tree behind ctx become its next tokens;
    returns the new length."""
    kept = {n: np.concatenate([read(cache, n, table, page, ctx + p, 1) for p in path]) for n in ("k", "v")}
    append(cache, kept["k"], kept["v"], table, page, ctx)
    return ctx + len(path)


def visible(ctx: int, n: int, parents, window: int, sinks: int) -> np.ndarray:
    """[n, ctx + n] bool: which tokens each new token's query sees."""
    sees = np.zeros((n, ctx + n), bool)
    depth = [0] * n
    lines = []
    for i in range(n):
        p = (i - 1) if parents is None else int(parents[i])
        if not 0 <= p < i:
            p = -1
        lines.append((lines[p] if p >= 0 else []) + [i])
        depth[i] = len(lines[i]) - 1
    at = list(range(ctx)) + [ctx + d for d in depth]
    for i in range(n):
        for j in list(range(ctx)) + [ctx + t for t in lines[i]]:
            sees[i, j] = window == 0 or at[ctx + i] - at[j] < window or at[j] < sinks
    return sees


def attention(q, cache, table, page, ctx, parents, scale, window, sinks):
    """One sequence's attention: q [n, heads, dim] -> out [n, heads, dim],
    lse [n, heads], and for error bounds sum_j p_j |v_j| like out and the
    largest sum_d |q_d k_d| * scale of a visible score like lse."""
    n, heads, dim = q.shape
    length = ctx + n
    k, v = (read(cache, name, table, page, 0, length) for name in ("k", "v"))
    sees = visible(ctx, n, parents, window, sinks)
    on_page = np.array([0 <= int(table[j // page]) < cache["k"].shape[0] for j in range(length)], bool)
    sees &= on_page[None, :]
    group = heads // k.shape[1]
    out, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    absolute, largest = np.zeros((n, heads, dim)), np.zeros((n, heads))
    for i in range(n):
        if not sees[i].any():
            continue
        for h in range(heads):
            kk, vv = k[sees[i], h // group], v[sees[i], h // group]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            lse[i, h] = m + math.log(e.sum())
            w = e / e.sum()
            out[i, h] = w @ vv
            absolute[i, h] = w @ np.abs(vv)
            largest[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absolute, largest
