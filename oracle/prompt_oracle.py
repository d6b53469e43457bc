"""A request's way into the cache in plain float64 numpy and Python: pages and
places, rotary positions, attention of a prompt.  One sequence, one page or
one head at a time; shares no code with the CUDA library."""
import math

import numpy as np

BAD_PARENT, BAD_PAGE, BAD_LENGTH, NO_PAGE = 2, 64, 128, 2048


def assign(free, count, table, held, ctx, page, counts, row0, total, max_new, parents=None):
    """Moves pages between ``free`` (a list, ``count`` of whose entries are the
    stack) and ``table`` / ``held`` (changed in place), for sequences with
    ctx[b] cached and counts[b] new tokens in the rows row0[b] ...  Returns
    (count, slots, positions, flags): slots and positions as dicts by row."""
    size, columns, batch = len(free), len(table[0]), len(held)
    flags = [0] * batch
    known = [row0[b] >= 0 and 0 <= counts[b] <= max_new and row0[b] + counts[b] <= total for b in range(batch)]
    good = [known[b] and ctx[b] >= 0 and ctx[b] + counts[b] <= columns * page and 0 <= held[b] <= columns for b in range(batch)]
    want = [math.ceil((ctx[b] + counts[b]) / page) if good[b] else held[b] for b in range(batch)]
    stack = list(free[:min(max(count, 0), size)])
    for b in reversed(range(batch)):
        for col in reversed(range(want[b], held[b])):
            stack.append(int(table[b][col]))
    free[:len(stack)] = stack[:size]
    stack = stack[:size]
    lacking = 0
    for b in range(batch):
        lack = max(0, want[b] - held[b])
        lacking += lack
        if not good[b]:
            flags[b] = BAD_LENGTH
        elif lack and len(stack) < lack or lack and NO_PAGE in flags:
            flags[b] = NO_PAGE
        else:
            for col in range(held[b], want[b]):
                table[b][col] = stack.pop()
            held[b] = want[b]
    slots, positions = {}, {}
    for b in range(batch):
        if not known[b]:
            continue
        depth = {}
        for i in range(counts[b]):
            r, j = row0[b] + i, ctx[b] + i
            if not good[b]:
                slots[r], positions[r] = -1, 0
                continue
            up = i - 1 if parents is None else int(parents[r])
            if parents is not None and (up != -1 if i == 0 else not 0 <= up < i):
                flags[b] |= BAD_PARENT
            depth[i] = depth[up] + 1 if 0 <= up < i else 0
            positions[r] = ctx[b] + depth[i]
            slots[r] = -1
            if flags[b] & NO_PAGE == 0:
                p = int(table[b][j // page])
                if 0 <= p < size:
                    slots[r] = p * page + j % page
                else:
                    flags[b] |= BAD_PAGE
    return len(stack), slots, positions, flags


def rope(x, positions, inv_freq, axis, adjacent):
    """x [rows, heads, dim], positions [axes, rows], inv_freq [pairs] as the
    float32 values they are, axis [pairs]: the turned x in float64, and the
    length sqrt(a^2 + b^2) of the pair that each value is of (0: stays)."""
    x = np.asarray(x, np.float64)
    out, size = x.copy(), np.zeros_like(x)
    half = len(inv_freq)
    for i in range(half):
        t = np.asarray(positions[axis[i]], np.longdouble) * np.longdouble(np.float32(inv_freq[i]))
        c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
        p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        a, b = x[:, :, p], x[:, :, q]
        out[:, :, p], out[:, :, q] = a * c - b * s, a * s + b * c
        size[:, :, p] = size[:, :, q] = np.hypot(a, b)
    return out, size


def sees(n, window, sinks):
    """[n, n] bool: which tokens each token's query sees."""
    i = np.arange(n)
    back = i[:, None] - i
    return (back >= 0) & ((window == 0) | (back < window) | (i < sinks)[None, :])


def attention(q, k, v, scale, window, sinks):
    """One sequence: q [n, heads, dim], k and v [n, kv_heads, dim] -> out,
    lse [n, heads], and for error bounds sum_j p_j |v_j| like out and the
    largest sum_d |q_d k_d| * scale of a visible score like lse.  What a query
    does not see is not touched."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, lse, absolute, largest = np.zeros((n, heads, dim)), np.zeros((n, heads)), np.zeros((n, heads, dim)), np.zeros((n, heads))
    visible = sees(n, window, sinks)
    for i in range(n):
        at = np.flatnonzero(visible[i])
        for h in range(heads):
            kk, vv = k[at, h // group], v[at, h // group]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            lse[i, h], out[i, h], absolute[i, h] = m + math.log(e.sum()), w @ vv, w @ np.abs(vv)
            largest[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absolute, largest
