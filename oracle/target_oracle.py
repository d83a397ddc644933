"""Plain 64-bit oracle of the target-side operators, straight from their definitions: page tables
and slot maps, the 4-bit form of keys and values, head norms with rotation, log probabilities.
Nothing is shared with the CUDA path.
"""
import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every e4m3 number without its sign, the two of the all-ones exponent and fraction (NaN) left out
E4M3 = np.array([(f / 8 * 2.0 ** -6) if e == 0 else (1 + f / 8) * 2.0 ** (e - 7) for e in range(16) for f in range(8)][:127])


def nearest(table, x):
    """Index of the entry nearest to each x (ascending table), of two as near the even one; the last beyond it."""
    out = np.zeros(x.shape, dtype=np.int64)
    for i in range(1, len(table)):
        mid = (table[i - 1] + table[i]) / 2
        out = np.where((x > mid) | ((x == mid) & (i % 2 == 0)), i, out)
    return out


def encode4(x, exp=0):
    """x [..., D] -> codes uint8 [..., D/2], scales uint8 [..., D/16]."""
    x = np.asarray(x, dtype=np.float64) * 2.0 ** -exp
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    fine = np.isfinite(g).all(-1, keepdims=True)
    g = np.where(fine, g, 0.0)
    scale = nearest(E4M3 * 6, np.abs(g).max(-1))
    s = E4M3[scale][..., None]
    code = np.zeros(g.shape, dtype=np.int64)
    for i in range(1, 8):
        mid = (GRID[i - 1] + GRID[i]) / 2 * s
        code = np.where((np.abs(g) > mid) | ((np.abs(g) == mid) & (i % 2 == 0)), i, code)
    code = np.where(s > 0, code + 8 * np.signbit(g), 0).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.astype(np.uint8)


def decode4(codes, scales, exp=0):
    code = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    return v * np.repeat(E4M3[scales], 16, -1) * 2.0 ** exp


def plan(length, n_new, held, table, free, page_size, n_rows, give_back):
    """A step's tables, request by request; free: the free page ids, the top last.  Returns a dict."""
    B, width = table.shape
    table, stack, held = table.copy(), list(free), list(held)
    fine, start = [], [0]
    for b in range(B):
        end = start[-1] + max(0, n_new[b])
        n = length[b] + n_new[b]
        fine.append(length[b] >= 0 and n_new[b] >= 0 and 0 <= held[b] <= width and n <= width * page_size
                    and length[b] <= held[b] * page_size and end <= n_rows)
        start.append(end)
    need = [-(-(length[b] + n_new[b]) // page_size) if fine[b] else 0 for b in range(B)]
    before = list(held)
    for b in range(B):
        if fine[b] and give_back and need[b] < held[b]:
            stack += table[b, need[b]:held[b]].tolist()
            held[b] = need[b]
    top, promised, served = len(stack), 0, []
    for b in range(B):
        more = max(0, need[b] - before[b]) if fine[b] else 0
        promised += more
        served.append(fine[b] and (more == 0 or promised <= top))
        if served[b] and more:
            for x in range(more):
                table[b, before[b] + x] = stack.pop()
            held[b] = need[b]
    pos, slot, req = np.full(n_rows, -1), np.full(n_rows, -1, np.int64), np.full(n_rows, -1)
    for b in range(B):
        for i in range(max(0, n_new[b])):
            r = start[b] + i
            if r >= n_rows:
                break
            req[r] = b
            if served[b]:
                j = length[b] + i
                pos[r], slot[r] = j, int(table[b, j // page_size]) * page_size + j % page_size
    return dict(seq_len=[length[b] + n_new[b] if served[b] else 0 for b in range(B)], row_start=[min(s, n_rows) for s in start], request=req,
                pos=pos, slot=slot, table=table, held=held, free=stack, short=B - sum(served))


def head_norm_rope(x, gain, eps, inv_freq, pos, interleaved):
    """x [rows, heads, D]; inv_freq [pairs] radians a position; angles reduced in Python's own precision."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if gain is None else np.asarray(gain, dtype=np.float64))
    half = len(inv_freq)
    if half == 0:
        return y
    angle = np.array([[math.remainder(float(p) * f, 2 * math.pi) for f in inv_freq] for p in pos])[:, None]
    c, s, out = np.cos(angle), np.sin(angle), y.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    return out


def token_logprobs(logits, tokens, temperature, k):
    """One row: (log probabilities of tokens, entropy, lse, ids of the k largest, their log probabilities)."""
    x = np.asarray(logits, dtype=np.float64)
    order = sorted(range(len(x)), key=lambda i: (-(-np.inf if np.isnan(x[i]) else x[i]), i))[:k]
    z = x / temperature
    if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        lse = -np.inf if (z == -np.inf).all() else np.nan
        return [0.0 if t == -1 else np.nan for t in tokens], np.nan, lse, order, [np.nan] * k
    m = z.max()
    e = np.exp(z - m)
    lse = m + np.log(e.sum())
    p = e / e.sum()
    lp = z - lse
    return [0.0 if t == -1 else lp[t] for t in tokens], -(p[p > 0] * lp[p > 0]).sum(), lse, order, [lp[i] for i in order]
