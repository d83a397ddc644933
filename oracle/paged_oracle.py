"""Plain fp64 oracle of the paged-cache operators, straight from their definitions.

A request is (keys [n, Hkv, D], values [n, Hkv, D]) in slot order; row i of r rows sits at
slot n - r + i and sees slot j iff 0 <= j <= p and (no window, or j > p - window, or
j < n_sink).  Nothing is shared with the CUDA path.
"""
import numpy as np


def visible(n, r, window, n_sink):
    """Boolean [r, n]: which slots each of the last r rows sees."""
    p = (n - r + np.arange(r))[:, None]
    j = np.arange(n)[None, :]
    see = j <= p
    if window:
        see = see & ((j > p - window) | (j < n_sink))
    return see


def attention(q, k, v, window, n_sink, scale):
    """q [r, Hq, D]; returns out [r, Hq, D], lse [r, Hq], and two sizes the tolerances are made
    of: spread [r, Hq, D] = sum_j p_j |v_j|, and size [r, Hq] = max_j scale |q|.|k_j|."""
    r, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    see = visible(n, r, window, n_sink)
    out, spread = np.zeros((r, hq, d)), np.zeros((r, hq, d))
    lse, size = np.full((r, hq), -np.inf), np.zeros((r, hq))
    for h in range(hq):
        g = h // (hq // hkv)
        for i in range(r):
            js = np.nonzero(see[i])[0]
            if len(js) == 0:
                continue
            kk, vv = k[js, g], v[js, g]
            s = scale * (kk @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[i, h], lse[i, h] = p @ vv, m + np.log(e.sum())
            with np.errstate(invalid="ignore"):
                spread[i, h] = p @ np.abs(vv)
                size[i, h] = (scale * (np.abs(kk) @ np.abs(q[i, h]))).max()
    return out, lse, spread, size


def weights(q, k, lse, used, window, n_sink, scale):
    """Attention weight each slot gets from the first `used` rows, summed over heads [n]."""
    r, hq, _ = q.shape
    n, hkv = k.shape[0], k.shape[1]
    see = visible(n, r, window, n_sink)
    w = np.zeros(n)
    for h in range(hq):
        g = h // (hq // hkv)
        for i in range(min(max(used, 0), r)):
            js = np.nonzero(see[i])[0]
            w[js] += np.exp(scale * (k[js, g] @ q[i, h]) - lse[i, h])
    return w


def evict(score, n, budget, n_sink, n_recent):
    """Slots that stay, ascending."""
    if n <= budget:
        return list(range(n))
    middle = [(-(-np.inf if np.isnan(score[j]) else float(score[j])), j) for j in range(n_sink, n - n_recent)]
    best = [j for _, j in sorted(middle)[:budget - n_sink - n_recent]]
    return sorted(list(range(n_sink)) + best + list(range(n - n_recent, n)))
