"""The serving operators in 64 bits, slot by slot: rotary positions, the paged
cache's append, attention of one new token and eviction by attention weight.

Test infrastructure only.  Everything is a plain loop over the definition in
include/attn_cache.h; inputs are NumPy arrays (fp16/bf16 values given as float64).
"""
from __future__ import annotations

import numpy as np


def axis_of(sections):
    """Axis of each frequency."""
    return np.repeat(np.arange(len(sections)), sections)


def rope(x, positions, inv_freq, sections, interleaved=False, inverse=False):
    """x [T, H, D]; positions [axes, T] integers; inv_freq float32 values."""
    x = np.asarray(x, np.float64).copy()
    n = len(inv_freq)
    ax = axis_of(sections)
    angle = np.asarray(positions, np.float64)[ax].T * np.asarray(inv_freq, np.float64)  # [T, n]
    if inverse:
        angle = -angle
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - v * s
    x[..., b] = u * s + v * c
    return x


def slot(table_row, page_size, j):
    return int(table_row[j // page_size]), j % page_size


def append_slots(cu, seqlens, tokens):
    """(sequence, slot, i) of each token, None behind the last sequence."""
    out = [None] * tokens
    for b in range(len(seqlens)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            out[t] = (b, int(seqlens[b]) + t - int(cu[b]), t - int(cu[b]))
    return out


def decode(q, k, v, scale, window_left=-1, softcap=0.0):
    """One sequence: q [Hq, D], k, v [n, Hk, D] (its slots in order).

    Returns a dict: o [Hq, D], lse [Hq], p [Hk, n] (the group's summed weights), and for
    error bounds absv = sum_j p_j |v_j| [Hq, D] and mag = max_j scale sum_d |q_d k_jd| [Hq].
    """
    hq, d = q.shape
    n, hk = k.shape[0], k.shape[1]
    r = {"o": np.zeros((hq, d)), "lse": np.full(hq, np.inf), "p": np.zeros((hk, n)),
         "absv": np.zeros((hq, d)), "mag": np.zeros(hq)}
    first = max(0, n - 1 - window_left) if window_left >= 0 else 0
    if n == 0:
        return r
    for h in range(hq):
        g = h // (hq // hk)
        s = scale * (k[first:, g] @ q[h])
        r["mag"][h] = abs(scale) * np.max(np.abs(k[first:, g]) @ np.abs(q[h]))
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        r["lse"][h] = m + np.log(e.sum())
        r["o"][h] = p @ v[first:, g]
        r["absv"][h] = p @ np.abs(v[first:, g])
        r["p"][g, first:] += p
    return r


def keep(weights, positions, seen, budget, recent):
    """Slots kept of one (sequence, head): its n weights and positions; ascending."""
    n = len(weights)
    if n <= budget:
        return list(range(n))

    def rank(j):
        if recent > 0 and positions[j] >= seen - recent:
            return (1, np.inf)
        return (0, 0.0) if np.isnan(weights[j]) else (1, weights[j])

    # largest rank first, equal ranks by the lower slot
    order = sorted(range(n), key=lambda j: (-rank(j)[0], -rank(j)[1], j))
    return sorted(order[:budget])


def moves(kept, budget):
    """(from, to): the i-th kept slot at or above the budget goes to the i-th freed one."""
    low = set(j for j in kept if j < budget)
    free = [j for j in range(budget) if j not in low]
    return list(zip([j for j in kept if j >= budget], free))
