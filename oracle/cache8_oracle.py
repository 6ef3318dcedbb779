"""The operators of a cache in 8 bits and of shared pages in 64 bits, entry by entry.

Test infrastructure only: plain loops over the definitions in include/attn_cache8.h.  Codes are
given as the numbers they stand for (a code of e4m3 as its value, of int8 as the integer).
"""
from __future__ import annotations

import math

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values():
    """The non-negative values of e4m3 in the order of their codes 0 .. 126."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    return np.array(sub + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119])


_E4M3 = e4m3_values()


def code(x, kind):
    """The nearest code of each number, ties to the even code; numbers beyond the largest become it."""
    x = np.clip(np.asarray(x, np.float64), -TOP[kind], TOP[kind])
    if kind == "int8":
        return np.rint(x) + 0.0
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, len(_E4M3) - 1)
    lo = hi - 1
    to_lo, to_hi = a - _E4M3[lo], _E4M3[hi] - a
    pick = np.where((to_hi < to_lo) | ((to_hi == to_lo) & (hi % 2 == 0)), hi, lo)
    return np.copysign(_E4M3[pick], x)


def factor(top, kind):
    """The smallest power of two s in [2^-60, 2^60] with top <= TOP s."""
    e = -60
    while e < 60 and top > TOP[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scales, table_row, page, old, x, kind):
    """Stores x [n, H, D] in slots old .. of a sequence; codes [pages, page, H, D] and scales
    [pages, blocks, H] are changed."""
    n, heads = x.shape[:2]
    block = page // scales.shape[1]
    j = old
    while j < old + n:
        base = j // block * block
        end = min(base + block, old + n)
        p, w = int(table_row[base // page]), base % page
        for h in range(heads):
            v = x[j - old:end - old, h]
            s = factor(np.abs(v).max(), kind)
            if j > base:
                was = scales[p, w // block, h]
                if s > was:
                    codes[p, w:w + j - base, h] = code(codes[p, w:w + j - base, h] * (was / s), kind)
                s = max(s, was)
            scales[p, w // block, h] = s
            codes[p, w + j - base:w + end - base, h] = code(v / s, kind)
        j = end


def values(codes, scales):
    """[pages, page, H, D] values of all slots."""
    block = codes.shape[1] // scales.shape[1]
    return codes * np.repeat(scales, block, axis=1)[..., None]


def fork(table, lens, refs, page, parents, room, share=True):
    """(table, lengths, refs, [(source, fresh page)], free pages, pages were missing)."""
    rows, width = table.shape
    refs = refs.copy()
    new = np.full_like(table, -1)
    heir, out_len, want, made, gone = {}, [0] * rows, [], [], []
    for b in range(rows):
        if parents[b] >= 0:
            heir.setdefault(int(parents[b]), b)
    for s in range(rows):
        if s not in heir:
            for e in table[s]:
                if e >= 0:
                    refs[e] -= 1
    for b in range(rows):
        s = int(parents[b])
        if s >= 0 and heir[s] != b and share:
            for e in table[s, :lens[s] // page]:
                refs[e] += 1
    for b in range(rows):
        s = int(parents[b])
        if s < 0:
            continue
        n = out_len[b] = int(lens[s])
        full, used, need = n // page, math.ceil(n / page), min(width, math.ceil((n + room[b]) / page))
        own = width if heir[s] == b else full if share else 0  # entries that are the parent's
        if heir[s] == b and any(e >= 0 and refs[e] > 1 for e in table[s, full:max(used, need)]):
            own = full  # others hold what this row would write
            gone += [e for e in table[s, full:] if e >= 0]
        for i in range(width):
            if i < own:
                new[b, i] = table[s, i]
            if i >= own and i < used:
                want.append((b, i, table[s, i]))
            elif i >= used and i < need and new[b, i] < 0:
                want.append((b, i, -1))
    free = [p for p in range(len(refs)) if refs[p] == 0]
    missing = len(want) > len(free)
    for (b, i, src), p in zip(want, free):
        new[b, i] = p
        refs[p] = 1
        if src >= 0:
            made.append((src, p))
    for e in gone:  # free from the next call on
        refs[e] -= 1
    return new, np.array(out_len), refs, made, int((refs == 0).sum()), missing
