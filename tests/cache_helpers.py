"""Paged caches, error bounds and oracle runs shared by the serving operators' tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache_oracle as co

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
# half a step of the type, relative to the value
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half a step of values below the normal range (fp16's steps stop shrinking at 2^-24)
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def f64(t):
    return t.detach().double().cpu().numpy()


def make_cache(lens_cap, heads, dim, page, dtype, seed, heads_first=False, fill=None, spare=2):
    """(k_cache, v_cache, block_table) with pages in a random order; ``fill``: the
    value of every slot (default: random)."""
    g = torch.Generator().manual_seed(seed)
    batch = len(lens_cap)
    per = max(1, max(-(-n // page) for n in lens_cap))
    pages = batch * per + spare
    shape = (pages, heads, page, dim) if heads_first else (pages, page, heads, dim)
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g) if fill is None else torch.full(shape, float(fill))
        t = t.to(dtype).cuda()
        out.append(t.transpose(1, 2) if heads_first else t)
    table = torch.randperm(pages, generator=g)[:batch * per].view(batch, per).to(torch.int32).cuda()
    return out[0], out[1], table


def rows_of(cache, table, b, n):
    """Slots 0 .. n-1 of sequence b as a [n, H, D] tensor."""
    page = cache.shape[1]
    j = torch.arange(n, device=cache.device)
    return cache[table[b].long()[j // page], j % page]


def put_rows(cache, table, b, rows, start=0):
    page = cache.shape[1]
    j = torch.arange(start, start + rows.shape[0], device=cache.device)
    cache[table[b].long()[j // page], j % page] = rows


def decode_bounds(ref, dim, dtype, softcap):
    """(abs bound of O [Hq, D], of LSE [Hq], relative bound of the weights [Hq]).

    A logit is a sum of `dim` exact products in fp32: at most dim * 2^-22 of the
    sum of magnitudes off (each partial sum may be truncated), plus the scaling's
    and the cap's roundings; a probability is off by that and the exponentials'
    2^-20 in all; O rounds each probability to the type once and itself once.
    """
    half = HALF_STEP[dtype]
    logit = dim * 2.0 ** -22 * ref["mag"] + softcap * 2.0 ** -20 + 2.0 ** -20 * (1 + ref["mag"])
    prob = 2 * logit + 2.0 ** -19
    o = half * np.abs(ref["o"]) + (half * 1.01 + prob)[:, None] * ref["absv"] + SMALLEST[dtype] * 2
    if dtype == torch.float16:  # probabilities below fp16's normal range: absolute steps
        o = o + 2.0 ** -24 * ref["vsum"]
    fin = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
    return o, logit + 2.0 ** -20 + np.abs(fin) * 2.0 ** -22, prob


def check_decode(o, lse, q, kc, vc, table, lens, scale, window=-1, softcap=0.0, weights=None,
                 weights_in=None, width=0):
    """Every sequence against the oracle; weights: the device's weights_out."""
    dtype, dim = q.dtype, q.shape[2]
    for b, n in enumerate(lens):
        k, v = f64(rows_of(kc, table, b, n)), f64(rows_of(vc, table, b, n))
        ref = co.decode(f64(q[b]), k, v, scale, window, softcap)
        g = q.shape[1] // kc.shape[2]
        first = max(0, n - 1 - window) if window >= 0 else 0
        ref["vsum"] = np.repeat(np.abs(v[first:]).sum(0), g, axis=0) if n else np.zeros_like(ref["o"])
        bo, bl, bp = decode_bounds(ref, dim, dtype, softcap)
        got = f64(o[b])
        assert np.isfinite(got).all(), f"sequence {b} (length {n}): not finite"
        off = np.abs(got - ref["o"]) - bo
        assert (off <= 0).all(), f"sequence {b} (length {n}): O is {off.max():.3e} beyond its bound"
        gl = f64(lse[b])
        if n == 0:
            assert np.isposinf(gl).all() and (got == 0).all()
        else:
            assert (np.abs(gl - ref["lse"]) <= bl).all(), \
                f"sequence {b}: LSE off by {np.abs(gl - ref['lse']).max():.3e}"
        if weights is not None:
            w, w0 = f64(weights[b]), f64(weights_in[b])
            want = w0.copy()
            want[:, :n] += ref["p"]
            bound = np.zeros_like(want)
            bound[:, :n] = ref["p"] * bp.reshape(-1, g).max(1)[:, None] + 2.0 ** -23 * (
                np.abs(want[:, :n]) + g * ref["p"]) + 2.0 ** -120
            assert (np.abs(w - want) <= bound).all(), f"sequence {b}: weights"
