"""Caches in 8 bits, error bounds and oracle runs shared by their tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache_oracle as co
from tests.cache_helpers import HALF_STEP, SMALLEST, f64

KIND = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def numbers(codes):
    """Codes as the numbers they stand for, in 64 bits."""
    return codes.float().double().cpu().numpy()


def to_device(x, kind):
    """Codes (as numbers) in the cache's type; all of them are representable."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    return t.to(KIND[kind]).cuda()


def make_cache8(cap, batch, heads, dim, page, block, kind, seed, heads_first=False, spare=2, exps=(-7, -4)):
    """(k_cache, v_cache, k_scale, v_scale, block_table): random codes, factors 2^exps[0] .. 2^exps[1]
    at random, pages in a random order."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, -(-cap // page))
    pages = batch * per + spare
    shape = (pages, heads, page, dim) if heads_first else (pages, page, heads, dim)
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g)
        t = (t * 36).round().clamp(-127, 127) if kind == "int8" else (t * 100).clamp(-448, 448)
        t = t.to(KIND[kind]).cuda()
        out.append(t.transpose(1, 2) if heads_first else t)
    for _ in range(2):
        out.append(torch.exp2(torch.randint(exps[0], exps[1] + 1, (pages, page // block, heads), generator=g).float()).cuda())
    table = torch.randperm(pages, generator=g)[:batch * per].view(batch, per).to(torch.int32).cuda()
    return (*out, table)


def slots_of(cache, scale, table, b, j):
    """Values [len(j), H, D] in 64 bits of slots j of sequence b."""
    page = cache.shape[1]
    j = torch.as_tensor(list(j), dtype=torch.long, device=cache.device)
    rows, w = table[b].long()[j // page], j % page
    codes = cache.view(torch.uint8)[rows, w].view(cache.dtype).float().double()
    block = page // scale.shape[1]
    return (codes * scale[rows, w // block].double()[..., None]).cpu().numpy()


def check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, scale, window=-1, softcap=0.0, skip=()):
    """Every sequence against the oracle.

    A logit is a sum of D products in fp32 (each partial sum may be truncated: D 2^-22 of the sum
    of magnitudes), of q in bf16 also off by 2^-25 of the row's largest element times sum |k|, plus
    the scaling's and the cap's roundings.  A probability is off by twice that and the
    exponentials' 2^-20.  Weights enter O to 2^-22 of themselves or 2^-39 of the largest weight
    (p_j vs_j, within a factor of 2); sums over n keys take n / 64 + 16 steps of 2^-23; O is
    rounded once.
    """
    half, dim = HALF_STEP[q.dtype], q.shape[2]
    group = q.shape[1] // kc.shape[2]
    for b, n in enumerate(lens):
        if b in skip:
            continue
        got, gl = f64(o[b]), f64(lse[b])
        if n == 0:
            assert np.isposinf(gl).all() and (got == 0).all()
            continue
        k, v = (slots_of(c, s, table, b, range(n)) for c, s in ((kc, ks), (vc, vs)))
        x = f64(q[b])
        ref = co.decode(x, k, v, scale, window, softcap)
        first = max(0, n - 1 - window) if window >= 0 else 0
        logit = (dim + 4) * 2.0 ** -22 * ref["mag"] + softcap * 2.0 ** -20 + 2.0 ** -20
        if q.dtype == torch.bfloat16:
            most = np.abs(k[first:]).sum(2).max(0)  # [Hk]
            logit = logit + 2.0 ** -25 * abs(scale) * np.abs(x).max(1) * np.repeat(most, group)
        steps = (n / 64 + 16) * 2.0 ** -23
        prob = 2 * logit + 2.0 ** -19 + steps
        bound = half * np.abs(ref["o"]) + 2 * SMALLEST[q.dtype] + ref["absv"] * (prob + 2.0 ** -22)[:, None] * (1 + half)
        # the largest weight, and each column's codes: sum_j |v8_j| 2^-38 max_j (p_j vs_j)
        page, block = kc.shape[1], kc.shape[1] // vs.shape[1]
        j = torch.arange(first, n, device=kc.device)
        f = vs[table[b].long()[j // page], j % page // block].double().cpu().numpy()  # [n, Hk]
        for h in range(q.shape[1]):
            g = h // group
            s = scale * (k[first:, g] @ x[h])
            s = softcap * np.tanh(s / softcap) if softcap > 0 else s
            p = np.exp(s - ref["lse"][h])
            codes = np.abs(v[first:, g]) / np.where(f[:, g:g + 1] > 0, f[:, g:g + 1], 1.0)
            bound[h] += 2.0 ** -38 * (p * f[:, g]).max() * codes.sum(0)
        assert np.isfinite(got).all(), f"sequence {b} (length {n}): not finite"
        off = np.abs(got - ref["o"]) - bound
        assert (off <= 0).all(), f"sequence {b} (length {n}): O is {off.max():.3e} beyond its bound"
        bl = logit + 2.0 ** -20 + steps + np.abs(ref["lse"]) * 2.0 ** -22
        assert (np.abs(gl - ref["lse"]) <= bl).all(), f"sequence {b}: LSE off by {np.abs(gl - ref['lse']).max():.3e}"
