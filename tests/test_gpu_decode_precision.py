"""attn_decode's weights in the product with V: their precision, small ones that make up the output
because the largest lies on a key of value zero (an attention sink), and infinite values."""
import math

import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache_oracle as co
from tests.cache_helpers import HALF_STEP, SMALLEST, decode_bounds, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [17.0, 24.9, 25.1, 30.0])
@pytest.mark.parametrize("d", [64, 80, 128, 192, 256])
def test_fp16_weights_far_below_the_largest_keep_their_share(d, bits):
    """One key, of value zero, lies `bits` powers of two above 16383 others; 300 sequences
    over the same pages, so that a block sees most of a sequence behind its sink.

    The bound: half a step of O's own rounding, half a step of each weight's, and for weights
    that are subnormal in fp16 half an absolute step, 2^-25 of a largest weight of 2^15, for
    each key: 2^-40 |v|.
    """
    n, page, batch, dt = 16384, 64, 300, torch.float16
    g = torch.Generator().manual_seed(50)
    pages = n // page
    k = torch.zeros(n, 1, d)
    v = 1.0 + 0.5 * torch.randn(n, 1, d, generator=g)
    k[:, 0, 1:] = 0.05 * torch.randn(n, d - 1, generator=g)
    k[5] = 0
    k[5, 0, 0], v[5] = bits * math.log(2.0), 0.0
    q = torch.randn(d, generator=g)
    q[0] = 8.0
    kc, vc = (x.to(dt).view(pages, page, 1, d).cuda() for x in (k, v))
    q1 = q.to(dt)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    o, lse = ab.attn_decode(q1.cuda().expand(batch, 1, d).contiguous(), kc, vc, table, lens, scale=0.125)
    ab.check_device_status()
    ref = co.decode(f64(q1)[None], f64(k.to(dt)), f64(v.to(dt)), 0.125)
    _, bl, prob = decode_bounds({**ref, "vsum": np.zeros((1, d))}, d, dt, 0.0)
    half = HALF_STEP[dt]
    bound = half * np.abs(ref["o"]) + (half * 1.01 + prob)[:, None] * ref["absv"] + \
        2.0 ** -40 * np.abs(f64(v.to(dt))).sum(0) + SMALLEST[dt]
    off = np.abs(f64(o) - ref["o"]) - bound
    assert (off <= 0).all(), f"O is {off.max():.3e} beyond its bound, at {np.abs(ref['o']).max():.3e}"
    assert (np.abs(f64(lse) - ref["lse"]) <= bl).all()


# of a weight that enters the product as a number of the type and its remainder in the type
WEIGHT = {torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}


@pytest.mark.parametrize("d", [8, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hk", [(8, 8), (16, 2), (18, 2), (32, 2), (40, 2)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_weights_are_more_precise_than_the_type(dt, hq, hk, d):
    """O within half a step of its own, the weights' error (two roundings to the type, the
    logits' and the exponential's) and the product's fp32 sums, 2^-22 of the magnitudes a key."""
    lens, page = [2, 3, 5, 9, 40, 300, 3000, 1], 16
    g = torch.Generator().manual_seed(60)
    per = -(-max(lens) // page)
    kc, vc = (torch.randn(len(lens) * per, page, hk, d, generator=g).to(dt) for _ in range(2))
    table = torch.randperm(len(lens) * per, generator=g).to(torch.int32).view(-1, per)
    q = torch.randn(len(lens), hq, d, generator=g).to(dt)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, _ = ab.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), n, scale=0.5 / d ** 0.5)
    ab.check_device_status()
    for b, m in enumerate(lens):
        rows = table[b].long()
        k, v = (f64(c[rows].flatten(0, 1)[:m]) for c in (kc, vc))
        ref = co.decode(f64(q[b]), k, v, 0.5 / d ** 0.5)
        _, _, prob = decode_bounds({**ref, "vsum": np.zeros((hq, d))}, d, dt, 0.0)
        bound = HALF_STEP[dt] * np.abs(ref["o"]) + (WEIGHT[dt] + m * 2.0 ** -22 + prob)[:, None] * ref["absv"] + \
            2.0 ** -39 * np.repeat(np.abs(v).sum(0), hq // hk, axis=0) + SMALLEST[dt]
        off = np.abs(f64(o[b]) - ref["o"]) - bound
        assert (off <= 0).all(), f"length {m}: O is {off.max():.3e} beyond its bound"


@pytest.mark.parametrize("hq", [2, 16, 20])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_infinite_values_stay_infinite(dt, hq):
    n, d, page = 500, 64, 16
    g = torch.Generator().manual_seed(61)
    k, v = (torch.randn(n // page + 1, page, 1, d, generator=g).to(dt) for _ in range(2))
    v.view(-1, d)[70, 3] = float("inf")
    v.view(-1, d)[300, 9] = -float("inf")
    table = torch.arange(n // page + 1, dtype=torch.int32)[None]
    o, _ = ab.attn_decode(torch.randn(1, hq, d, generator=g).to(dt).cuda(), k.cuda(), v.cuda(), table.cuda(),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), scale=0.05)
    assert torch.isposinf(o[0, :, 3]).all() and torch.isneginf(o[0, :, 9]).all()
    rest = [c for c in range(d) if c not in (3, 9)]
    assert o[0][:, rest].isfinite().all()


def test_the_longest_sequence():
    """2^31 - 8192 keys, nearly all of them on one page that the table names again and again: the
    weights lie on the first key and on the last."""
    n, page, d, dt = 2**31 - 8192, 4096, 8, torch.float16
    g = torch.Generator().manual_seed(62)
    kc = torch.full((3, page, 1, d), -6e4).to(dt).cuda()
    vc = torch.randn(3, page, 1, d, generator=g).to(dt).cuda()
    table = torch.zeros(2, 2**31 // page - 1, dtype=torch.int32, device="cuda")
    last = (n - 1) // page, (n - 1) % page
    table[0, 0], table[0, last[0]] = 1, 2
    kc[1, 0], kc[2, last[1]] = 0.25, 0.5
    kc[2, last[1] + 1:] = 6e4  # behind the last key
    q = torch.ones(2, 1, d, dtype=dt, device="cuda")
    lens = torch.tensor([n, 0], dtype=torch.int32, device="cuda")
    o, lse = ab.attn_decode(q, kc, vc, table, lens, max_seqlen=n, scale=1.0)
    ab.check_device_status()
    k = np.array([[[0.25] * d], [[0.5] * d]])
    v = np.stack([f64(vc[1, 0]), f64(vc[2, last[1]])])
    ref = co.decode(np.ones((1, d)), k, v, 1.0)
    _, bl, prob = decode_bounds({**ref, "vsum": np.zeros((1, d))}, d, dt, 0.0)
    bound = HALF_STEP[dt] * np.abs(ref["o"]) + (WEIGHT[dt] + 2.0 ** -20 + prob)[:, None] * ref["absv"]
    assert (np.abs(f64(o[0]) - ref["o"]) <= bound).all()
    assert (np.abs(f64(lse[0]) - ref["lse"]) <= bl).all()
    assert (o[1] == 0).all() and torch.isposinf(lse[1]).all()
