"""Queries whose elements differ much in size, over an 8-bit cache."""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache_oracle as co
from tests.cache8_helpers import make_cache8, slots_of
from tests.cache_helpers import HALF_STEP, SMALLEST, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("exp", [4, 12, 18, 22, 24])
@pytest.mark.parametrize("group", [2, 12])
def test_decode_of_one_large_element_that_no_key_meets(kind, exp, group):
    """bf16 queries with one element 2^exp times the others, where the keys are 0: the others keep the
    precision that the sum's fp32 has.

    Bounds: a logit is a sum of D products in fp32, each partial sum may be truncated (D 2^-22 of the
    sum of magnitudes); q enters with steps of 2^-40 of its largest element; a probability is off by
    twice that and the exponentials' 2^-20; sums over n keys take n / 64 + 16 steps of 2^-23.
    """
    n, d, hk = 700, 64, 2
    kc, vc, ks, vs, table = make_cache8(n, 1, hk, d, 16, 16, kind, 51)
    codes = kc.float()
    codes[..., 5] = 0.0
    kc.view(torch.uint8).copy_(codes.to(kc.dtype).view(torch.uint8))
    q = torch.randn(1, hk * group, d, generator=torch.Generator().manual_seed(2))
    q[..., 5] = 1.5 * 2.0 ** exp
    q = q.bfloat16().cuda()
    scale = 0.25
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
    ab.check_device_status()
    k, v = slots_of(kc, ks, table, 0, range(n)), slots_of(vc, vs, table, 0, range(n))
    ref = co.decode(f64(q[0]), k, v, scale)
    most = np.repeat(np.abs(k).sum(2).max(0), group)
    logit = (d + 4) * 2.0 ** -22 * ref["mag"] + 2.0 ** -20 + 2.0 ** -40 * scale * np.abs(f64(q[0])).max(1) * most
    # (q's part is at most 2^-40 x 1.5 x 2^24 x 0.25 sum |k|, of sums near 500 0.003: beside logits that lost
    # elements of size 1 it tells)
    assert logit.max() < 2.0 ** -7
    steps = (n / 64 + 16) * 2.0 ** -23
    half = HALF_STEP[q.dtype]
    bound = half * np.abs(ref["o"]) + ref["absv"] * (2 * logit + 2.0 ** -19 + steps + 2.0 ** -22)[:, None] * (1 + half) + \
        2 * SMALLEST[q.dtype]
    assert (np.abs(f64(lse[0]) - ref["lse"]) <= logit + 2.0 ** -20 + steps + np.abs(ref["lse"]) * 2.0 ** -22).all()
    assert (np.abs(f64(o[0]) - ref["o"]) <= bound).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_decode_of_large_queries_over_large_factors_of_zeros(kind, softcap):
    # q's size times the factor is beyond fp32, but the codes that it meets are 0: all keys are alike
    n, d = 300, 64
    kc, vc, ks, vs, table = make_cache8(n, 1, 1, d, 16, 16, kind, 52)
    codes = kc.float()
    codes[..., 5] = 0.0
    kc.view(torch.uint8).copy_(codes.to(kc.dtype).view(torch.uint8))
    ks.fill_(2.0 ** 60)
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 2.0 ** 100
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, torch.tensor([n], dtype=torch.int32, device="cuda"), softcap=softcap)
    ab.check_device_status()
    v = slots_of(vc, vs, table, 0, range(n))
    want, half = v.mean(0), HALF_STEP[q.dtype]
    bound = half * np.abs(want) + np.abs(v).mean(0) * 2.0 ** -17  # exponentials 2^-20, sums of 300 keys 21 steps of 2^-23
    assert (np.abs(f64(o[0]) - want) <= bound).all()
    assert np.abs(f64(lse[0]) - np.log(n)).max() <= 2.0 ** -17
