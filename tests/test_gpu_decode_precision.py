"""attn_decode where most of the softmax's weight lies on keys whose values are zero (attention
sinks), so that the output is made of the small weights alone."""
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
