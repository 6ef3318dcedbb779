"""Factors of the 8-bit cache that its own append does not make: 0, no powers of two, far apart.

An append re-rounds what stands behind them and takes the nearest codes, a read-back rounds each
value once, attention keeps every weight that the factors leave in O.
"""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8
from tests.cache8_helpers import check_decode8, make_cache8, numbers
from tests.cache_helpers import DT, f64

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def appended(kc, vc, ks, vs, table, page, old, cu, k, v, kind):
    """Appends k and v (not turned) and compares every code and factor with the oracle's."""
    tab = table.cpu().numpy()
    want = [(numbers(c), f64(s)) for c, s in ((kc, ks), (vc, vs))]
    ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, ints(old), ints(cu))
    ab.check_device_status()
    for (codes, fac), x, got, got_s in zip(want, (k, v), (kc, vc), (ks, vs)):
        for b, n in enumerate(old):
            c8.append(codes, fac, tab[b], page, n, f64(x)[cu[b]:cu[b + 1]], kind)
        assert np.array_equal(f64(got_s), fac)
        assert np.array_equal(numbers(got), codes)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,block,old,new", [
    (64, 16, 4, [3, 5, 0], [1, 1, 1]),            # a token each
    (128, 64, 64, [40, 63], [24, 200]),           # warps share the rows of a head
    (256, 128, 128, [100, 7], [300, 121]),        # more tokens than the warps hold
])
def test_append_behind_a_factor_of_zero(kind, d, page, block, old, new):
    # earlier slots whose factor is 0 stand for zeros, whatever their codes are, and go on to
    kc, vc, ks, vs, table = make_cache8(max(a + b for a, b in zip(old, new)), len(old), 2, d, page, block, kind, 31)
    ks.zero_()
    vs[:, :, 1] = 0.0  # of one head only
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v = torch.randn(2, cu[-1], 2, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    v[:, 0] *= 64.0  # the other head's factor grows
    assert (numbers(kc) != 0).any() and (numbers(vc) != 0).any()
    appended(kc, vc, ks, vs, table, page, old, cu, k, v, kind)
