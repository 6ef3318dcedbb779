"""The forms of the 8-bit append that sizes, turns and the spread of lengths choose between, against the
64-bit oracle: rows held by one, two or four warps, or read twice; each way in which pairs are turned;
q in place.
"""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8
from oracle import cache_oracle as co
from tests.cache8_helpers import make_cache8, numbers
from tests.cache_helpers import DT, HALF_STEP, SMALLEST, f64

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [9, 10, 11])
def test_pairs_behind_the_turned_ones_pass_whatever_their_neighbour_is(kind, n):
    """Interleaved pairs from n on are not turned: an infinity or a NaN there touches no other element."""
    d, t = 32, 3
    kc, vc, ks, vs, table = make_cache8(t, 1, 1, d, 1, 1, kind, 41)
    q, k = torch.zeros(2, t, 1, d)
    for x in (q, k):
        x[..., 2 * n] = 3.0
        x[..., 2 * n + 1] = torch.tensor([float("inf"), -float("inf"), float("nan")])[:, None]
        x[..., 30] = float("nan")   # a pair beyond the chunk that the turned ones end in
        x[..., 31] = -2.0
        x[..., 0] = 1.0
    pos, inv = ints([1, 2, 3]), torch.rand(n, device="cuda")
    zero = torch.zeros(t, 1, d).half().cuda()
    got = ab.attn_cache_append8(k.half().cuda(), zero, kc, vc, ks, vs, table, ints([0]), ints([0, t]), q=q.half().cuda(),
                                positions=pos, inv_freq=inv, interleaved=True)
    ab.check_device_status()
    assert torch.equal(got[..., 2 * n:].cpu().nan_to_num(7.0), q[..., 2 * n:].half().nan_to_num(7.0))
    assert got[..., :2 * n].isfinite().all()
    rows = table[0].long().cpu().numpy()
    codes, s, top = numbers(kc)[rows, 0, 0], c8.factor(3.0, kind), c8.TOP[kind]
    assert (f64(ks)[rows, 0, 0] == s).all()
    nan = np.nan if kind == "e4m3" else 0.0
    assert np.array_equal(codes[:, 2 * n], [c8.code(3.0 / s, kind)] * 3)
    assert np.array_equal(codes[:, 2 * n + 1], [top, -top, nan], equal_nan=True)
    assert np.array_equal(codes[:, 30:], [[nan, c8.code(-2.0 / s, kind)]] * 3, equal_nan=True)
