"""The serving operators' 64-bit oracle against closed forms and attn_oracle."""
import numpy as np
import pytest

from oracle import attn_oracle, cache_oracle as co

RNG = np.random.default_rng(5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_lengths_and_relative_angles(interleaved):
    n, d = 5, 16
    inv = (0.7 ** np.arange(n)).astype(np.float32)
    q, k = RNG.standard_normal((2, 1, 1, d))
    f = lambda x, p: co.rope(x, [[p], [p]], inv, (2, 3), interleaved)[0, 0]  # noqa: E731
    assert np.isclose(np.linalg.norm(f(q, 9)), np.linalg.norm(q))
    # the product of a rotated q and k depends on the difference of the positions alone
    assert np.isclose(f(q, 9) @ f(k, 4), f(q, 105) @ f(k, 100))
    assert np.array_equal(f(q, 9)[2 * n:], q[0, 0, 2 * n:])
    back = co.rope(co.rope(q, [[9], [3]], inv, (2, 3), interleaved), [[9], [3]], inv, (2, 3),
                   interleaved, inverse=True)
    assert np.allclose(back, q, atol=1e-14)


def test_rope_gradient_is_the_inverse_rotation():
    n, d, h = 3, 8, 1e-6
    inv = np.array([1.0, 0.1, 0.01], np.float32)
    x, dy = RNG.standard_normal((2, 2, 1, d))
    pos = [[4, 11]]
    got = co.rope(dy, pos, inv, (n,), True, inverse=True)
    for t in range(2):
        for i in range(d):
            e = np.zeros_like(x)
            e[t, 0, i] = h
            diff = (co.rope(x + e, pos, inv, (n,), True) - co.rope(x - e, pos, inv, (n,), True)) / (2 * h)
            assert np.isclose(np.sum(diff * dy), got[t, 0, i], atol=1e-8)


def test_rope_sections_take_their_own_axis():
    inv = np.array([0.5, 0.25], np.float32)
    x = np.array([[[1.0, 1.0, 0.0, 0.0]]])
    y = co.rope(x, [[2], [4]], inv, (1, 1))[0, 0]
    assert np.allclose(y, [np.cos(1.0), np.cos(1.0), np.sin(1.0), np.sin(1.0)])


@pytest.mark.parametrize("window,cap", [(-1, 0.0), (4, 0.0), (0, 0.0), (-1, 3.0)])
def test_decode_is_the_last_row_of_attention(window, cap):
    n, hq, hk, d = 13, 4, 2, 8
    q = RNG.standard_normal((hq, d))
    k, v = RNG.standard_normal((2, n, hk, d))
    got = co.decode(q, k, v, 0.3, window, cap)
    for h in range(hq):
        o, lse, _ = attn_oracle.head_forward(q[h:h + 1], k[:, h // 2], v[:, h // 2], 0.3, False,
                                             (window, -1), cap)
        assert np.allclose(got["o"][h], o[0], atol=1e-12) and np.isclose(got["lse"][h], lse[0])
    assert np.isclose(got["p"].sum(), hq)


def test_keep_and_moves():
    w = np.array([5.0, 1.0, 3.0, 3.0, np.nan, 3.0, 0.0])
    pos = np.arange(7)
    assert co.keep(w, pos, 7, 3, 0) == [0, 2, 3]        # of equal weights the lower slots
    assert co.keep(w, pos, 7, 3, 2) == [0, 5, 6]        # the two newest stay
    assert co.keep(w, pos, 7, 6, 0) == [0, 1, 2, 3, 5, 6]  # NaN goes first
    assert co.keep(w, pos, 7, 7, 0) == list(range(7))
    assert co.moves([0, 5, 6], 3) == [(5, 1), (6, 2)]
