"""The 64-bit oracle of the 8-bit cache and of shared pages against torch's own type, closed forms
and invariants (no GPU needed)."""
import numpy as np
import pytest
import torch

from oracle import cache8_oracle as c8

RNG = np.random.default_rng(8)


def test_e4m3_codes_are_those_of_the_type():
    all_codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(all_codes, c8.e4m3_values())
    x = np.concatenate([RNG.standard_normal(4000) * 2.0 ** RNG.integers(-12, 9, 4000), all_codes,
                        (all_codes[1:] + all_codes[:-1]) / 2])  # and every tie
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(c8.code(x, "e4m3"), want)
    assert np.array_equal(c8.code([0.5, 1.5, -2.5, 300, -129], "int8"), [0, 2, -2, 127, -127])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_factor_is_the_smallest_power_of_two(kind):
    top = c8.TOP[kind]
    for e in (-20, -3, 0, 5):
        assert c8.factor(top * 2.0 ** e, kind) == 2.0 ** e
        assert c8.factor(top * 2.0 ** e * (1 + 2.0 ** -40), kind) == 2.0 ** (e + 1)
    assert c8.factor(0.0, kind) == 2.0 ** -60 and c8.factor(1e300, kind) == 2.0 ** 60


@pytest.mark.parametrize("kind,rel", [("e4m3", 2.0 ** -4), ("int8", 2.0 ** -1)])
def test_values_are_a_rounding_off_and_pieces_end_alike(kind, rel):
    heads, dim, page, block = 2, 16, 8, 4
    x = RNG.standard_normal((19, heads, dim)) * 2.0 ** RNG.integers(-2, 3, (19, 1, 1))
    whole = (np.zeros((4, page, heads, dim)), np.ones((4, 2, heads)))
    c8.append(*whole, [2, 0, 3, 1], page, 0, x, kind)
    got = c8.values(*whole)[[2, 0, 3]].reshape(-1, heads, dim)[:19]
    step = np.repeat(whole[1][[2, 0, 3]].reshape(-1, heads), block, 0)[:19, :, None]
    bound = np.abs(x) * rel + step * 2.0 ** -10 if kind == "e4m3" else step * rel
    assert (np.abs(got - x) <= bound).all()
    # one by one: the same factors, since they only follow the largest value so far
    parts = (np.zeros((4, page, heads, dim)), np.ones((4, 2, heads)))
    for t in range(19):
        c8.append(*parts, [2, 0, 3, 1], page, t, x[t:t + 1], kind)
    assert np.array_equal(parts[1], whole[1])
    again = c8.values(*parts)[[2, 0, 3]].reshape(-1, heads, dim)[:19]
    assert (np.abs(again - x) <= 2 * bound).all()  # rounded again where a factor grew


@pytest.mark.parametrize("share", [True, False])
def test_fork_keeps_the_count_of_references(share):
    page, rows, width, pages = 4, 6, 5, 40
    lens = np.array([0, 3, 8, 13, 17, 20])
    table, refs, at = np.full((rows, width), -1), np.zeros(pages, int), iter(RNG.permutation(pages))
    for b in range(rows):
        for i in range(-(-lens[b] // page)):
            table[b, i] = next(at)
            refs[table[b, i]] = 1
    for parents in ([0, 1, 2, 3, 4, 5], [5, 5, 3, 3, -1, 1], [-1] * 6, [4, 4, 4, 4, 4, 4]):
        t, n, r, made, free, missing = c8.fork(table, lens, refs, page, parents, [3] * rows, share)
        assert not missing and free == (r == 0).sum()
        count = np.bincount(t[t >= 0], minlength=pages)
        assert np.array_equal(count, r)
        for b, s in enumerate(parents):
            assert n[b] == (lens[s] if s >= 0 else 0)
            assert (t[b, :-(-min(n[b] + 3, width * page) // page)] >= 0).all() or s < 0
            # no slot that a row may write lies in a page of another row
            if s >= 0 and n[b] < width * page:
                assert r[t[b, n[b] // page]] == 1
        assert len({p for _, p in made}) == len(made)
