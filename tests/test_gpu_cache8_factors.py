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


def borders(kind):
    """Numbers half way between neighbouring codes."""
    if kind == "int8":
        return np.arange(0.5, 127)
    v = c8.e4m3_values()
    return (v[1:] + v[:-1])[40:] / 2


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_append_takes_the_nearest_code_behind_any_factor(kind, dt):
    """x next to the middle of two codes of a factor that is no power of two: that middle is missed by
    less than 2^-24 of it, where x times the factor's reciprocal lies on the other side or on it."""
    batch, heads, d, page = 64, 8, 16, 2
    kc, vc, ks, vs, table = make_cache8(2, batch, heads, d, page, 2, kind, 32)
    rng = np.random.default_rng(4)
    mids = borders(kind)
    mid = rng.choice(mids[mids <= c8.TOP[kind] / 2], (batch, heads))  # so that the factor stays
    x = torch.from_numpy(rng.uniform(1.0, 2.0, (batch, heads))).to(DT[dt])
    factor = (f64(x) / mid).astype(np.float32)
    # the reciprocal's way: it rounds off another code than the nearest for some
    near = c8.code(f64(x) / factor.astype(np.float64), kind)
    twice = c8.code((x.float().numpy() * (np.float32(1.0) / factor)).astype(np.float64), kind)
    assert (near != twice).sum() > 20
    for s in (ks, vs):
        s[table[:, 0].long(), 0] = torch.from_numpy(factor).cuda()
    k, v = torch.zeros(2, batch, heads, d, dtype=DT[dt])
    k[:, :, 3], v[:, :, 12] = x, -x
    v[::2, :, 5] = float("inf")  # (its code is the largest one)
    want = [(numbers(c), f64(s)) for c, s in ((kc, ks), (vc, vs))]
    ab.attn_cache_append8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, ints([1] * batch))
    ab.check_device_status()
    rows = table[:, 0].long().cpu().numpy()
    for (codes, fac), at, sign, got, got_s in zip(want, (3, 12), (1, -1), (kc, vc), (ks, vs)):
        codes[rows, 1] = 0
        codes[rows, 1, :, at] = sign * near
        if at == 12:
            codes[rows[::2], 1, :, 5] = c8.TOP[kind]
        assert np.array_equal(f64(got_s), fac)
        assert np.array_equal(numbers(got), codes)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_rounds_earlier_codes_of_any_factor_to_the_nearest(kind):
    # code * factor / 2^e next to the middle of two codes
    batch, heads, d, page = 64, 8, 16, 2
    kc, vc, ks, vs, table = make_cache8(2, batch, heads, d, page, 2, kind, 33)
    rng = np.random.default_rng(5)
    low = borders(kind)
    mid = rng.choice(low[low < c8.TOP[kind] / 8], (batch, heads))
    code = c8.code(rng.uniform(0.6, 0.95, (batch, heads)) * c8.TOP[kind], kind)
    factor = (mid / code).astype(np.float32)  # below 1 / 4, and the new factor is 1
    product = code * factor.astype(np.float64)
    assert (c8.code(product, kind) != c8.code((code.astype(np.float32) * factor).astype(np.float64), kind)).sum() > 20
    rows = table[:, 0].long()
    for c, s in ((kc, ks), (vc, vs)):
        n = c.float()
        n[rows, 0] = 0.0
        n[rows, 0, :, 7] = torch.from_numpy(code).float().cuda()
        c.view(torch.uint8).copy_(n.to(c.dtype).view(torch.uint8))
        s[rows, 0] = torch.from_numpy(factor).cuda()
    x = torch.zeros(batch, heads, d).half()
    x[:, :, 0] = c8.TOP[kind]
    appended(kc, vc, ks, vs, table, page, [1] * batch, list(range(batch + 1)), x.cuda(), -x.cuda(), kind)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_of_prompts_behind_any_factors(kind):
    old, new, d, page, block = [5, 0, 70, 130], [90, 33, 1, 200], 96, 128, 32
    kc, vc, ks, vs, table = make_cache8(330, 4, 3, d, page, block, kind, 34)
    g = torch.Generator().manual_seed(6)
    for s in (ks, vs):
        s.mul_((1.0 + torch.rand(s.shape, generator=g)).cuda())
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v = torch.randn(2, cu[-1], 3, d, generator=g).half().cuda()
    v *= 20.0
    appended(kc, vc, ks, vs, table, page, old, cu, k, v, kind)


def rounded(x, dt):
    """x (64 bits) rounded once to `dt`, ties to even; within the type's normal range."""
    bits = 11 if dt == "fp16" else 8
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("heads,d", [(8, 128), (1, 16)])
def test_load_rounds_once_behind_any_factor(kind, dt, heads, d):
    """code * factor next to the middle of two numbers of the type, which its rounding to fp32 makes a tie."""
    pages, page = 64, 32
    kc, vc, ks, vs, table = make_cache8(pages * page, 1, heads, d, page, 1, kind, 35, spare=0)
    rng = np.random.default_rng(7)
    bits = 11 if dt == "fp16" else 8
    # a factor for each slot and head, and codes of which one in it makes such a product
    code = c8.code(rng.uniform(0.6, 0.95, (pages, page, heads)) * c8.TOP[kind], kind)
    mid = (2.0 ** bits / 2 + rng.integers(0, 2 ** (bits - 1), code.shape) + 0.5) / 2.0 ** bits
    factor = (mid / code).astype(np.float32)
    once = rounded(code * factor.astype(np.float64), dt)
    twice = rounded((code.astype(np.float32) * factor).astype(np.float64), dt)
    assert (once != twice).sum() > 50
    for c, s in ((kc, ks), (vc, vs)):
        n = c.float()
        n[..., 3] = torch.from_numpy(code).float().cuda()
        c.view(torch.uint8).copy_(n.to(c.dtype).view(torch.uint8))
        s.copy_(torch.from_numpy(factor).cuda())
    got = ab.attn_cache_load8(kc, vc, ks, vs, table, ints([0]), ints([0, pages * page]), pages * page, dtype=DT[dt])
    ab.check_device_status()
    rows = table[0].long().cpu().numpy()
    for x, c in zip(got, (kc, vc)):
        want = rounded(numbers(c) * factor.astype(np.float64)[..., None], dt)[rows].reshape(-1, heads, d)
        small = np.abs(want) < 2.0 ** -14  # fp16's steps below: rounded at 2^-24
        assert np.array_equal(f64(x)[~small], want[~small])
        assert (np.abs(f64(x) - want)[small] <= 2.0 ** -24).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("gap", [120, 128, 136, 144])
@pytest.mark.parametrize("n,group", [(4096, 2), (30000, 1), (700, 16)])
def test_decode_of_improbable_keys_whose_values_are_large(kind, gap, n, group):
    """Most keys are 2^-gap times as probable as one of them and have values up to 2^120 times as large,
    in other blocks' parts of the sequence: they make up O where the gap is small enough, and are as
    good as nothing beside it where it is not."""
    d = 64
    kc, vc, ks, vs, table = make_cache8(n, 1, 1, d, 16, 16, kind, 36, exps=(0, 0))
    for c in (kc, vc):
        c.view(torch.uint8).zero_()
    rows = table[0].long()
    vs.fill_(2.0 ** 60)
    vs[rows[(n - 1) // 16]] = 2.0 ** -60
    at = (rows[torch.arange(n) // 16], torch.arange(n) % 16)
    k, v = kc.float(), vc.float()
    # base-2 logits are sums of two codes; the last block's keys but one take no part
    k[at[0], at[1], 0, 0] = -104.0
    k[at[0], at[1], 0, 1] = 104.0 - gap
    last = torch.arange((n - 1) // 16 * 16, n)
    k[at[0][last], at[1][last], 0, 0] = -112.0
    k[at[0][last], at[1][last], 0, 1] = -112.0
    k[at[0][n - 1], at[1][n - 1], 0, :2] = 0.0
    g = torch.Generator().manual_seed(8)
    v[at[0], at[1], 0] = torch.randint(1, 9, (n, d), generator=g).float().cuda()
    for c, x in ((kc, k), (vc, v)):
        c.view(torch.uint8).copy_(x.to(c.dtype).view(torch.uint8))
    q = torch.zeros(1, group, d, dtype=torch.bfloat16, device="cuda")
    q[..., :2] = 1.0
    scale = float(np.log(2.0))
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints([n]), scale=scale)
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, [n], scale)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_decode_behind_factors_that_are_no_powers_of_two(kind):
    lens, d = [900, 0, 77, 3000], 128
    kc, vc, ks, vs, table = make_cache8(3000, 4, 2, d, 48, 12, kind, 37)
    g = torch.Generator().manual_seed(9)
    for s in (ks, vs):
        s.mul_((1.0 + torch.rand(s.shape, generator=g)).cuda())
    for dt, group in (("fp16", 4), ("bf16", 12)):
        q = torch.randn(4, 2 * group, d, generator=g).to(DT[dt]).cuda()
        o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
        ab.check_device_status()
        check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5)
