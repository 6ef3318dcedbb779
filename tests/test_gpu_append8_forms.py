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


def step_of(x, s, kind):
    """Half a step between codes at values x (beyond them by at most one binade) of factor s."""
    if kind == "int8":
        return s / 2
    e = np.floor(np.log2(np.maximum(np.abs(x) / s, 2.0 ** -6)))
    return s * np.exp2(e - 4)


LONG, MIXED, MANY = ([130, 255, 0], [300, 5, 256]), ([3, 200, 9, 50] + [17] * 60, [1, 700, 1, 1] + [1] * 60), \
    ([64, 9], [300, 200])
FORMS = [
    # dtype, kind, (old, new), hq, hk, D, page, block, n_freq, sections, interleaved
    # blocks of more tokens than four warps hold
    ("bf16", "e4m3", LONG, 4, 2, 256, 256, 256, 128, (128,), False),
    ("fp16", "int8", LONG, 2, 1, 256, 256, 256, 96, (40, 56), True),
    ("bf16", "int8", LONG, 2, 2, 192, 256, 256, 20, (20,), False),
    ("fp16", "e4m3", LONG, 4, 2, 256, 256, 256, 11, (11,), False),
    ("bf16", "e4m3", LONG, 2, 1, 144, 256, 256, 11, (5, 6), True),
    ("fp16", "int8", LONG, 9, 3, 128, 256, 256, 64, (64,), False),
    # a prompt beside many single tokens: the rule takes one warp or two, its blocks hold more
    ("bf16", "e4m3", MIXED, 8, 2, 128, 64, 64, 64, (64,), False),
    ("fp16", "int8", MIXED, 2, 2, 256, 128, 128, 20, (20,), False),
    ("bf16", "int8", MIXED, 3, 1, 128, 128, 128, 22, (10, 12), True),
    ("fp16", "e4m3", MIXED, 2, 1, 96, 256, 256, 11, (11,), False),
    # held by four warps, by two, by one
    ("bf16", "int8", MANY, 4, 2, 256, 64, 64, 20, (20,), False),
    ("fp16", "e4m3", MANY, 4, 2, 128, 128, 128, 11, (11,), True),
    ("bf16", "e4m3", MANY, 5, 1, 128, 64, 64, 11, (3, 8), False),
    ("fp16", "int8", MANY, 2, 2, 64, 64, 32, 20, (20,), False),
    ("bf16", "e4m3", MANY, 3, 3, 80, 32, 16, 36, (36,), False),
    ("fp16", "int8", MANY, 2, 1, 16, 128, 128, 5, (5,), True),
]


@pytest.mark.parametrize("case", FORMS, ids=[f"{c[0]}-{c[1]}-n{max(c[2][1])}of{len(c[2][1])}-d{c[5]}-b{c[7]}-f{c[8]}"
                                             f"{'-pairs' if c[10] else ''}" for c in FORMS])
def test_append_in_each_form(case):
    dt, kind, (old, new), hq, hk, d, page, block, n, sec, inter = case
    dt = DT[dt]
    g = torch.Generator().manual_seed(3)
    cu = np.concatenate([[0], np.cumsum(new)])
    t = int(cu[-1])
    cap = max(a + b for a, b in zip(old, new))
    # earlier factors so small that most grow: their codes are rounded again
    kc, vc, ks, vs, table = make_cache8(cap, len(old), hk, d, page, block, kind, 42, exps=(-12, -5))
    want = [(numbers(c), f64(s)) for c, s in ((kc, ks), (vc, vs))]
    before = numbers(kc)
    q, k, v = (torch.randn(t, h, d, generator=g) for h in (hq, hk, hk))
    k[::7] *= 9.0
    v[::5] *= 0.01
    q, k, v = (x.to(dt) for x in (q, k, v))
    pos = torch.randint(0, 3000, (len(sec), t), generator=g, dtype=torch.int32)
    inv = (1.0 / 500.0 ** (torch.arange(n) / n)).float()
    q2 = q.cuda()
    got = ab.attn_cache_append8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, ints(old), ints(cu), q=q2, positions=pos.cuda(),
                                inv_freq=inv.cuda(), sections=sec, interleaved=inter, out_q=q2)
    ab.check_device_status()
    assert got is q2
    rk = co.rope(f64(k), pos.numpy(), inv.numpy(), sec, inter)
    rq = co.rope(f64(q), pos.numpy(), inv.numpy(), sec, inter)
    tab = table.cpu().numpy()
    for b, was in enumerate(old):
        at = slice(cu[b], cu[b + 1])
        c8.append(*want[0], tab[b], page, was, rk[at], kind)
        c8.append(*want[1], tab[b], page, was, f64(v)[at], kind)
    assert np.array_equal(f64(vs), want[1][1]) and np.array_equal(numbers(vc), want[1][0])
    # k is turned in fp32: off by at most 2^-19 of its largest elements before it is rounded
    off = 2.0 ** -19 * 2 * np.abs(f64(k)).max()
    assert np.array_equal(f64(ks), want[0][1])
    full, got_k = np.repeat(want[0][1], block, 1)[..., None], numbers(kc)
    touched = np.zeros(got_k.shape[:2], bool)
    for b, was in enumerate(old):
        for i in range(new[b]):
            p, w = co.slot(tab[b], page, was + i)
            touched[p, w] = True
            bound = step_of(rk[cu[b] + i], full[p, w], kind) + off
            assert (np.abs(got_k[p, w] * full[p, w] - rk[cu[b] + i]) <= bound).all()
    assert np.array_equal(got_k[~touched], want[0][0][~touched])  # earlier tokens, rounded again, too
    assert (got_k[~touched] != before[~touched]).any()
    amp = 2.0 ** -19 * 2 * np.abs(f64(q)).max()
    assert (np.abs(f64(q2) - rq) <= HALF_STEP[dt] * np.abs(rq) + amp + SMALLEST[dt]).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [64, 256])  # held, read twice
def test_append_of_what_is_not_finite_in_a_prompt(kind, block):
    """An infinity in one chunk of a block's tokens, a NaN in another: the finite values of all count."""
    d, t = 256, 250
    kc, vc, ks, vs, table = make_cache8(256, 1, 1, d, block, block, kind, 43)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(t, 1, d, generator=g)
    x[7, 0, 9], x[200, 0, 3], x[249, 0, 0] = float("inf"), float("nan"), 40.0
    x = x.bfloat16()
    ab.attn_cache_append8(x.cuda(), x.cuda(), kc, vc, ks, vs, table, ints([0]), ints([0, t]))
    ab.check_device_status()
    y = f64(x)[:, 0]
    tab = table[0].cpu().numpy()
    for codes, s in ((numbers(kc), f64(ks)), (numbers(vc), f64(vs))):
        for p in range(-(-t // block)):
            rows = y[p * block:(p + 1) * block]
            f = c8.factor(np.abs(rows[np.isfinite(rows)]).max(), kind)
            assert s[tab[p], 0, 0] == f
            want = c8.code(np.nan_to_num(rows, nan=0.0, posinf=1e30) / f, kind)
            if kind == "e4m3":
                want[np.isnan(rows)] = np.nan
            assert np.array_equal(codes[tab[p], :len(rows), 0], want, equal_nan=True)
