"""The cache in 8 bits on the GPU: append, read-back, single-token attention, and the three with
forked pages as a serving loop, against the 64-bit oracle.

Bad pages and lengths below are given in arrays of their full size: the kernels look at an entry
before they use it, so nothing is read or written out of range.
"""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8
from oracle import cache_oracle as co
from tests.cache8_helpers import check_decode8, make_cache8, numbers, slots_of
from tests.cache_helpers import DT, HALF_STEP, SMALLEST, f64

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def step_of(x, s, kind):
    """Half a step between codes at values x (beyond them by at most one binade) of factor s."""
    if kind == "int8":
        return s / 2
    e = np.floor(np.log2(np.maximum(np.abs(x) / s, 2.0 ** -6)))
    return s * np.exp2(e - 4)


# ------------------------------------------------------------------ append and read-back

APPEND = [
    # dtype, kind, old lengths, new lengths, hq, hk, D, page, block, heads_first, n_freq, sections, interleaved
    ("bf16", "e4m3", [0], [1], 1, 1, 64, 16, 16, False, 32, (32,), False),
    ("fp16", "int8", [5, 0, 63, 17], [3, 0, 65, 1], 4, 2, 128, 16, 4, False, 64, (16, 24, 24), False),
    ("bf16", "int8", [7, 0, 200], [0, 300, 29], 6, 2, 80, 48, 48, True, 20, (12, 8), True),
    ("fp16", "e4m3", [1, 2, 3], [5, 40, 1], 2, 2, 96, 1, 1, False, 11, (5, 6), False),
    ("bf16", "e4m3", [100] * 9, [1] * 9, 32, 8, 128, 64, 16, False, 64, (64,), False),
    ("bf16", "int8", [0, 12], [700, 900], 16, 16, 256, 100, 20, True, 128, (128,), True),
    ("fp16", "e4m3", [3, 250], [600, 260], 3, 3, 16, 256, 256, False, 8, (8,), False),
    ("bf16", "e4m3", [9, 31], [70, 5], 5, 1, 144, 32, 8, True, 36, (20, 16), False),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[0]}-{c[1]}-{len(c[2])}seq-d{c[6]}-p{c[7]}-b{c[8]}" for c in APPEND])
def test_append_rounds_rotated_keys_and_values(case):
    dt, kind, old, new, hq, hk, d, page, block, hf, n, sec, inter = case
    dt = DT[dt]
    g = torch.Generator().manual_seed(2)
    cu = np.concatenate([[0], np.cumsum(new)])
    t = int(cu[-1]) + 2  # two tokens behind the last sequence
    cap = max(a + b for a, b in zip(old, new))
    kc, vc, ks, vs, table = make_cache8(cap, len(old), hk, d, page, block, kind, 3, hf)
    want = [numbers(kc), numbers(vc)]
    fac = [f64(ks), f64(vs)]
    q, k, v = (torch.randn(t, h, d, generator=g) for h in (hq, hk, hk))
    k[::7] *= 9.0
    v[::5] *= 0.01
    q, k, v = (x.to(dt) for x in (q, k, v))
    pos = torch.randint(0, 3000, (len(sec), t), generator=g, dtype=torch.int32)
    inv = (1.0 / 500.0 ** (torch.arange(n) / n)).float()
    oq = torch.full_like(q, 5.0).cuda()
    got = ab.attn_cache_append8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, ints(old), ints(cu), q=q.cuda(),
                                positions=pos.cuda(), inv_freq=inv.cuda(), sections=sec, interleaved=inter, out_q=oq)
    ab.check_device_status()
    assert got is oq
    rk = co.rope(f64(k), pos.numpy(), inv.numpy(), sec, inter)
    rq = co.rope(f64(q), pos.numpy(), inv.numpy(), sec, inter)
    tab = table.cpu().numpy()
    for b, was in enumerate(old):
        at = slice(cu[b], cu[b + 1])
        c8.append(want[0], fac[0], tab[b], page, was, rk[at], kind)
        c8.append(want[1], fac[1], tab[b], page, was, f64(v)[at], kind)
    # v is rounded from its own values: every code and factor is the oracle's
    assert np.array_equal(f64(vs), fac[1])
    assert np.array_equal(numbers(vc), want[1])
    # k from its rotation in fp32: off by at most 2^-19 of its largest element before the rounding
    off = 2.0 ** -19 * 2 * np.abs(f64(k)).max()
    assert np.array_equal(f64(ks), fac[0])
    full = np.repeat(fac[0], block, 1)[..., None]
    got_k, want_k = numbers(kc), want[0]
    touched = np.zeros(got_k.shape[:2], bool)
    for b, was in enumerate(old):
        for i in range(new[b]):
            p, w = co.slot(tab[b], page, was + i)
            touched[p, w] = True
            bound = step_of(rk[cu[b] + i], full[p, w], kind) + off
            assert (np.abs(got_k[p, w] * full[p, w] - rk[cu[b] + i]) <= bound).all()
    assert np.array_equal(got_k[~touched], want_k[~touched])  # earlier tokens too
    live = np.arange(t) < cu[-1]
    amp = 2.0 ** -19 * 2 * np.abs(f64(q)).max()
    assert (np.abs(f64(oq) - rq)[live] <= (HALF_STEP[dt] * np.abs(rq) + amp + SMALLEST[dt])[live]).all()
    assert (f64(oq)[~live] == 5.0).all()
    # in place, as a decode step does, q's rotation is the same
    q2 = q.cuda()
    ab.attn_cache_append8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, ints(old), ints(cu), q=q2, positions=pos.cuda(),
                          inv_freq=inv.cuda(), sections=sec, interleaved=inter, out_q=q2)
    assert torch.equal(q2[:cu[-1]], oq[:cu[-1]])
    assert np.array_equal(numbers(vc), want[1]) and np.array_equal(f64(vs), fac[1])  # the same tokens again
    # read back: the codes times the factors, rounded once
    rows = int(cu[-1])
    out = [torch.full((rows + 1, hk, d), 3.0, dtype=dt, device="cuda") for _ in range(2)]
    ab.attn_cache_load8(kc, vc, ks, vs, table, ints(old), ints(cu), rows + 1, dtype=dt, out_k=out[0], out_v=out[1])
    ab.check_device_status()
    for x, codes, s in ((out[0], kc, ks), (out[1], vc, vs)):
        for b, was in enumerate(old):
            ref = slots_of(codes, s, table, b, range(was, was + new[b]))
            assert torch.equal(x[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(ref).float().to(dt))
        assert (x[rows] == 3.0).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_without_rotation_one_token_each(kind):
    kc, vc, ks, vs, table = make_cache8(20, 3, 2, 64, 8, 4, kind, 4)
    k, v = torch.randn(2, 3, 2, 64).half().cuda()
    old = [0, 7, 16]
    codes, fac, tab = numbers(vc), f64(vs), table.cpu().numpy()
    kcodes, kfac = numbers(kc), f64(ks)
    assert ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, ints(old)) is None
    ab.check_device_status()
    for b, n in enumerate(old):
        c8.append(codes, fac, tab[b], 8, n, f64(v[b:b + 1]), kind)
        c8.append(kcodes, kfac, tab[b], 8, n, f64(k[b:b + 1]), kind)
    assert np.array_equal(numbers(vc), codes) and np.array_equal(f64(vs), fac)
    assert np.array_equal(numbers(kc), kcodes) and np.array_equal(f64(ks), kfac)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_of_borders_zeros_and_what_is_not_finite(kind):
    top = c8.TOP[kind]
    kc, vc, ks, vs, table = make_cache8(8, 1, 1, 16, 8, 1, kind, 5)
    x = torch.zeros(8, 1, 16)
    x[0, 0, 3] = top                       # the largest value of factor 1
    x[1, 0, 3] = top * (1 + 2.0 ** -7)     # the next one in bf16
    x[2, 0, :2] = torch.tensor([2.0 ** 100, -1.0])   # beyond the factors
    x[3, 0, :2] = torch.tensor([2.0 ** -100, 0.0])   # below them
    x[4, 0, :3] = torch.tensor([float("inf"), 2.0, -float("inf")])
    x[5, 0, :2] = torch.tensor([float("nan"), -3.0])
    x = x.bfloat16().cuda()
    ab.attn_cache_append8(x, x, kc, vc, ks, vs, table, ints([0]), ints([0, 8]))
    ab.check_device_status()
    p = int(table[0, 0])
    s, c = f64(vs)[p, :, 0], numbers(vc)[p, :, 0]
    two = c8.factor(2.0, kind)
    assert np.array_equal(s, [1.0, 2.0, 2.0 ** 60, 2.0 ** -60, two, c8.factor(3.0, kind), 2.0 ** -60, 2.0 ** -60])
    assert c[0, 3] == top and c[1, 3] == c8.code(float(x[1, 0, 3]) / 2, kind)
    assert c[2, 0] == top and c[2, 1] == 0 and c[3, 0] == 0
    assert list(c[4, :3]) == [top, 2.0 / two, -top]
    assert (np.isnan(c[5, 0]) if kind == "e4m3" else c[5, 0] == 0) and c[5, 1] == c8.code(-3 / s[5], kind)
    assert (c[6:] == 0).all()


def test_append_leaves_out_what_does_not_fit_and_reports_it():
    kc, vc, ks, vs, table = make_cache8(16, 4, 2, 64, 8, 8, "e4m3", 5)
    table[1, 1] = kc.shape[0]      # a page that does not exist
    table[2, 0] = -1
    before = [x.clone() for x in (kc, vc, ks, vs)]
    k, v = torch.randn(2, 5, 2, 64).half().cuda()
    q = torch.randn(5, 2, 64).half().cuda()
    pos, inv = ints([0] * 5), torch.ones(32, device="cuda")
    got = ab.attn_cache_append8(k[:4], v[:4], kc, vc, ks, vs, table, ints([3, 9, 0, 16]), q=q[:4], positions=pos[:4],
                                inv_freq=inv)  # the last one is full
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert e.value.code == -9
    ab.check_device_status()  # cleared
    assert torch.equal(got, q[:4])  # position 0; rotated all the same
    p = int(table[0, 0])
    for x, was in zip((kc, vc, ks, vs), before):
        y = x.view(torch.uint8) if x.dtype is not torch.float32 else x
        z = was.view(torch.uint8) if x.dtype is not torch.float32 else was
        changed = (y != z).flatten(1).any(1).nonzero().view(-1).tolist()
        assert changed in ([p], [])
    # a negative length; offsets that do not ascend: their tokens are left out
    ab.attn_cache_append8(k, v, kc, vc, ks, vs, table[:1].expand(3, -1).contiguous(), ints([0, -1, 0]), ints([0, 2, 4, 3]))
    with pytest.raises(ab.AttnError):
        ab.check_device_status()
    # a read-back of the same: rows of zeros
    out = ab.attn_cache_load8(kc, vc, ks, vs, table, ints([3, 9, 0, 16]), ints([0, 1, 2, 3, 4]), 4, dtype=torch.float16)
    with pytest.raises(ab.AttnError):
        ab.check_device_status()
    for x in out:
        assert (x[1:] == 0).all() and (x[0] != 0).any()


def test_append_and_load_with_strides_and_a_huge_cache():
    # pages behind 2^32 bytes, factors with strides of their own, k and v slices of a larger tensor
    pages, page, hk, d = 70000, 64, 8, 128
    kc, vc = (torch.zeros(pages, page, hk, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(hk, pages, 4, device="cuda").permute(1, 2, 0) for _ in range(2))
    table = ints([[pages - 1, 1, pages - 2], [pages // 2, 0, pages - 3]])
    qkv = torch.randn(150, 3 * hk, d, device="cuda").bfloat16()
    k, v = qkv[:, hk:2 * hk], qkv[:, 2 * hk:]
    old, cu = [60, 3], [0, 80, 150]
    ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, ints(old), ints(cu))
    gk, gv = ab.attn_cache_load8(kc, vc, ks, vs, table, ints(old), ints(cu), 150)
    ab.check_device_status()
    for got, x in ((gk, k), (gv, v)):
        # half a step of int8 is at most 2^-7 of the block's largest value or, where the block's earlier
        # slots had a factor of 1, half of it; and bf16's own rounding
        assert (f64(got) - f64(x)).max() <= 0.5 + 2.0 ** -5
        assert np.abs(f64(got) - f64(x))[30:80].max() <= np.abs(f64(x)).max() * (2.0 ** -7 + 2.0 ** -8)
    q = torch.randn(2, 16, d, device="cuda").bfloat16()
    lens = [o + n for o, n in zip(old, (80, 70))]
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5)


# ------------------------------------------------------------------ attention

DECODE = [
    # dtype, kind, lengths, hq, hk, D, page, block, heads_first, window, softcap
    ("bf16", "e4m3", [1, 0, 128, 127, 129], 4, 4, 64, 16, 16, False, -1, 0.0),
    ("fp16", "int8", [256, 255, 257, 1], 8, 2, 128, 16, 8, False, -1, 0.0),
    ("fp16", "e4m3", [1000, 3, 0, 777], 6, 2, 128, 64, 16, True, -1, 0.0),
    ("bf16", "int8", [513, 2000], 16, 2, 96, 48, 24, False, -1, 0.0),
    ("bf16", "e4m3", [300, 4097], 18, 2, 128, 100, 25, False, -1, 0.0),
    ("fp16", "int8", [5, 900, 31], 16, 1, 64, 1, 1, False, -1, 0.0),
    ("bf16", "e4m3", [700, 64], 20, 1, 256, 32, 32, True, -1, 0.0),
    ("fp16", "e4m3", [2500, 16, 17], 3, 1, 192, 128, 128, False, -1, 0.0),
    ("bf16", "int8", [600, 1500], 9, 1, 192, 64, 8, False, 100, 0.0),
    ("fp16", "int8", [1, 1023, 1024, 1500], 4, 4, 256, 48, 24, False, 1022, 30.0),
    ("bf16", "e4m3", [40, 800], 5, 1, 16, 8, 2, False, 0, 0.0),
    ("fp16", "e4m3", [333, 90], 2, 2, 80, 24, 8, True, 64, 5.0),
    ("bf16", "int8", [2049, 130, 1], 32, 8, 112, 256, 64, False, -1, 0.0),
    ("fp16", "int8", [450], 12, 1, 144, 16, 16, False, -1, 20.0),
    ("bf16", "e4m3", [100] * 70, 8, 8, 128, 16, 16, False, -1, 0.0),
    ("bf16", "e4m3", [130, 7] * 40, 16, 16, 64, 16, 16, True, -1, 0.0),
    ("fp16", "e4m3", [30000], 4, 1, 128, 64, 16, False, -1, 0.0),
    ("bf16", "int8", [9000, 0, 12000], 40, 2, 64, 64, 64, False, -1, 0.0),
]


@pytest.mark.parametrize("case", DECODE, ids=[f"{c[0]}-{c[1]}-{c[3]}h{c[4]}-d{c[5]}-p{c[6]}b{c[7]}-n{max(c[2])}" for c in DECODE])
def test_decode(case):
    dt, kind, lens, hq, hk, d, page, block, hf, window, cap = case
    kc, vc, ks, vs, table = make_cache8(max(lens), len(lens), hk, d, page, block, kind, 7, hf)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(1)).to(DT[dt]).cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens), max_seqlen=max(lens), window=(window, -1), softcap=cap)
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5, window, cap)
    # a loose bound of the lengths cuts the work otherwise; each of the two gives the same bits again
    o2, lse2 = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens), window=(window, -1), softcap=cap)
    check_decode8(o2, lse2, q, kc, vc, ks, vs, table, lens, d ** -0.5, window, cap)
    o3, lse3 = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens), max_seqlen=max(lens), window=(window, -1), softcap=cap)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [2, 8, 11, 16])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_decode_every_width_and_group(kind, group, d):
    lens = [777, 0, 130, 2500]
    kc, vc, ks, vs, table = make_cache8(2500, 4, 2, d, 32, 16, kind, 22, heads_first=d == 96)
    q = torch.randn(4, 2 * group, d, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    for window, cap in ((-1, 0.0), (300, 25.0)):
        o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens), window=(window, 0), softcap=cap)
        ab.check_device_status()
        check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5, window, cap)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("exps", [(-40, 30), (-60, -50), (50, 60)])
def test_decode_with_factors_far_apart(dt, kind, exps):
    # V's factors anywhere in their range; K's near 1 and q small, so that the logits are moderate
    lens, d = [600, 90], 64
    kc, vc, ks, vs, table = make_cache8(600, 2, 2, d, 32, 16, kind, 11)
    g = torch.Generator().manual_seed(11)
    vs.copy_(torch.exp2(torch.randint(exps[0], exps[1] + 1, vs.shape, generator=g).float()))
    vs[::7] = 0.0  # blocks of zeros
    if dt == "fp16":  # the output stays within fp16
        vs.mul_(2.0 ** -exps[1])
        vs.copy_(torch.where(vs > 0, vs.clamp(min=2.0 ** -60), vs))
    q = (torch.randn(2, 4, d, generator=g) * 0.5).to(DT[dt]).cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("low,high", [(0.0, 60), (-60, 60), (60, -60), (60, 0.0)])
@pytest.mark.parametrize("n,cut", [(4096, 2048), (600, 320), (200, 16)])
def test_decode_where_factors_change_along_the_sequence(kind, low, high, n, cut):
    """The maximum that weights are taken from follows V's factors; the softmax's sum must not.  The
    first keys, up to 2^20 times less probable, have one factor (0.0: none), the others another."""
    d = 64
    kc, vc, ks, vs, table = make_cache8(n, 1, 1, d, 16, 16, kind, 18, exps=(-6, -6))
    rows = table[0].long()
    for lo, hi, f in ((0, cut // 16, low), (cut // 16, len(rows), high)):
        vs[rows[lo:hi]] = 2.0 ** f if f != 0.0 else 0.0
    g = torch.Generator().manual_seed(5)
    for shift in (0.0, -8.0, -20.0, 8.0):  # of the first keys' base-2 logits
        first = (torch.arange(n) < cut).float()
        want = torch.randn(n, generator=g) + shift * first
        kc.view(torch.uint8).zero_()
        page, at = rows[torch.arange(n) // 16], torch.arange(n) % 16
        # a logit is code * factor * q: codes of 1 / 4 of a step, q makes them base-2 logits
        code = (want * 4).round().clamp(-100, 100)
        codes = kc.float()
        codes[page, at, 0, 0] = code.cuda()
        kc.view(torch.uint8).copy_(codes.to(kc.dtype).view(torch.uint8))
        q = torch.zeros(1, 2, d, dtype=torch.bfloat16, device="cuda")
        q[0, :, 0] = 16.0
        scale = float(np.log(2.0))
        o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints([n]), scale=scale)
        ab.check_device_status()
        check_decode8(o, lse, q, kc, vc, ks, vs, table, [n], scale)


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
def test_decode_of_queries_far_from_one(size):
    lens, d = [300], 128
    kc, vc, ks, vs, table = make_cache8(300, 1, 2, d, 16, 16, "e4m3", 12)
    q = (torch.randn(1, 8, d) * size).bfloat16().cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens), scale=d ** -0.5 / size)
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5 / size)


def test_decode_of_weights_far_below_the_largest():
    # one key of 2^30 times the others' weight, and of value 0
    n, d = 16384, 64
    kc, vc, ks, vs, table = make_cache8(n, 1, 1, d, 64, 64, "int8", 13, exps=(0, 0))
    kc.zero_()
    vc.fill_(64)
    page, at = int(table[0, 100]), 5
    vc[page, at] = 0
    kc[page, at, 0, 0] = 64
    q = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda")
    q[0, 0, 0] = 30 * np.log(2.0) / 64
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints([n]), scale=1.0)
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, [n], 1.0)
    assert (o > 0).all()


def test_decode_of_a_key_that_is_not_a_number():
    kc, vc, ks, vs, table = make_cache8(200, 2, 2, 64, 16, 16, "e4m3", 14)
    nan = torch.full((1,), 0x7f, dtype=torch.uint8, device="cuda")
    p = int(table[0, 3])
    kc.view(torch.uint8)[p, 2, 1, 7] = nan
    # behind the last slot, and in the second sequence's unused pages: takes no part
    kc.view(torch.uint8)[int(table[0, 12]), 8:] = nan
    vc.view(torch.uint8)[int(table[0, 12]), 8:] = nan
    q = torch.randn(2, 4, 64).half().cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints([200, 150]))
    ab.check_device_status()
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert o[0, :2].isfinite().all() and o[1].isfinite().all()


def test_decode_leaves_out_bad_pages_and_lengths_and_reports_them():
    lens = [200, 100, 60]
    kc, vc, ks, vs, table = make_cache8(256, 3, 2, 128, 16, 8, "int8", 15)
    good = table.clone()
    table[0, 2] = kc.shape[0]
    table[1, 0] = -5
    q = torch.randn(3, 4, 128).bfloat16().cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
    with pytest.raises(ab.AttnError):
        ab.check_device_status()
    # the same as without these slots: their keys' weights are 0
    for b, gone in ((0, range(32, 48)), (1, range(0, 16))):
        j = [x for x in range(lens[b]) if x not in gone]
        k, v = slots_of(kc, ks, good, b, j), slots_of(vc, vs, good, b, j)
        ref = co.decode(f64(q[b]), k, v, 128 ** -0.5)
        assert np.abs(f64(o[b]) - ref["o"]).max() <= 2.0 ** -8 * np.abs(ref["o"]).max() + 2.0 ** -12 * ref["absv"].max()
        assert np.abs(f64(lse[b]) - ref["lse"]).max() <= 2.0 ** -14
    check_decode8(o, lse, q, kc, vc, ks, vs, good, lens, 128 ** -0.5, skip=(0, 1))
    for bad in ([200, 257, 60], [200, -1, 60]):
        o, lse = ab.attn_decode8(q, kc, vc, ks, vs, good, ints(bad), max_seqlen=256)
        with pytest.raises(ab.AttnError):
            ab.check_device_status()
        check_decode8(o, lse, q, kc, vc, ks, vs, good, [200, 0, 60], 128 ** -0.5)
    table[0] = -1  # every key's page is bad: a row without keys
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
    with pytest.raises(ab.AttnError):
        ab.check_device_status()
    assert (o[0] == 0).all() and lse[0].isposinf().all()


def test_decode_into_strided_outputs_on_a_stream_and_in_a_graph():
    lens = [500, 31, 900]
    kc, vc, ks, vs, table = make_cache8(900, 3, 4, 64, 16, 16, "e4m3", 16)
    wide = torch.randn(3, 12, 2, 64).half().cuda()
    q = wide[:, :, 1]
    out = torch.full((3, 12, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    n = ints(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, n, out=out[:, :, 0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, 64 ** -0.5)
    assert (out[:, :, 1] == 7.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, n)
    for k in range(3):
        lens = [max(0, x - 13 * k) for x in lens]
        n.copy_(ints(lens))
        wide.copy_(torch.randn(3, 12, 2, 64).half())
        graph.replay()
        ab.check_device_status()
        check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, 64 ** -0.5)


@pytest.mark.parametrize("d", [32, 48, 160, 176, 208, 224, 240])
def test_other_head_dims(d):
    # a prompt and single tokens into blocks of 8, and attention over them
    dt, kind, page, hk = torch.float16, "e4m3" if d % 32 else "int8", 24, 2
    kc, vc, ks, vs, table = make_cache8(300, 2, hk, d, page, 8, kind, 20)
    want, fac, tab = numbers(vc), f64(vs), table.cpu().numpy()
    lens = [0, 5]
    for new in ([250, 3], [1, 1], [1, 1]):
        cu = [0, new[0], sum(new)]
        q, k, v = (torch.randn(cu[2], h, d).to(dt).cuda() for h in (3 * hk, hk, hk))
        pos, inv = ints(list(range(cu[2]))), torch.rand(d // 2, device="cuda")
        got = ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, ints(lens), ints(cu), q=q, positions=pos, inv_freq=inv)
        ab.check_device_status()
        for b in range(2):
            c8.append(want, fac, tab[b], page, lens[b], f64(v)[cu[b]:cu[b + 1]], kind)
        assert np.array_equal(numbers(vc), want) and np.array_equal(f64(vs), fac)
        rq = co.rope(f64(q), [list(range(cu[2]))], inv.cpu().numpy(), (d // 2,))
        assert (np.abs(f64(got) - rq) <= HALF_STEP[dt] * np.abs(rq) + 2.0 ** -19 * 2 * np.abs(f64(q)).max()).all()
        lens = [a + b for a, b in zip(lens, new)]
        last = got[[cu[1] - 1, cu[2] - 1]]
        o, lse = ab.attn_decode8(last, kc, vc, ks, vs, table, ints(lens))
        ab.check_device_status()
        check_decode8(o, lse, last, kc, vc, ks, vs, table, lens, d ** -0.5)


def test_many_sequences():
    # more of them than a block has threads, some without keys
    batch, hk, d, page = 700, 2, 64, 16
    rng = np.random.default_rng(21)
    lens = rng.integers(0, 60, batch)
    kc, vc, ks, vs, table = make_cache8(64, batch, hk, d, page, 16, "int8", 21)
    want, fac, tab = numbers(vc), f64(vs), table.cpu().numpy()
    new = rng.integers(0, 4, batch)
    cu = np.concatenate([[0], np.cumsum(new)])
    k, v = torch.randn(2, int(cu[-1]), hk, d).half().cuda()
    ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, ints(lens), ints(cu))
    ab.check_device_status()
    for b in range(batch):
        c8.append(want, fac, tab[b], page, int(lens[b]), f64(v)[cu[b]:cu[b + 1]], "int8")
    assert np.array_equal(numbers(vc), want) and np.array_equal(f64(vs), fac)
    gk, gv = ab.attn_cache_load8(kc, vc, ks, vs, table, ints(lens), ints(cu), int(cu[-1]), dtype=torch.float16)
    ab.check_device_status()
    for b in range(0, batch, 7):
        j = range(int(lens[b]), int(lens[b] + new[b]))
        assert torch.equal(gv[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(slots_of(vc, vs, table, b, j)).half())
        assert torch.equal(gk[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(slots_of(kc, ks, table, b, j)).half())
    lens = [int(x) for x in lens + new]
    q = torch.randn(batch, 4, d).bfloat16().cuda()
    o, lse = ab.attn_decode8(q, kc, vc, ks, vs, table, ints(lens))
    ab.check_device_status()
    check_decode8(o, lse, q, kc, vc, ks, vs, table, lens, d ** -0.5)


@pytest.mark.parametrize("inter", [False, True])
def test_append_and_load_on_a_stream_and_in_a_graph(inter):
    kind, page, hk, d = "int8", 16, 2, 64
    kc, vc, ks, vs, table = make_cache8(80, 3, hk, d, page, 8, kind, 19)
    q, k, v = (torch.randn(9, h, d).half().cuda() for h in (4, hk, hk))
    n, cu, pos, inv = ints([3, 40, 7]), ints([0, 4, 5, 9]), ints(list(range(9))), torch.rand(32, device="cuda")
    twin = [x.clone() for x in (kc, vc, ks, vs)]

    def run(cache, stream=None):
        got = ab.attn_cache_append8(k, v, *cache, table, n, cu, q=q, positions=pos, inv_freq=inv, interleaved=inter,
                                    stream=stream)
        return got, *ab.attn_cache_load8(*cache, table, n, cu, 9, dtype=torch.float16, stream=stream)

    want = run(twin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run((kc, vc, ks, vs), side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run((kc, vc, ks, vs))
    for old in ([0, 9, 64], [5, 5, 5]):
        n.copy_(ints(old))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape))
        graph.replay()
        want = run(twin)
        ab.check_device_status()
        for x, y in zip((*got, kc, vc, ks, vs), (*want, *twin)):
            assert torch.equal(x, y)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind,dt,hf", [("e4m3", "bf16", False), ("int8", "fp16", True)])
def test_beams_over_an_8_bit_cache(kind, dt, hf):
    """Prompts, forked into beams that change places, end and start again: every step makes room,
    copies the pages that two beams would write, appends a token each and attends."""
    dtype, page, block, hq, hk, d = DT[dt], 8, 4, 6, 2, 64
    rows, width, pages = 6, 12, 60
    rng = np.random.default_rng(3)
    kc, vc, ks, vs, _ = make_cache8(page, pages - 2, hk, d, page, block, kind, 17, hf)
    assert kc.shape[0] == pages
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0] * rows), ints([0] * pages)
    inv = (1.0 / 100.0 ** (torch.arange(32) / 32)).float().cuda()
    history = [[] for _ in range(rows)]  # (k, v) of each token, as given, rotated
    sizes = [13, 20, 1, 0, 0, 0]
    steps = [(sizes, list(range(rows)))] + [([1] * rows, p) for p in
             ([0, 0, 0, 1, 1, 2], [2, 1, 1, 5, 5, 5], [0, -1, 2, 3, -1, 5], [0, 0, 3, 3, 3, 5], [5, 4, 3, 2, 1, 0])]
    for new, parents in steps:
        if new is not sizes:
            new = [0 if p < 0 else 1 for p in parents]
        _, _, _, copies, counts = ab.attn_cache_fork(table, lens, refs, page, parents=ints(parents), room=ints(new))
        ab.attn_cache_copy(kc, vc, copies, counts, ks, vs)
        history = [list(history[p]) if p >= 0 else [] for p in parents]
        cu = np.concatenate([[0], np.cumsum(new)])
        t = int(cu[-1])
        q, k, v = (torch.from_numpy(rng.standard_normal((t, h, d))).to(dtype).cuda() for h in (hq, hk, hk))
        pos = [len(history[b]) + i for b in range(rows) for i in range(new[b])]
        rq = ab.attn_cache_append8(k, v, kc, vc, ks, vs, table, lens, ints(cu), q=q, positions=ints(pos), inv_freq=inv)
        rk = co.rope(f64(k), [pos], inv.cpu().numpy(), (32,))
        for b in range(rows):
            history[b] += [(rk[i], f64(v[i])) for i in range(cu[b], cu[b + 1])]
        lens += ints(new)
        ab.check_device_status()
        assert lens.tolist() == [len(h) for h in history]
        held = table[table >= 0].cpu().numpy()
        assert np.array_equal(np.bincount(held, minlength=pages), refs.cpu().numpy())
        assert counts[1].item() == (refs == 0).sum().item()
        last = torch.zeros(rows, hq, d, dtype=dtype, device="cuda")
        for b in range(rows):
            if new[b]:
                last[b] = rq[cu[b + 1] - 1]
        o, lse = ab.attn_decode8(last, kc, vc, ks, vs, table, lens)
        ab.check_device_status()
        check_decode8(o, lse, last, kc, vc, ks, vs, table, lens.tolist(), d ** -0.5)
        # what the cache holds is what was appended, to a step of the block's factor
        for b, h in enumerate(history):
            if h:
                for codes, s, which in ((kc, ks, 0), (vc, vs, 1)):
                    got = slots_of(codes, s, table, b, range(len(h)))
                    want = np.stack([x[which] for x in h])
                    f = slots_of(torch.ones_like(codes.float()).to(codes.dtype), s, table, b, range(len(h)))
                    # rounded once and, where the factor grew, again: with e4m3 a step is 2^-3 of the value
                    # or 2^-9 of the factor, and each of the growths rounds to at most half the last step
                    bound = f * 1.0 + 2.0 ** -16 if kind == "int8" else np.abs(want) * 2.0 ** -3 + f * 2.0 ** -8
                    assert (np.abs(got - want) <= bound).all()
    # a chunk of a prompt attends a prefix that is read back
    n = lens.tolist()
    cu = np.concatenate([[0], np.cumsum(n)])
    k, v = ab.attn_cache_load8(kc, vc, ks, vs, table, ints([0] * rows), ints(cu), int(cu[-1]), dtype=dtype)
    ab.check_device_status()
    for b in range(rows):
        assert torch.equal(k[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(slots_of(kc, ks, table, b, range(n[b]))).to(dtype))
        assert torch.equal(v[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(slots_of(vc, vs, table, b, range(n[b]))).to(dtype))
