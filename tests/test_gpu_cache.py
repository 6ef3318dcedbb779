"""The paged cache on the GPU: append, single-token attention, eviction, and the three
as a serving loop, against the 64-bit oracle.

Bad pages and lengths below are given in arrays of their full size: the kernels look at
an entry before they use it, so nothing is read or written out of range.
"""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache_oracle as co
from tests.cache_helpers import (DT, HALF_STEP, SMALLEST, check_decode, f64, make_cache, put_rows, rows_of)

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

APPEND = [
    # dtype, old lengths, new lengths, hq, hk, D, page, heads_first, n_freq, sections, interleaved
    ("bf16", [0], [1], 1, 1, 64, 16, False, 32, (32,), False),
    ("fp16", [5, 0, 63, 17], [3, 0, 65, 1], 4, 2, 128, 16, False, 64, (16, 24, 24), False),
    ("bf16", [7, 0, 200], [0, 300, 29], 6, 2, 80, 48, True, 20, (12, 8), True),
    ("fp16", [1, 2, 3], [5, 40, 1], 2, 2, 72, 1, False, 11, (5, 6), False),
    ("bf16", [100] * 9, [1] * 9, 32, 8, 128, 64, False, 64, (64,), False),
    ("bf16", [0, 12], [700, 900], 16, 16, 256, 100, True, 128, (128,), True),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[0]}-{len(c[1])}seq-d{c[5]}-p{c[6]}" for c in APPEND])
def test_append_stores_rotated_keys_and_values(case):
    dt, old, new, hq, hk, d, page, hf, n, sec, inter = case
    dt = DT[dt]
    g = torch.Generator().manual_seed(2)
    cu = np.concatenate([[0], np.cumsum(new)])
    t = int(cu[-1]) + 2  # two tokens behind the last sequence
    caps = [a + b for a, b in zip(old, new)]
    kc, vc, table = make_cache(caps, hk, d, page, dt, 3, hf)
    k0, v0 = kc.clone(), vc.clone()
    q, k, v = (torch.randn(t, h, d, generator=g).to(dt) for h in (hq, hk, hk))
    pos = torch.randint(0, 3000, (len(sec), t), generator=g, dtype=torch.int32)
    inv = (1.0 / 500.0 ** (torch.arange(n) / n)).float()
    width = max(caps) + 3
    slots = torch.full((len(old), hk, width), -7, dtype=torch.int32, device="cuda")
    seen = [x + 11 for x in old]
    oq = torch.full_like(q, 5.0).cuda()
    got = ab.attn_cache_append(k.cuda(), v.cuda(), kc, vc, table, ints(old), ints(cu), q=q.cuda(),
                               positions=pos.cuda(), inv_freq=inv.cuda(), sections=sec, interleaved=inter,
                               out_q=oq, slot_positions=slots, seen=ints(seen))
    ab.check_device_status()
    assert got is oq
    rk = co.rope(f64(k), pos.numpy(), inv.numpy(), sec, inter)
    rq = co.rope(f64(q), pos.numpy(), inv.numpy(), sec, inter)
    want_k, want_v = f64(k0), f64(v0)
    want_s = np.full((len(old), hk, width), -7)
    tab = table.cpu().numpy()
    place = co.append_slots(cu, old, t)
    touched = np.zeros(want_k.shape[:2], bool)
    for i, at in enumerate(place):
        if at is None:
            assert (f64(oq[i]) == 5.0).all()
            continue
        b, j, nth = at
        p, w = co.slot(tab[b], page, j)
        want_k[p, w], want_v[p, w] = rk[i], f64(v[i])
        want_s[b, :, j] = seen[b] + nth
        touched[p, w] = True
    def near(x, ref, amp):
        bound = HALF_STEP[dt] * np.abs(ref) + 2.0 ** -19 * amp + SMALLEST[dt]
        return (np.abs(x - ref) <= bound).all()
    gk = f64(kc)
    amp = 2 * max(np.abs(f64(k)).max(), np.abs(f64(q)).max())
    assert near(gk[touched], want_k[touched], amp)
    assert np.array_equal(gk[~touched], want_k[~touched])
    assert np.array_equal(f64(vc), want_v)
    assert np.array_equal(slots.cpu().numpy(), want_s)
    live = [i for i, at in enumerate(place) if at is not None]
    assert near(f64(oq)[live], rq[live], amp)


def test_append_without_rotation_one_token_each():
    kc, vc, table = make_cache([20, 20, 20], 2, 64, 8, torch.float16, 4)
    k, v = torch.randn(2, 3, 2, 64).half().cuda()
    old = [0, 7, 15]
    assert ab.attn_cache_append(k, v, kc, vc, table, ints(old)) is None
    ab.check_device_status()
    for b, n in enumerate(old):
        assert torch.equal(rows_of(kc, table, b, n + 1)[n], k[b])
        assert torch.equal(rows_of(vc, table, b, n + 1)[n], v[b])


def test_append_leaves_out_what_does_not_fit_and_reports_it():
    kc, vc, table = make_cache([16, 16, 16, 16], 2, 64, 8, torch.float16, 5)
    k0 = kc.clone()
    table[1, 1] = kc.shape[0]      # a page that does not exist
    table[2, 0] = -1
    k, v = torch.randn(2, 4, 2, 64).half().cuda()
    ab.attn_cache_append(k, v, kc, vc, table, ints([3, 9, 0, 16]))  # the last one is full
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert e.value.code == -9
    ab.check_device_status()  # cleared
    p = int(table[0, 0])
    assert torch.equal(kc[p, 3], k[0])
    k0[p, 3] = k[0]
    assert torch.equal(kc, k0)
    # lengths below zero, and offsets that descend
    for lens, cu, t in (([-1, 0, 0, 0], None, 4), ([0] * 4, [0, 3, 2, 4, 4], 4)):
        k2 = kc.clone()
        v2 = vc.clone()
        good = make_cache([16] * 4, 2, 64, 8, torch.float16, 5)[2]
        ab.attn_cache_append(k[:t], v[:t], k2, v2, good, ints(lens), None if cu is None else ints(cu))
        with pytest.raises(ab.AttnError) as e:
            ab.check_device_status()
        assert e.value.code == -9
    # a report here does not stop varlen calls, unlike a failed cu_seqlens check there
    ab.attn_cache_append(k, v, kc, vc, table, ints([3, 9, 0, 16]))
    q = torch.randn(6, 2, 64).half().cuda()
    o, _ = ab.attn_fwd(q, q, q, cu_seqlens_q=ints([0, 6]), cu_seqlens_k=ints([0, 6]), max_seqlen_q=6,
                       max_seqlen_k=6, out=torch.full_like(q, float("nan")))
    torch.cuda.synchronize()
    assert o.isfinite().all()
    with pytest.raises(ab.AttnError):
        ab.check_device_status()


# ------------------------------------------------------------------ decode

DECODE = [
    # dtype, lengths, hq, hk, D, page, heads_first, window, cap
    ("fp16", [1], 1, 1, 64, 16, False, -1, 0.0),
    ("bf16", [0, 1, 2, 15, 16, 17, 63, 64, 65], 4, 2, 64, 16, False, -1, 0.0),
    ("fp16", [128], 2, 2, 64, 16, True, -1, 0.0),
    ("bf16", [300, 0, 1, 1000], 32, 8, 128, 64, False, -1, 0.0),
    ("fp16", [257, 31], 20, 1, 96, 48, False, -1, 0.0),      # groups above 16
    ("bf16", [129, 700], 48, 2, 128, 32, True, -1, 30.0),
    ("fp16", [500, 3], 6, 2, 80, 1, False, -1, 0.0),         # pages of one slot
    ("bf16", [90, 1100], 5, 1, 72, 100, False, 64, 0.0),
    ("fp16", [1, 2, 1300, 200], 16, 16, 256, 48, False, 1024, 30.0),
    ("bf16", [33, 640], 8, 8, 192, 128, True, 0, 0.0),       # a window of one slot
    ("fp16", [77, 401], 3, 3, 8, 7, False, -1, 20.0),
    ("bf16", [2500], 8, 1, 248, 256, False, 2000, 0.0),
    ("bf16", [6000], 8, 2, 64, 16, False, -1, 0.0),          # split over the length
    ("fp16", [1 + (i * 37) % 300 for i in range(70)], 4, 2, 32, 16, False, -1, 0.0),
    ("bf16", [6000, 77], 12, 2, 88, 16, True, -1, 0.0),
    ("fp16", [3, 5000, 900], 20, 10, 96, 1, False, 4000, 15.0),
]


def _decode_inputs(lens, hq, hk, d, page, hf, dt, seed=11, fill_rest=float("nan")):
    """Slots behind each length, and pages of nobody, hold NaN."""
    kc, vc, table = make_cache([max(1, n) for n in lens], hk, d, page, dt, seed, hf, fill=fill_rest)
    g = torch.Generator().manual_seed(seed + 1)
    for b, n in enumerate(lens):
        for c in (kc, vc):
            put_rows(c, table, b, torch.randn(n, hk, d, generator=g).to(dt).cuda())
    q = torch.randn(len(lens), hq, d, generator=g).to(dt).cuda()
    return q, kc, vc, table


@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("case", DECODE, ids=[f"{c[0]}-{len(c[1])}seq-h{c[2]}/{c[3]}-d{c[4]}-p{c[5]}" for c in DECODE])
def test_decode_matches_the_oracle(case, weights):
    dt, lens, hq, hk, d, page, hf, window, cap = case
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, page, hf, DT[dt])
    width = max(lens) + 5
    w0 = torch.rand(len(lens), hk, width, device="cuda") if weights else None
    w = w0.clone() if weights else None
    most = max(1, max(lens)) if hf else None
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens), max_seqlen=most if most else max(lens),
                            window=None if window < 0 else (window, -1), softcap=cap, weights=w)
    ab.check_device_status()
    check_decode(o, lse, q, kc, vc, table, lens, d ** -0.5, window, cap, w, w0)


MANY = [
    # batch, length of sequence i, hq, hk, D, page, window: more sequences than a block has
    # threads or keeps lengths of, empty ones among them; and heads that do and do not divide
    # the blocks, up to more heads than blocks
    (700, lambda i: (i * 29) % 45 if i % 7 else 0, 4, 2, 64, 16, -1),
    (400, lambda i: 300 + i % 3 if i % 50 == 0 else (i * 7) % 12, 6, 3, 128, 16, -1),
    (330, lambda i: 0 if i < 300 else 260 + i, 2, 1, 64, 64, 500),
    (2, lambda i: 700 * i + 30, 40, 40, 64, 32, -1),
    (2, lambda i: 500 * i + 9, 70, 35, 96, 32, -1),
    (1, lambda i: 600, 320, 320, 16, 16, -1),
    (2, lambda i: 290 + i, 130, 65, 192, 16, -1),
]


@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("case", MANY, ids=[f"{c[0]}seq-h{c[2]}/{c[3]}-d{c[4]}" for c in MANY])
def test_decode_of_many_sequences_and_heads(case, weights):
    batch, length, hq, hk, d, page, window = case
    lens = [length(i) for i in range(batch)]
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, page, False, torch.bfloat16)
    w0 = torch.rand(batch, hk, max(lens), device="cuda") if weights else None
    w = w0.clone() if weights else None
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens), max_seqlen=max(lens),
                            window=None if window < 0 else (window, 0), weights=w)
    ab.check_device_status()
    check_decode(o, lse, q, kc, vc, table, lens, d ** -0.5, window, 0.0, w, w0)


@pytest.mark.parametrize("window", [-1, 900])
def test_decode_weights_of_long_among_many_under_a_loose_bound(window):
    """A block of the weights' kernel takes more than one stretch of its keys."""
    batch, hq, hk, d, page, top = 320, 16, 8, 64, 16, 3000
    lens = [1300 + i if i % 40 == 3 else i % 11 for i in range(batch)]
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, page, False, torch.float16)
    wide = torch.full((batch, -(-top // page)), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    w0, w1 = torch.rand(batch, hk, top, device="cuda"), torch.full((batch, hk, top), -3.0, device="cuda")
    o, lse = ab.attn_decode(q, kc, vc, wide, ints(lens), window=None if window < 0 else (window, 0),
                            max_seqlen=top, weights=w0, weights_out=w1)
    ab.check_device_status()
    base = w0.clone()
    for b, n in enumerate(lens):
        base[b, :, n:] = -3.0
    check_decode(o, lse, q, kc, vc, wide, lens, d ** -0.5, window, weights=w1, weights_in=base)


def test_pages_behind_2_to_the_32_elements():
    """A cache of more than 2^32 elements (10 GB, keys and values in the same pages): append,
    decode and evict on its last pages."""
    page, hk, d, pages = 256, 8, 64, 33200  # 4.35e9 elements
    dt, lens, budget = torch.float16, [300, 40], 100
    pool = torch.empty(pages, page, hk, d, dtype=dt, device="cuda")
    assert pool.numel() > 2**32
    table = ints([[pages - 1, pages - 3], [pages - 2, pages - 4]])
    g = torch.Generator().manual_seed(40)
    k = torch.randn(340, hk, d, generator=g).to(dt).cuda()
    ab.attn_cache_append(k, k, pool, pool, table, ints([0, 0]), ints([0, 300, 340]))
    ab.check_device_status()
    assert torch.equal(pool[pages - 1], k[:256]) and torch.equal(pool[pages - 3, :44], k[256:300])
    assert torch.equal(pool[pages - 2, :40], k[300:])
    q = torch.randn(2, 16, d, generator=g).to(dt).cuda()
    o, lse = ab.attn_decode(q, pool, pool, table, ints(lens), max_seqlen=300)
    ab.check_device_status()
    check_decode(o, lse, q, pool, pool, table, lens, d ** -0.5)
    w = torch.rand(2, hk, 300, generator=g)
    before = rows_of(pool, table, 0, 300).clone()
    n2, _, _ = ab.attn_cache_evict(pool, pool, table, ints(lens), w.cuda(), budget, max_seqlen=300)
    ab.check_device_status()
    assert n2.tolist() == [100, 40]
    after = rows_of(pool, table, 0, 300)
    for h in range(hk):
        kept = co.keep(w[0, h].numpy(), None, 0, budget, 0)
        want = before[:, h].clone()
        for a, z in co.moves(kept, budget):
            want[z] = before[a, h]
        assert torch.equal(after[:, h], want)


def test_decode_outputs_and_weights_in_other_arrays_and_strides():
    lens, hq, hk, d = [40, 170], 4, 2, 64
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, 16, False, torch.bfloat16)
    wide = torch.randn(2, hq, 2 * d).to(torch.bfloat16).cuda()
    wide[:, :, :d] = q
    out = torch.full((hq, 2, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.empty(2, hq, device="cuda")
    w0, w1 = torch.rand(2, hk, 200, device="cuda"), torch.full((2, hk, 200), -3.0, device="cuda")
    keep = w0.clone()
    o, l2 = ab.attn_decode(wide[:, :, :d], kc, vc, table, ints(lens), max_seqlen=176, scale=0.2,
                           out=out, lse=lse, weights=w0, weights_out=w1)
    ab.check_device_status()
    assert o is out and l2 is lse and torch.equal(w0, keep)
    base = w0.clone()
    for b, n in enumerate(lens):
        base[b, :, n:] = -3.0
    check_decode(o, lse, q, kc, vc, table, lens, 0.2, weights=w1, weights_in=base)


def test_decode_keys_of_the_lowest_value_and_infinite_values():
    """Logits at the type's lowest finite value, and an infinity that a masked slot holds."""
    lens, hq, hk, d = [50], 2, 2, 64
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, 16, False, torch.bfloat16, fill_rest=float("inf"))
    q.fill_(1.0)
    rows = rows_of(kc, table, 0, 50)
    rows[:] = torch.finfo(torch.bfloat16).min / 128  # sums to the lowest of fp32's range
    rows[17] = torch.finfo(torch.bfloat16).min / 256
    put_rows(kc, table, 0, rows)
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens), scale=1.0)
    ab.check_device_status()
    assert torch.equal(o[0], rows_of(vc, table, 0, 50)[17])  # all weight on one key
    # every logit equal and huge: the mean of the values
    rows[17] = rows[0]
    put_rows(kc, table, 0, rows)
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens), scale=1.0)
    v = f64(rows_of(vc, table, 0, 50))
    bound = 2.0 ** -8 * np.abs(v.mean(0)) + (2.0 ** -8 + 2.0 ** -15) * np.abs(v).mean(0)
    assert (np.abs(f64(o[0]) - v.mean(0)) <= bound).all()


def test_decode_nan_in_a_key_reaches_its_heads_alone():
    lens, hq, hk, d = [50, 30], 4, 2, 64
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, 16, False, torch.float16, fill_rest=0.0)
    rows = rows_of(kc, table, 0, 50)
    rows[20, 1, 3] = float("nan")
    put_rows(kc, table, 0, rows)
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens))
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert o[0, :2].isfinite().all() and o[1].isfinite().all()


def test_decode_bad_lengths_and_pages_are_reported():
    lens, hq, hk, d = [40, 40, 40, 40], 2, 1, 64
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, 8, False, torch.float16, fill_rest=0.0)
    for bad in ([40, -1, 40, 40], [40, 41, 40, 40]):
        w = torch.zeros(4, hk, 64, device="cuda")
        o, lse = ab.attn_decode(q, kc, vc, table, ints(bad), max_seqlen=40, weights=w)
        with pytest.raises(ab.AttnError) as e:
            ab.check_device_status()
        assert e.value.code == -9 and "length" in str(e.value)
        assert (o[1] == 0).all() and torch.isposinf(lse[1]).all() and (w[1] == 0).all()
        check_decode(o[2:], lse[2:], q[2:], kc, vc, table[2:], lens[2:], d ** -0.5)
    # the keys of a page that does not exist take no part
    table[3, 2] = 1 << 30
    table[3, 4] = -5
    o, lse = ab.attn_decode(q, kc, vc, table, ints(lens), max_seqlen=40)
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert e.value.code == -9 and "page" in str(e.value)
    check_decode(o[:3], lse[:3], q[:3], kc, vc, table[:3], lens[:3], d ** -0.5)
    t = table.clone()
    t[3, :3] = table[3, [0, 1, 3]]
    check_decode(o[3:], lse[3:], q[3:], kc, vc, t[3:], [24], d ** -0.5)


def test_decode_gives_the_same_bits_again_and_on_replay():
    lens, hq, hk, d = [3000, 1, 0, 777, 64], 16, 2, 128
    q, kc, vc, table = _decode_inputs(lens, hq, hk, d, 64, False, torch.bfloat16)
    n = ints(lens)
    w0 = torch.rand(5, hk, 3008, device="cuda")
    w = torch.empty_like(w0)
    a = ab.attn_decode(q, kc, vc, table, n, max_seqlen=3000, weights=w0, weights_out=w)
    ws = ab.alloc_decode_workspace(q, kc, 3000, weights=True)
    ws.fill_(255)  # what the workspace held does not matter
    w2 = torch.empty_like(w0)
    out, lse = torch.empty_like(q), torch.empty(5, hq, device="cuda")
    kw = dict(max_seqlen=3000, weights=w0, weights_out=w2, out=out, lse=lse, workspace=ws)
    ab.attn_decode(q, kc, vc, table, n, **kw)
    for b, m in enumerate(lens):
        assert torch.equal(w[b, :, :m], w2[b, :, :m])
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ab.attn_decode(q, kc, vc, table, n, **kw)
    # shorter lengths, other queries and another workspace content at replay
    new = [17, 0, 2999, 5, 300]
    n.copy_(ints([min(x, y) for x, y in zip(new, lens)]))
    new = n.tolist()
    q.copy_(torch.randn(q.shape).to(q.dtype))
    ws.fill_(127)
    g.replay()
    torch.cuda.synchronize()
    ab.check_device_status()
    base = w0.clone()
    for b, m in enumerate(new):
        base[b, :, m:] = w2[b, :, m:]
    check_decode(out, lse, q, kc, vc, table, new, d ** -0.5, weights=w2, weights_in=base)


def test_lengths_beyond_32_bits_are_refused():
    lens, hq, hk, d, page, dt = [20, 9], 4, 2, 64, 8, torch.float16
    q = torch.randn(2, hq, d, dtype=dt, device="cuda")
    kc, vc, table = make_cache(lens, hk, d, page, dt, 3)
    for kw in (dict(max_seqlen=2**32 + 5), dict(window=(2**32, -1))):
        with pytest.raises(ab.AttnError):
            ab.attn_decode(q, kc, vc, table, ints(lens), **kw)
    w = torch.zeros(2, hk, 24, device="cuda")
    for budget, recent in ((2**32 + 5, 0), (5, 2**32)):
        with pytest.raises(ab.AttnError):
            ab.attn_cache_evict(kc, vc, table, ints(lens), w, budget, recent, max_seqlen=20)


def test_append_offsets_far_below_zero_are_reported():
    kc, vc, table = make_cache([16, 16], 2, 64, 8, torch.float16, 5)
    k0, v0 = kc.clone(), vc.clone()
    k, v = torch.randn(2, 4, 2, 64).half().cuda()
    # the last one's place in its sequence passes 2^31
    for first in (-1, -2**31):
        ab.attn_cache_append(k, v, kc, vc, table, ints([0, 0]), ints([first, 4, 4]))
        with pytest.raises(ab.AttnError) as e:
            ab.check_device_status()
        assert e.value.code == -9
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_decode_on_two_streams_at_once():
    lens, hq, hk, d = [900, 40], 8, 2, 64
    sets = [_decode_inputs(lens, hq, hk, d, 16, False, torch.float16, seed=s) for s in (21, 22)]
    streams = [torch.cuda.Stream() for _ in sets]
    n = ints(lens)
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(5):
        for i, (x, s) in enumerate(zip(sets, streams)):
            got[i].append(ab.attn_decode(*x, n, stream=s))
    torch.cuda.synchronize()
    for x, r in zip(sets, got):
        for o, lse in r:
            check_decode(o, lse, *x, lens, d ** -0.5)


# ------------------------------------------------------------------ eviction

EVICT = [
    # dtype, lengths, hk, D, page, heads_first, budget, recent
    ("bf16", [10, 5, 3, 0], 2, 64, 4, False, 4, 2),
    ("fp16", [100, 64, 65, 1], 3, 80, 16, True, 64, 0),
    ("bf16", [2000, 1500], 2, 128, 48, False, 500, 100),
    ("fp16", [5000], 1, 256, 1, False, 4097, 4097),   # recent = budget
    ("bf16", [1088] * 6, 4, 8, 64, False, 1024, 128),
    ("fp16", [777, 3], 2, 64, 100, False, 1, 1),
]


def _evict_check(kc, vc, table, lens, w, pos, seen, budget, recent, before, out):
    """Against the oracle; before = (k, v) copies, out = (seqlens, weights, positions)."""
    n2, w2, p2 = (None if t is None else t.cpu().numpy() for t in out)
    page, tab = kc.shape[1], table.cpu().numpy()
    bk, bv = (t.cpu() for t in before)
    wk, wv = bk.clone(), bv.clone()
    for b, n in enumerate(lens):
        m = min(n, budget)
        assert n2[b] == m
        for h in range(kc.shape[2]):
            kept = co.keep(w[b, h, :n], pos[b, h, :n] if pos is not None else None, seen[b], budget, recent)
            ww = w[b, h].copy()
            pp = pos[b, h].copy() if pos is not None else None
            for a, z in co.moves(kept, budget) if n > budget else []:
                s, t = co.slot(tab[b], page, a), co.slot(tab[b], page, z)
                wk[t[0], t[1], h], wv[t[0], t[1], h] = bk[s[0], s[1], h], bv[s[0], s[1], h]
                ww[z] = ww[a]
                if pp is not None:
                    pp[z] = pp[a]
            ww[m:n] = 0
            assert np.array_equal(w2[b, h, :n], ww[:n], equal_nan=True), (b, h)
            if pp is not None:
                pp[m:n] = -1
                assert np.array_equal(p2[b, h, :n], pp[:n]), (b, h)
    assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "apart"])
@pytest.mark.parametrize("ranks", ["spread", "equal", "coarse", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=[f"{c[0]}-{len(c[1])}seq-d{c[3]}-to{c[6]}" for c in EVICT])
def test_evict_matches_the_oracle(case, ranks, inplace):
    dt, lens, hk, d, page, hf, budget, recent = case
    kc, vc, table = make_cache([max(1, n) for n in lens], hk, d, page, DT[dt], 6, hf)
    rng = np.random.default_rng(7)
    width = max(lens) + 3
    shape = (len(lens), hk, width)
    w = {"spread": np.exp(3 * rng.standard_normal(shape)), "equal": np.full(shape, 0.25),
         "coarse": rng.integers(0, 4, shape) / 4.0,
         "odd": rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, -1.0, 2.0], shape)}[ranks].astype(np.float32)
    pos = np.stack([[rng.permutation(width) for _ in range(hk)] for _ in lens]).astype(np.int32)
    seen = [n + 2 for n in lens]
    before = kc.clone(), vc.clone()
    dw, dp, n = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda(), ints(lens)
    kw = {} if inplace else dict(weights_out=torch.full_like(dw, -9.0), positions_out=torch.full_like(dp, -9))
    out = ab.attn_cache_evict(kc, vc, table, n, dw, budget, recent, dp, ints(seen), max_seqlen=max(lens), **kw)
    ab.check_device_status()
    _evict_check(kc, vc, table, lens, w, pos, seen, budget, recent, before, out)
    for b, m in enumerate(lens):  # entries behind the lengths stay
        rest = out[1][b, :, m:].cpu().numpy(), out[2][b, :, m:].cpu().numpy()
        if inplace:
            assert np.array_equal(rest[0], w[b, :, m:], equal_nan=True) and np.array_equal(rest[1], pos[b, :, m:])
        else:
            assert (rest[0] == -9).all() and (rest[1] == -9).all()


LARGE = [
    # one block a head with more slots than it keeps keys of; several blocks a head; eight
    ("bf16", [5000 - 3 * i for i in range(20)], 16, 8, 64, False, 4500, 50),
    ("fp16", [2100 - i for i in range(25)], 4, 8, 16, True, 700, 100),
    ("bf16", [40000, 38001], 2, 8, 100, False, 20000, 1000),
    # eight blocks with more slots than they keep keys of; many heads of several blocks each
    ("fp16", [70001, 5], 1, 8, 64, False, 1000, 10),
    ("bf16", [8700 - i for i in range(20)], 16, 8, 64, False, 8600, 50),
]


@pytest.mark.parametrize("ranks", ["coarse", "odd"])
@pytest.mark.parametrize("case", LARGE, ids=[f"{len(c[1])}seq-h{c[2]}-to{c[6]}" for c in LARGE])
def test_evict_of_long_and_many(case, ranks):
    test_evict_matches_the_oracle(case, ranks, ranks == "coarse")


@pytest.mark.parametrize("batch", [2, 40])
def test_evict_under_a_loose_bound(batch):
    """Lengths far below max_seqlen: some or all but one of a head's blocks leave."""
    lens = ([1500, 300, 90, 2500, 70, 0, 5000, 64] * 5)[:batch]
    hk, d, page, budget, recent, top = 8, 8, 16, 64, 9, 20000
    kc, vc, table = make_cache(lens, hk, d, page, torch.float16, 12)
    wide = torch.full((batch, -(-top // page)), 1 << 30, dtype=torch.int32, device="cuda")  # no such page
    wide[:, :table.shape[1]] = table
    rng = np.random.default_rng(13)
    w = rng.integers(0, 9, (batch, hk, top)).astype(np.float32)
    pos = np.stack([[rng.permutation(top) for _ in range(hk)] for _ in lens]).astype(np.int32)
    seen = [n + 2 for n in lens]
    before = kc.clone(), vc.clone()
    out = ab.attn_cache_evict(kc, vc, wide, ints(lens), torch.from_numpy(w).cuda(), budget, recent,
                              torch.from_numpy(pos).cuda(), ints(seen))
    ab.check_device_status()
    _evict_check(kc, vc, wide, lens, w, pos, seen, budget, recent, before, out)


def test_evict_without_positions_long_and_captured():
    lens, hk, d, budget = [40000, 300], 2, 64, 1000
    kc, vc, table = make_cache(lens, hk, d, 64, torch.bfloat16, 8)
    before = kc.clone(), vc.clone()
    w = np.random.default_rng(9).random((2, hk, 40000)).astype(np.float32)
    dw, n = torch.from_numpy(w).cuda(), ints(lens)
    n2, w2 = torch.empty_like(n), torch.zeros_like(dw)
    ws = ab.alloc_evict_workspace(n, kc, budget, 40000)
    ws.fill_(255)
    kw = dict(weights_out=w2, seqlens_out=n2, workspace=ws)
    ab.attn_cache_evict(kc, vc, table, n, dw, budget, **kw)
    ab.check_device_status()
    _evict_check(kc, vc, table, lens, w, None, [0, 0], budget, 0, before, (n2, w2, None))
    kc.copy_(before[0])
    vc.copy_(before[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ab.attn_cache_evict(kc, vc, table, n, dw, budget, **kw)
    w = np.random.default_rng(10).random(w.shape).astype(np.float32)
    dw.copy_(torch.from_numpy(w))
    g.replay()
    torch.cuda.synchronize()
    _evict_check(kc, vc, table, lens, w, None, [0, 0], budget, 0, before, (n2, w2, None))


def test_evict_reports_bad_lengths_and_pages():
    lens, hk, d, budget = [40, 40, 40], 2, 64, 10
    kc, vc, table = make_cache(lens, hk, d, 8, torch.float16, 12)
    w = np.random.default_rng(1).random((3, hk, 40)).astype(np.float32)
    before = kc.clone(), vc.clone()
    dw = torch.from_numpy(w).cuda()
    n2, w2, _ = ab.attn_cache_evict(kc, vc, table, ints([40, 41, -2]), dw, budget, max_seqlen=40)
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert e.value.code == -9
    assert n2.tolist() == [10, 0, 0]
    assert np.array_equal(w2[1:].cpu().numpy(), w[1:])
    _evict_check(kc, vc, table, [40], w, None, [0], budget, 0, before, (n2, w2, None))
    # a source page that does not exist: its rows are not copied
    kc.copy_(before[0])
    vc.copy_(before[1])
    table[:, 4] = kc.shape[0] + 3
    ab.attn_cache_evict(kc, vc, table, ints(lens), torch.from_numpy(w).cuda(), budget, max_seqlen=40)
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert "page" in str(e.value)


@pytest.mark.parametrize("bad", [4, 0], ids=["source", "target"])
def test_evict_leaves_out_the_rows_of_bad_pages_alone(bad):
    """Rows that would come from or go to a page that does not exist stay out; every other row,
    and all of the state, moves as it would without it."""
    lens, hk, d, budget, page = [40, 40, 37], 2, 64, 10, 8
    kc, vc, table = make_cache(lens, hk, d, page, torch.float16, 12)
    rng = np.random.default_rng(2)
    w = rng.random((3, hk, 40)).astype(np.float32)
    pos = np.stack([[rng.permutation(40) for _ in range(hk)] for _ in lens]).astype(np.int32)
    before = kc.clone(), vc.clone()
    good = table.cpu().numpy().copy()
    table[:2, bad] = torch.tensor([kc.shape[0] + 3, -1], dtype=torch.int32, device="cuda")
    n2, w2, p2 = ab.attn_cache_evict(kc, vc, table, ints(lens), torch.from_numpy(w).cuda(), budget, 0,
                                     torch.from_numpy(pos).cuda(), max_seqlen=40)
    with pytest.raises(ab.AttnError) as e:
        ab.check_device_status()
    assert e.value.code == -9 and "page" in str(e.value)
    ab.check_device_status()
    assert n2.tolist() == [budget] * 3
    want = [t.cpu().clone() for t in before]
    moved = left_out = 0
    for b, n in enumerate(lens):
        for h in range(hk):
            kept = co.keep(w[b, h, :n], None, 0, budget, 0)
            ww, pp = w[b, h].copy(), pos[b, h].copy()
            for a, z in co.moves(kept, budget):
                ww[z], pp[z] = ww[a], pp[a]
                if b < 2 and (a if bad == 4 else z) // page == bad:
                    left_out += 1
                    continue
                moved += 1
                s, t = co.slot(good[b], page, a), co.slot(good[b], page, z)
                for x, old in zip(want, before):
                    x[t[0], t[1], h] = old[s[0], s[1], h].cpu()
            ww[budget:n], pp[budget:n] = 0, -1
            assert np.array_equal(w2[b, h].cpu().numpy(), ww) and np.array_equal(p2[b, h].cpu().numpy(), pp)
    assert moved > 0 and left_out > 0
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


# ------------------------------------------------------------------ together

def test_serving_loop_with_eviction():
    """Prompts enter the cache, tokens are decoded one by one with their weights gathered, and
    the cache is cut back whenever it passes its budget: each step against the oracle run on
    a plain list of slots kept in step."""
    dt, hq, hk, d, page = torch.bfloat16, 8, 2, 64, 16
    prompt, budget, recent, limit = [70, 20, 0], 48, 16, 56
    width, n = 96, 32
    g = torch.Generator().manual_seed(30)
    kc, vc, table = make_cache([width] * 3, hk, d, page, dt, 31, fill=float("nan"))
    inv = (1.0 / 1000.0 ** (torch.arange(n) / n)).float().cuda()
    w = torch.zeros(3, hk, width, device="cuda")
    slots = torch.full((3, hk, width), -1, dtype=torch.int32, device="cuda")
    lens, seen = ints([0, 0, 0]), ints([0, 0, 0])

    def rand(t, h):
        return torch.randn(t, h, d, generator=g).to(dt).cuda()

    cu = [0, 70, 90, 90]
    pos = torch.cat([torch.arange(x) for x in prompt]).to(torch.int32).cuda()
    k, v = rand(90, hk), rand(90, hk)
    ab.attn_cache_append(k, v, kc, vc, table, lens, ints(cu), positions=pos, inv_freq=inv,
                         slot_positions=slots, seen=seen)
    lens += ints(prompt)
    seen += ints(prompt)
    evictions = 0
    for step in range(40):
        q, k, v = rand(3, hq), rand(3, hk), rand(3, hk)
        q = ab.attn_cache_append(k, v, kc, vc, table, lens, q=q, positions=seen.clone(), inv_freq=inv,
                                 slot_positions=slots, seen=seen)
        lens += 1
        seen += 1
        w0 = w.clone()
        o, lse = ab.attn_decode(q, kc, vc, table, lens, max_seqlen=width, weights=w)
        ab.check_device_status()
        now = lens.tolist()
        check_decode(o, lse, q, kc, vc, table, now, d ** -0.5, weights=w, weights_in=w0)
        if max(now) > limit:
            evictions += 1
            before = kc.clone(), vc.clone()
            hw, hp = w.cpu().numpy(), slots.cpu().numpy()
            out = ab.attn_cache_evict(kc, vc, table, lens, w, budget, recent, slots, seen, max_seqlen=width)
            ab.check_device_status()
            page_k = [t.nan_to_num(7.0) for t in (kc, vc, *before)]
            _evict_check(page_k[0], page_k[1], table, now, hw, hp, seen.tolist(), budget, recent,
                         (page_k[2], page_k[3]), out)
            lens = out[0]
            # the newest tokens are all still there
            for b, m in enumerate(lens.tolist()):
                for h in range(hk):
                    held = set(slots[b, h, :m].tolist())
                    assert set(range(int(seen[b]) - min(m, recent), int(seen[b]))) <= held
    assert evictions >= 3
