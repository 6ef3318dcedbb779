"""Pages that sequences share on the GPU: forking, freeing, room and the copy of pages, against
plain loops."""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda() if isinstance(v, np.ndarray) else \
        torch.tensor(v, dtype=torch.int32, device="cuda")


def pool(rng, lens, page, width, pages, shared=0):
    """(table, refs): pages of each sequence at random; the first `shared` full pages of odd rows are
    those of the row before."""
    rows = len(lens)
    table, refs = np.full((rows, width), -1), np.zeros(pages, int)
    at = iter(rng.permutation(pages))
    for b in range(rows):
        for i in range(-(-lens[b] // page)):
            same = b % 2 and i < shared and (i + 1) * page <= min(lens[b], lens[b - 1])
            table[b, i] = table[b - 1, i] if same else next(at)
            refs[table[b, i]] += 1
    return table, refs


def check(table, lens, refs, page, parents, room, share, got, before):
    t, n, r, copies, counts = got
    want_t, want_n, want_r, made, free, missing = c8.fork(table, lens, refs, page, parents, room, share)
    assert np.array_equal(n.cpu().numpy(), want_n)
    assert np.array_equal(t.cpu().numpy(), want_t)
    assert np.array_equal(r.cpu().numpy(), want_r)
    assert counts.tolist() == [len(made), free]
    assert copies[:len(made)].tolist() == [list(map(int, m)) for m in made]
    if before is not None:
        assert torch.equal(copies[len(made):], before[len(made):])
    return missing


CASES = [
    # rows, longest, page, pages, room, share, shared
    (1, 0, 16, 1, 0, True, 0), (1, 1, 1, 4, 1, True, 0), (5, 40, 8, 60, 1, True, 2), (33, 100, 16, 500, 17, True, 3),
    (64, 700, 7, 9000, 3, True, 0), (9, 300, 32, 400, 1, False, 2), (40, 64, 64, 100, 100, False, 0),
    (300, 500, 16, 20000, 1, True, 1), (3, 9000, 1, 40000, 5, False, 0),
    (2100, 60, 16, 9001, 1, True, 2),   # more rows than a block has threads
    (700, 2000, 16, 90001, 20, True, 3), (40, 9000, 3, 121000, 2, False, 0), (1, 100000, 1, 100000, 1, True, 0),
    (8200, 20, 16, 20000, 1, True, 1),   # more rows than shared memory keeps
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}rows-n{c[1]}-p{c[2]}-of{c[3]}-{'share' if c[5] else 'own'}" for c in CASES])
@pytest.mark.parametrize("kind", ["mixed", "stay", "one", "end"])
def test_fork(case, kind):
    rows, longest, page, pages, more, share, shared = case
    rng = np.random.default_rng(rows + longest)
    lens = rng.integers(0, longest + 1, rows)
    width = max(1, -(-(longest + more) // page))
    table, refs = pool(rng, lens, page, width, pages, shared)
    parents = {"mixed": rng.integers(-1, rows, rows), "stay": np.arange(rows), "one": np.full(rows, rng.integers(rows)),
               "end": np.full(rows, -1)}[kind]
    room = rng.integers(0, more + 1, rows)
    most = rows if share else rows * width
    copies = torch.full((most + 1, 2), -9, dtype=torch.int32, device="cuda")
    before = copies.clone()
    a = (ints(table), ints(lens), ints(refs))
    outs = [torch.full_like(x, 77) for x in a]
    got = ab.attn_cache_fork(*a, page, parents=ints(parents), room=ints(room), share=share, table_out=outs[0],
                             seqlens_out=outs[1], refs_out=outs[2], copies=copies)
    missing = check(table, lens, refs, page, parents, room, share, got, before)
    for x, y in zip(a, (table, lens, refs)):
        assert np.array_equal(x.cpu().numpy(), y)  # inputs are left as they were
    for k in range(2):
        if missing:
            with pytest.raises(ab.AttnError):
                ab.check_device_status()
        ab.check_device_status()
        if k == 0:  # in place
            got = ab.attn_cache_fork(*a, page, parents=ints(parents), room=ints(room), share=share)
            assert all(x is y for x, y in zip(got, a))
            check(table, lens, refs, page, parents, room, share, got, None)


def test_fork_without_parents_makes_room_alone():
    table, refs = pool(np.random.default_rng(1), [5, 16, 0], 8, 4, 20)
    got = ab.attn_cache_fork(ints(table), ints([5, 16, 0]), ints(refs), 8, room=4)
    ab.check_device_status()
    check(table, [5, 16, 0], refs, 8, [0, 1, 2], [4] * 3, True, got, None)
    # reserved pages stay: no more are taken while there is room
    t, n, r, _, _ = got
    t0 = t.cpu().numpy().copy()
    ab.attn_cache_fork(t, n, r, 8, room=3)
    assert np.array_equal(t.cpu().numpy(), t0)


def test_fork_keeps_pages_that_others_hold_and_reserved_ones():
    # page 3 is held elsewhere (a reference of the caller's); row 0 has a reserved page beyond its length
    table = np.array([[3, 5, 7, -1], [1, -1, -1, -1]])
    refs = np.zeros(9, int)
    refs[[3, 5, 7, 1]] = [2, 1, 1, 1]
    for parents in ([0, 0], [1, -1], [-1, 0]):
        got = ab.attn_cache_fork(ints(table), ints([6, 2]), ints(refs), 4, parents=ints(parents), room=1)
        ab.check_device_status()
        check(table, [6, 2], refs, 4, parents, [1, 1], True, got, None)
        assert got[2][3] >= 1


def test_fork_reports_what_it_cannot_do():
    table, refs = pool(np.random.default_rng(2), [9, 12, 3], 4, 3, 8)
    args = lambda: (ints(table), ints([9, 12, 3]), ints(refs), 4)  # noqa: E731

    def told():
        with pytest.raises(ab.AttnError) as e:
            ab.check_device_status()
        assert e.value.code == -9
        ab.check_device_status()
        return str(e.value)

    got = ab.attn_cache_fork(*args(), parents=ints([0, 0, 0]), room=1)  # 3 pages free, 6 wanted of row 1's and 2's
    check(table, [9, 12, 3], refs, 4, [0, 0, 0], [1] * 3, True, got, None)
    got = ab.attn_cache_fork(*args(), parents=ints([0, 1, 7]))
    assert "parent" in told()
    check(table, [9, 12, 3], refs, 4, [0, 1, 2], [0] * 3, True, got, None)
    got = ab.attn_cache_fork(*args(), room=1)  # row 1 is full
    assert "length" in told()
    check(table, [9, 12, 3], refs, 4, [0, 1, 2], [1, 0, 1], True, got, None)
    got = ab.attn_cache_fork(ints(table), ints([9, 13, -1]), ints(refs), 4)
    assert "length" in told() and got[1].tolist() == [9, 0, 0]
    broken = table.copy()
    broken[1, 0] = 99
    got = ab.attn_cache_fork(ints(broken), ints([9, 12, 3]), ints(refs), 4, parents=ints([0, 1, 1]))
    assert "page" in told() and got[0][2, 0] == -1 and got[0][2, 1] == int(table[1, 1])
    few = ints(refs)
    few[few == 0] = 1  # no page is free
    got = ab.attn_cache_fork(ints(table), ints([9, 11, 3]), few, 4, parents=ints([0, 1, 1]), room=1)
    # but the one that the old third row leaves
    assert got[4].tolist() == [1, 0] and got[0][2].tolist() == [*table[1, :2].tolist(), table[2, 0]]
    ab.check_device_status()
    few[table[2, 0]] = 2  # which something else holds, too
    few[table[1, 2]] = 1
    got = ab.attn_cache_fork(ints(table), ints([9, 11, 3]), few, 4, parents=ints([0, 1, 1]), room=1)
    assert "no free page" in told() and got[4].tolist() == [0, 0] and got[0][2].tolist() == [*table[1, :2].tolist(), -1]


@pytest.mark.parametrize("pages", [200, 120000])  # one launch, a launch a step
def test_fork_of_strided_tables_in_a_graph(pages):
    rng = np.random.default_rng(4)
    lens, page = rng.integers(1, 60, 8), 8
    table, refs = pool(rng, lens, page, 9, pages)
    big = torch.full((8, 20), 55, dtype=torch.int32, device="cuda")
    t, n, r, who = big[:, 3:12], ints(lens), ints(refs), ints(list(range(8)))
    t.copy_(ints(table))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ab.attn_cache_fork(t, n, r, page, parents=who, room=2)
    for k in range(4):
        parents = rng.integers(-1 if k == 2 else 0, 8, 8)
        table, lens, refs = (x.cpu().numpy().copy() for x in (t, n, r))
        who.copy_(ints(parents))
        graph.replay()
        ab.check_device_status()
        check(table, lens, refs, page, parents, [2] * 8, True, got, None)
        assert (big[:, :3] == 55).all() and (big[:, 12:] == 55).all()


COPY = [
    # dtype, page, heads, D, block, heads_first
    (torch.bfloat16, 64, 8, 128, 0, False), (torch.float16, 1, 1, 8, 0, False), (torch.float16, 16, 4, 72, 0, True),
    (torch.float8_e4m3fn, 64, 8, 128, 16, False), (torch.int8, 48, 3, 80, 1, True), (torch.int8, 7, 2, 16, 7, False),
    (torch.bfloat16, 100, 5, 256, 0, True),
]


@pytest.mark.parametrize("case", COPY, ids=[f"{str(c[0])[6:]}-p{c[1]}-h{c[2]}-d{c[3]}" for c in COPY])
@pytest.mark.parametrize("padded", [False, True])
def test_copy_moves_whole_pages_and_nothing_else(case, padded):
    dtype, page, heads, d, block, hf = case
    pages, pairs = 37, [[3, 8], [3, 9], [36, 0], [5, 35], [12, 12]]
    g = torch.Generator().manual_seed(6)

    def made():
        shape = (pages, heads, page, d) if hf else (pages, page, heads, d)
        extra = 16 if padded else 0
        t = torch.randint(0, 256, (*shape[:3], (d + extra) * (2 if dtype.itemsize == 2 else 1)), generator=g, dtype=torch.uint8)
        t = t.cuda().view(dtype)[..., :d]
        return t.transpose(1, 2) if hf else t

    kc, vc = made(), made()
    f = [torch.rand(pages, page // block, heads, generator=g).cuda() for _ in range(2)] if block else [None, None]
    raw = lambda t: t.contiguous().view(torch.uint8).clone() if t.dtype is not torch.float32 else t.clone()  # noqa: E731
    want = [raw(x) if x is not None else None for x in (kc, vc, *f)]
    counts = ints([4, 0])
    for n, c in ((5, None), (4, counts), (0, ints([-3])), (5, ints([100]))):
        for w in want:
            if w is not None:
                for s, t in pairs[:n]:
                    w[t] = w[s]
        ab.attn_cache_copy(kc, vc, ints(pairs), c, *f)
        ab.check_device_status()
        for x, w in zip((kc, vc, *f), want):
            assert x is None or torch.equal(raw(x), w)
        for x in (kc, vc, *f):  # other contents for the next call
            if x is not None:
                y = x.view(torch.uint8) if x.dtype.itemsize == 1 else x
                y.copy_(y.roll(1, 0))
        want = [raw(x) if x is not None else None for x in (kc, vc, *f)]


def test_copy_reports_bad_pages():
    kc, vc = torch.randn(2, 6, 4, 2, 64).half().cuda()
    k0 = kc.clone()
    ab.attn_cache_copy(kc, vc, ints([[0, 6], [-1, 2], [1, 3]]))
    with pytest.raises(ab.AttnError):
        ab.check_device_status()
    k0[3] = k0[1]
    assert torch.equal(kc, k0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ab.attn_cache_copy(kc, vc, ints([[4, 5]]), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(kc[5], kc[4])


def test_calls_on_a_stream_of_their_own():
    rng = np.random.default_rng(7)
    for pages in (300, 120000):
        lens, page = rng.integers(1, 60, 8), 8
        table, refs = pool(rng, lens, page, 9, pages)
        a = (ints(table), ints(lens), ints(refs))
        parents, twin = rng.integers(0, 8, 8), [x.clone() for x in a]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = ab.attn_cache_fork(*a, page, parents=ints(parents), room=2, stream=side)
        handle = ab.attn_cache_fork(*twin, page, room=0, stream=0)  # the default stream
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        ab.check_device_status()
        check(table, lens, refs, page, parents, [2] * 8, True, got, None)
        assert handle[4][0].item() == 0


def test_copy_of_pages_behind_4_gib():
    pages = 70000
    kc, vc = (torch.zeros(pages, 64, 8, 128, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(pages, 4, 8, device="cuda") for _ in range(2))
    for x in (kc, vc, ks, vs):
        x[pages - 1] = 3
    ab.attn_cache_copy(kc, vc, ints([[pages - 1, 5], [5 + 1, pages - 2]]), None, ks, vs)
    ab.check_device_status()
    for x in (kc, vc, ks, vs):
        assert (x[5] == 3).all() and (x[pages - 1] == 3).all() and (x[4] == x[3]).all()
