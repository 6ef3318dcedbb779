"""Pages that a row which goes on would write while others hold them, too: after a length was lowered into
a page that a fork had shared, or where the caller holds a reference."""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8
from tests.cache8_helpers import KIND

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device="cuda")


def check(table, lens, refs, page, parents, room, share, got):
    """Against the oracle, and what an append relies on."""
    t, n, r, copies, counts = got
    want_t, want_n, want_r, made, free, missing = c8.fork(table, lens, refs, page, parents, room, share)
    assert not missing
    assert np.array_equal(n.cpu().numpy(), want_n)
    assert np.array_equal(t.cpu().numpy(), want_t)
    assert np.array_equal(r.cpu().numpy(), want_r)
    assert counts.tolist() == [len(made), free]
    assert copies[:len(made)].tolist() == [list(map(int, m)) for m in made]
    for b, s in enumerate(parents):
        if s >= 0:
            held = want_t[b, want_n[b] // page:-(-(want_n[b] + room[b]) // page)]
            assert (want_r[held[held >= 0]] == 1).all()
            assert (held >= 0).all()


@pytest.mark.parametrize("rows,width,page,pages", [(6, 8, 4, 200), (40, 20, 8, 3000), (300, 300, 1, 120000),
                                                   (513, 40, 16, 30000), (8200, 3, 16, 60000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_after_lengths_were_lowered(rows, width, page, pages, in_place):
    rng = np.random.default_rng(rows)
    table, refs, at = np.full((rows, width), -1), np.zeros(pages, int), iter(rng.permutation(pages))
    lens = rng.integers(0, width * page - page + 1, rows)
    for b in range(rows):
        for i in range(-(-lens[b] // page)):
            table[b, i] = next(at)
            refs[table[b, i]] = 1
    state = (ints(table), ints(lens), ints(refs))
    given_up = 0
    for step in range(6):
        parents = rng.integers(-1 if step % 3 == 2 else 0, rows, rows) if step % 2 == 0 else np.arange(rows)
        room = rng.integers(0, page + 2, rows)
        room = np.minimum(room, width * page - np.where(parents >= 0, lens[parents], 0))
        outs = {} if in_place else dict(zip(("table_out", "seqlens_out", "refs_out"), (torch.full_like(x, 77) for x in state)))
        got = ab.attn_cache_fork(*state, page, parents=ints(parents), room=ints(room), **outs)
        ab.check_device_status()
        check(table, lens, refs, page, parents, room, True, got)
        if not in_place:
            for x, y in zip(state, (table, lens, refs)):
                assert np.array_equal(x.cpu().numpy(), y)
        heirs = {int(s): b for b, s in reversed(list(enumerate(parents))) if s >= 0}
        state = got[:3]
        old = table
        table, lens, refs = (x.cpu().numpy().astype(int) for x in state)
        given_up += sum(((table[b] != old[s]) & (old[s] >= 0)).any() for s, b in heirs.items())
        assert np.array_equal(np.bincount(table[table >= 0], minlength=pages), refs)
        lens = np.maximum(lens - rng.integers(0, 3 * page, rows) * (rng.random(rows) < 0.5), 0)  # some roll back
        state = (state[0], ints(lens), state[2])
    assert given_up > 0


def test_fork_leaves_pages_that_the_caller_holds():
    # page 2, partly full, is also the caller's: a row that goes on writes a copy of it
    table, refs = np.array([[5, 2, -1, -1]]), np.zeros(9, int)
    refs[[5, 2]] = [1, 2]
    got = ab.attn_cache_fork(ints(table), ints([6]), ints(refs), 4, room=3)
    ab.check_device_status()
    assert got[0].tolist() == [[5, 0, 1, -1]] and got[2].tolist() == [1, 1, 1, 0, 0, 1, 0, 0, 0]
    assert got[4].tolist() == [1, 5] and got[3][:1].tolist() == [[2, 0]]
    check(table, [6], refs, 4, [0], [3], True, got)
    # a page given up that nobody holds any more is free for the next call
    table, refs = np.array([[5, 2, 7, 8]]), np.zeros(9, int)
    refs[[5, 2, 7, 8]] = [1, 1, 2, 1]
    got = ab.attn_cache_fork(ints(table), ints([6]), ints(refs), 4, room=3)
    ab.check_device_status()
    assert got[0].tolist() == [[5, 0, 1, -1]] and got[2].tolist() == [1, 1, 0, 0, 0, 1, 0, 1, 0]
    check(table, [6], refs, 4, [0], [3], True, got)
    # a full page that others hold stays shared, whatever the room
    table, refs = np.array([[5, 2, -1, -1]]), np.zeros(9, int)
    refs[[5, 2]] = [2, 2]
    got = ab.attn_cache_fork(ints(table), ints([8]), ints(refs), 4, room=1)
    assert got[0].tolist() == [[5, 2, 0, -1]] and got[4].tolist() == [0, 6]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_rolled_back_rows_do_not_touch_their_siblings(kind):
    """Drafts are taken back into a page that a fork had shared; the next append re-rounds and writes its
    copy, and the sibling reads what it read before."""
    page, block, hk, d, pages = 8, 4, 2, 64, 20
    kc, vc = (torch.zeros(pages, page, hk, d).to(KIND[kind]).cuda() for _ in range(2))
    ks, vs = (torch.ones(pages, page // block, hk, device="cuda") for _ in range(2))
    table = torch.full((2, 5), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0, 0]), ints([0] * pages)

    def step(parents, room):
        _, _, _, copies, counts = ab.attn_cache_fork(table, lens, refs, page, parents=ints(parents), room=ints(room))
        ab.attn_cache_copy(kc, vc, copies, counts, ks, vs)

    def append(new, size):
        cu = np.concatenate([[0], np.cumsum(new)])
        k, v = size * torch.randn(2, int(cu[-1]), hk, d, generator=torch.Generator().manual_seed(int(size)))
        ab.attn_cache_append8(k.half().cuda(), v.half().cuda(), kc, vc, ks, vs, table, lens, ints(cu))
        lens.add_(ints(new))

    def read(b):
        n = int(lens[b])
        return ab.attn_cache_load8(kc, vc, ks, vs, table, ints([0, 0]), ints([0, n, n] if b == 0 else [0, 0, n]), n,
                                   dtype=torch.float16)

    step([0, 1], [16, 0])
    append([16, 0], 1.0)
    step([0, 0], [0, 0])           # both hold both pages
    for n in (11, 3, 8):           # the second takes tokens back
        lens.copy_(ints([16, n]))
        before = read(0)
        step([0, 1], [0, 3])
        append([0, 3], 100.0)      # the block's factor grows
        ab.check_device_status()
        assert all(torch.equal(x, y) for x, y in zip(before, read(0)))
        assert all(x[n:].abs().max() > 100 for x in read(1))
        step([0, 0], [0, 0])
