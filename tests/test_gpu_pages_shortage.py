"""Forks that want more pages than are free: which rows get them, which copies are listed and what is
reported, in a launch of all steps and in a launch a step."""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache8_oracle as c8

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,width,spare", [(7, 6, 3), (40, 30, 11), (300, 60, 25), (300, 60, 0), (8200, 3, 500)])
@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("rolled_back", [False, True])
def test_fork_when_pages_run_out(rows, width, spare, share, rolled_back):
    page, rng = 4, np.random.default_rng(rows + spare)
    lens = rng.integers(0, width * page - page + 1, rows)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    table, refs, at = np.full((rows, width), -1), np.zeros(pages, int), iter(rng.permutation(pages))
    for b in range(rows):
        for i in range(held[b]):
            table[b, i] = next(at)
            refs[table[b, i]] += 1
    if rolled_back:  # pages that others hold, behind shortened lengths
        refs[rng.permutation(pages)[:pages // 3]] += 1
        lens = np.maximum(lens - rng.integers(0, 2 * page, rows), 0)
    parents = np.where(rng.random(rows) < 0.6, np.arange(rows), rng.integers(0, rows, rows))
    for b in set(range(rows)) - set(parents.tolist()):  # what rows leave stays the caller's, so that it is not free
        refs[table[b, table[b] >= 0]] += 1
    room = np.minimum(rng.integers(0, 2 * page, rows), width * page - lens[parents])
    want_t, want_n, want_r, made, free, missing = c8.fork(table, lens, refs, page, parents, room, share)
    assert missing and free == (want_r == 0).sum()
    most = rows if share else rows * width
    copies = torch.full((most, 2), -9, dtype=torch.int32, device="cuda")
    for outs in ({}, {"table_out": torch.full((rows, width), 77, dtype=torch.int32, device="cuda")}):
        copies.fill_(-9)
        t, n, r, got, counts = ab.attn_cache_fork(ints(table), ints(lens), ints(refs), page, parents=ints(parents),
                                                  room=ints(room), share=share, copies=copies, **outs)
        with pytest.raises(ab.AttnError, match="no free page"):
            ab.check_device_status()
        ab.check_device_status()
        assert np.array_equal(n.cpu().numpy(), want_n)
        assert np.array_equal(t.cpu().numpy(), want_t)
        assert np.array_equal(r.cpu().numpy(), want_r)
        assert counts.tolist() == [len(made), free]
        assert got[:len(made)].tolist() == [list(map(int, m)) for m in made]
        assert (got[len(made):] == -9).all()
