"""Sizes next to 2^31 of the 8-bit cache and of shared pages (no GPU needed): the kernels step past the
last token, page or entry in 32 bits, so that the calls refuse what leaves no room for a step.

The C calls get made-up pointers, which only calls that are refused before any launch may get.
"""
import pytest

from tests.test_cache8_checks import P, SHAPE, append, fork, lib, load, paged8  # noqa: F401
from tests.test_cache_checks import T

BIG = 2**31 - 1
CASES = [
    (append, dict(t=BIG, cu=P)), (append, dict(t=BIG - 65534, cu=P)), (load, dict(t=BIG)), (load, dict(t=BIG - 65534)),
    (append, dict(c=paged8(size=1 << 27, block=1 << 27), k=T(), v=T())),
    (load, dict(c=paged8(size=1 << 27, block=1 << 27))),
    (fork, dict(pages=BIG)), (fork, dict(pages=BIG - (1 << 20) + 1)),
    (fork, dict(rows=1, per=BIG, page=1, ts=BIG, ts2=BIG)), (fork, dict(rows=BIG, per=1, page=1, ts=1, ts2=1)),
    (fork, dict(rows=2, per=(BIG - (1 << 20)) // 2 + 1, page=1, ts=1 << 30, ts2=1 << 30)),
]


@pytest.mark.parametrize("f,kw", CASES, ids=[f"{f.__name__}-{i}" for i, (f, _) in enumerate(CASES)])
def test_sizes_without_room_for_a_step_are_refused(lib, f, kw):  # noqa: F811
    if "c" in kw:
        kw = dict(kw, t=0, cu=P)  # nothing could be launched anyway
    assert f(lib, **kw) == SHAPE
    assert lib.attn_last_error()


def test_workspace_sizes_of_such_forks(lib):  # noqa: F811
    most = BIG - (1 << 20)
    assert lib.attn_cache_fork_workspace_size(1, 8, most + 1) == 0
    assert lib.attn_cache_fork_workspace_size(1, most + 1, 8) == 0
    assert lib.attn_cache_fork_workspace_size(1, 8, most) > 0
    assert lib.attn_cache_fork_workspace_size(1, most, 8) > 0
