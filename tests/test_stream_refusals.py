"""Calls on an explicit stream refuse bad tensors as the others do, before anything is allocated for them (no
GPU needed)."""
import pytest
import torch

import attention_backward_bwd_gb300 as ab

Q, KC, T, N, S = torch.zeros(2, 2, 64).half(), torch.zeros(4, 8, 2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.int32), \
    torch.zeros(2, dtype=torch.int32), torch.ones(4, 1, 2)


def decode(stream, q=Q, kc=KC, table=T, n=N):
    return ab.attn_decode8(q, kc, KC, S, S, table, n, stream=stream)


def append(stream, k=Q, q=Q, table=T):
    return ab.attn_cache_append8(k, Q, KC, KC, S, S, table, N, q=q, positions=N, inv_freq=S, stream=stream)


def load(stream, kc=KC, tokens=4):
    return ab.attn_cache_load8(kc, KC, S, S, T, N, N, tokens, stream=stream)


def fork(stream, table=T, refs=N):
    return ab.attn_cache_fork(table, N, refs, 8, stream=stream)


def copy(stream, kc=KC):
    return ab.attn_cache_copy(kc, KC, T, k_scale=S, v_scale=S, stream=stream)


CASES = [(decode, dict(q=N)), (decode, dict(q=None)), (decode, dict(kc=T)), (decode, dict(kc=None)), (decode, dict(table=N)),
         (decode, dict(table=None)), (append, dict(k=None)), (append, dict(q=3.0)), (load, dict(kc=N)), (load, dict(kc=None)),
         (fork, dict(table=N)), (fork, dict(table=None)), (fork, dict(refs=None)), (fork, dict(refs=T[0, 0])),
         (copy, dict(kc=None))]


@pytest.mark.parametrize("f,kw", CASES, ids=[f"{f.__name__}-{next(iter(kw))}-{i}" for i, (f, kw) in enumerate(CASES)])
@pytest.mark.parametrize("stream", [None, 0])
def test_bad_tensors_are_refused_alike(f, kw, stream):
    import __graft_entry__ as g
    g.build()
    with pytest.raises(ab.AttnError):
        f(stream, **kw)
