"""attn_check_device_status with several conditions pending: each is reported, one a call."""
import pytest
import torch

import attention_backward_bwd_gb300 as ab

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bad_offsets():
    q = torch.randn(6, 2, 64, device="cuda").half()
    bad = ints([0, 5])  # does not end at 6
    ab.attn_fwd(q, q, q, cu_seqlens_q=bad, cu_seqlens_k=bad, max_seqlen_q=6, max_seqlen_k=6)


def _wait():
    ab.diag_wait_timeout(20_000_000)


def _decode(lens, table):
    c = torch.zeros(4, 8, 1, 64, device="cuda").half()
    ab.attn_decode(torch.zeros(2, 1, 64, device="cuda").half(), c, c, ints(table), ints(lens), max_seqlen=16)


def _bad_page():
    _decode([16, 3], [[0, 4], [2, 3]])


def _bad_length():
    _decode([16, 17], [[0, 1], [2, 3]])


def _reports(n):
    got = []
    for _ in range(n):
        with pytest.raises(ab.AttnError) as e:
            ab.check_device_status()
        got.append((e.value.code, str(e.value)))
    ab.check_device_status()  # nothing is left
    return got


SAYS = {_bad_offsets: (-9, "cu_seqlens"), _wait: (-8, "wait"), _bad_page: (-9, "page"), _bad_length: (-9, "length")}


@pytest.mark.parametrize("causes", [(_wait, _bad_page), (_bad_offsets, _bad_length), (_wait, _bad_offsets),
                                    (_bad_page, _bad_offsets, _wait)], ids=lambda c: "-".join(f.__name__ for f in c))
def test_every_pending_condition_is_reported(causes):
    ab.check_device_status()
    for cause in causes:
        cause()
    got = _reports(len(causes))
    for cause in causes:
        code, word = SAYS[cause]
        assert any(c == code and word in text for c, text in got), (cause.__name__, got)


@pytest.mark.parametrize("causes", [(_bad_page, _bad_length), (_bad_length, _bad_page)], ids=["page", "length"])
def test_conditions_of_the_serving_calls_share_a_report(causes):
    ab.check_device_status()
    for cause in causes:
        cause()
    (code, text), = _reports(1)
    assert code == -9 and "page" in text and "length" in text
