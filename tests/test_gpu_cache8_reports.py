"""What check_device_status says of bad offsets of the 8-bit cache's calls, and which rows they leave."""
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from tests.cache8_helpers import make_cache8

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [2, 3, 4, 5], [-1, 2, 4, 5]])
def test_a_read_back_names_its_offsets(cu):
    kc, vc, ks, vs, table = make_cache8(8, 3, 2, 64, 8, 8, "int8", 61)
    k, v = (torch.full((6, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    ab.attn_cache_load8(kc, vc, ks, vs, table, ints([0, 0, 0]), ints(cu), 6, dtype=torch.float16, out_k=k, out_v=v)
    with pytest.raises(ab.AttnError, match="read-back"):
        ab.check_device_status()
    ab.check_device_status()
    for x in (k, v):
        assert (x[5] == 7.0).all()     # behind the last sequence
        if cu[0] > 0:
            assert (x[:cu[0]] == 7.0).all()
        assert (x[4] != 7.0).any()     # the last sequence's
