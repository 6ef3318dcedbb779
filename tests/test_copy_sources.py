"""What the kernels' sources do not use (no GPU needed)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_backward_bwd_gb300", "csrc")


def test_asynchronous_copies_by_threads_have_no_cache_policy():
    # (cp.async of 4 to 16 bytes; bulk copies are another instruction) kernels that had one ended with an
    # illegal instruction, and it was not found why others did not
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            found = re.findall(r"cp\.async\.c[ag]\.shared\.global\S*cache_hint", f.read())
        assert not found, name
