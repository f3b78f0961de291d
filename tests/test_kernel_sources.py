"""Rules of the kernels that no run shows as long as all goes well, checked in their source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "reference_residual_kv_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block_at(src, at):
    """The text between the braces that open behind `at`."""
    i = src.index("{", at)
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        if depth == 0:
            return src[i + 1: j]
        j += 1


# a warp whose wait for a copy ran out waits once more before it leaves: its shared memory may be
# another CTA's when the copy lands
@pytest.mark.parametrize("name", ["rkv_dense_write.cu", "rkv_dense_attention.cu"])
def test_no_warp_leaves_with_a_copy_in_flight(name):
    src = source(name)
    branches = [block_at(src, m.start()) for m in re.finditer(r"if \(!__all_sync\(", src)]
    given_up = [b for b in branches if "RKV_ERR_DEVICE_TIMEOUT" in b or "ok = false" in b]
    assert given_up
    for b in given_up:
        assert "um::mbar_wait(" in b, b
