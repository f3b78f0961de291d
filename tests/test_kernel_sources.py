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


# a kernel that is launched while the one before it still runs must not take that one's outputs as
# read-only: such loads may be moved before its wait, or come from a cache that does not follow writes
@pytest.mark.parametrize("name,kernel,outputs", [
    ("rkv_dense_attention.cu", "k_dense_finish", ("part", "ml", "place")),
    ("rkv_dense_select.cu", "k_block_pick", ("scores",)),
    ("rkv_attention.cu", "k_attn_combine", ("part",))])
def test_outputs_of_the_kernel_before_are_not_read_only(name, kernel, outputs):
    src = source(name)
    at = src.index(kernel + "(")
    args, body = src[at: src.index("{", at)], block_at(src, at)
    assert "griddepcontrol.wait" in body
    for x in outputs:
        assert re.search(r"const \w+ \*%s\b" % x, args), x
        assert not re.search(r"__ldg\([^,;]*\b%s\b" % x, body), x


def test_every_kernel_that_waits_for_the_one_before_is_listed():
    waiting = [f for f in os.listdir(CSRC) if f.endswith(".cu") for _ in re.findall(r"griddepcontrol\.wait", source(f))]
    assert sorted(waiting) == ["rkv_attention.cu", "rkv_dense_attention.cu", "rkv_dense_select.cu"]
