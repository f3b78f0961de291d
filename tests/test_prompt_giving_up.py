"""The prompt attention kernel (csrc/rkv_prompt_attention.cu) where a wait runs out, on the CPU."""
import pytest

from test_kernel_sources import block_at, source


@pytest.fixture(scope="module")
def kernel():
    src = source("rkv_prompt_attention.cu")
    return block_at(src, src.index("k_prompt_attention(const __grid_constant__"))


def test_no_store_to_tensor_memory_is_under_way_when_it_is_freed(kernel):
    # a wait for the products so far comes between a tile's first exponentials, which are stored, and
    # the wait for stores behind the second ones
    rows = block_at(kernel, kernel.index("else if (warp >= 4)"))
    loop_at = rows.index("take(i, w)")
    loop = block_at(rows, loop_at)
    behind = rows[rows.index(loop, loop_at) + len(loop):]
    assert "tmem_st16(" in loop and "break;" in loop
    assert "tmem_wait_st();" in behind
    assert kernel.index(behind) < kernel.index("um::tmem_dealloc(")
