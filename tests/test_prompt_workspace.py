"""The scratch of pieces behind their cached text: host arithmetic, no GPU."""
import pytest

from reference_residual_kv_gb300 import build, rkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("n", [65, 512, 4096])
def test_the_scratch_of_pieces_is_bounded(n):
    # bf16 rows of 4 GiB or of one sequence, whichever is more; 608 partials of 256 rows (128 of D = 256); items of
    # 32 bytes, 16 tokens at least to each, with their joins of 16 bytes
    for S, T, N, H, D in ((1, 131072, 8, 32, 128), (16, 131072, 8, 32, 128), (64, 131072, 8, 32, 128), (300, 32768, 4, 28, 128),
                          (2, 1 << 21, 8, 32, 128), (5, 1 << 20, 2, 2, 256), (1000, 4096, 8, 64, 64)):
        p = rkv.make_dense_params(S, T, N, D)
        one = 4 * T * N * D
        rows = min(S * one, max(one, 4 << 30))
        tiles = S * (n // 16 + 1)
        assert rkv.rkv_chunk_attention_workspace(p, H, n) <= rows + 608 * 256 * (4 * D + 8) + 48 * (tiles + 608) + 4096


def test_all_at_a_time_where_they_fit():
    p = rkv.make_dense_params(8, 16384, 4, 128)
    assert rkv.rkv_chunk_attention_workspace(p, 28, 512) >= 8 * 16384 * 4 * 4 * 128
