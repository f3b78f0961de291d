"""What DenseCache keeps and refuses: host checks, no GPU."""
import ctypes

import pytest
import torch

from reference_residual_kv_gb300 import build, rkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_a_cache_keeps_its_own_params():
    # one params object, changed between two caches: the first one's sizes stay those of its buffers
    p = rkv.make_dense_params(2, 100, 4, 128)
    c = rkv.DenseCache(p, device="cpu")
    p.T, p.S, p.bits = 4000, 50, 2
    d = rkv.DenseCache(p, device="cpu")
    assert (c.p.S, c.p.T, c.p.N, c.p.D, c.p.bits) == (2, 100, 4, 128, 4)
    assert (d.p.S, d.p.T, d.p.bits) == (50, 4000, 2)
    assert c.codes.numel() == rkv.rkv_dense_sizes(c.p)[0] and d.codes.numel() == rkv.rkv_dense_sizes(d.p)[0]
    assert c._p_ref._obj is c.p


def test_a_stream_of_another_device_is_refused():
    # its launches would take this device's buffers to that one
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 1

    c = rkv.DenseCache(rkv.make_dense_params(2, 100, 4, 128), device="cpu")
    c.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        c._call("rkv_dense_write", Stream(), None)


def test_the_workspace_of_a_tree_is_that_of_its_output_type():
    # fp32 outputs take a partial for every 96 blocks of capacity; bf16 ones for the CTAs of a GPU and
    # the sequences, whatever the capacity, and a call asks for no more than that
    L, B = rkv.lib(), ctypes.byref
    for S, T, N, H, D, n in ((32, 131072, 8, 32, 128, 64), (16, 131072, 8, 32, 128, 16), (3, 500, 2, 16, 64, 20),
                             (4, 9000, 2, 8, 256, 30), (5, 4000, 4, 8, 128, 2)):
        p = rkv.make_dense_params(S, T, N, D)
        need = {dt: rkv.rkv_tree_attention_workspace(p, H, n, dt) for dt in (rkv.RKV_F32, rkv.RKV_BF16)}
        assert rkv.rkv_dense_attention_workspace(p, H, n) == max(need.values()) == need[rkv.RKV_F32]
        if n * H // N > 32 and D <= 128:
            # (what keeps a share's sums, in accumulators that cut, from growing long)
            assert need[rkv.RKV_F32] >= S * (T // 32) / 96 * 2 * n * H * (4 * D + 8)
            # two partials and their {max, sum} for each share of a KV head and each sequence
            rows = (152 // N + S) * 2 * n * H
            assert need[rkv.RKV_BF16] <= 1.1 * (rows * (4 * D + 8) + 4 * (S + 1)) + 1024
        else:
            assert need[rkv.RKV_BF16] == need[rkv.RKV_F32]
        ok = rkv.rkv_dense_cache(16, 16, 16)
        for dt, size in need.items():
            # a pointer that is not aligned is what is left to refuse once the size will do
            for nb, want in ((size, rkv.RKV_ERR_ALIGNMENT), (size - 1, rkv.RKV_ERR_WORKSPACE)):
                assert L.rkv_tree_attention(B(p), H, 16, n, 16, 16, B(ok), 16, 16, dt, 16, nb, 16, None) == want
    c = rkv.DenseCache(rkv.make_dense_params(32, 131072, 8, 64, 2), device="meta")
    sizes = [c._size("tree", 32, 64, dt) for dt in (rkv.RKV_F32, rkv.RKV_BF16)]
    assert sizes == [rkv.rkv_tree_attention_workspace(c.p, 32, 64, dt) for dt in (rkv.RKV_F32, rkv.RKV_BF16)]
    for H, n, dt in ((32, 0, 0), (32, 65, 0), (0, 4, 0), (9, 4, 1), (32, 4, 2)):
        with pytest.raises(rkv.RkvError):
            rkv.rkv_tree_attention_workspace(c.p, H, n, dt)
    assert L.rkv_tree_attention_workspace(B(c.p), 32, 4, 0, None) == rkv.RKV_ERR_INVALID_ARG
