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


def test_the_workspace_of_a_tree_does_not_grow_with_the_capacity():
    # two partials and their {max, sum} for each share (as many as the GPU has CTAs, shared out among
    # the KV heads) and each sequence, whatever the output type and the capacity, and a call asks for
    # no more than that
    L, B = rkv.lib(), ctypes.byref
    for S, T, N, H, D, n in ((32, 131072, 8, 32, 128, 64), (16, 131072, 8, 32, 128, 16), (3, 500, 2, 16, 64, 20)):
        p = rkv.make_dense_params(S, T, N, D)
        need = rkv.rkv_dense_attention_workspace(p, H, n)
        rows = (152 // N + S) * 2 * n * H
        assert need <= 1.1 * (rows * (4 * D + 8) + 4 * (S + 1)) + 1024
        ok = rkv.rkv_dense_cache(16, 16, 16)
        for dt in (rkv.RKV_F32, rkv.RKV_BF16):
            # a pointer that is not aligned is what is left to refuse once the size will do
            for nb, want in ((need, rkv.RKV_ERR_ALIGNMENT), (need - 1, rkv.RKV_ERR_WORKSPACE)):
                assert L.rkv_tree_attention(B(p), H, 16, n, 16, 16, B(ok), 16, 16, dt, 16, nb, 16, None) == want
