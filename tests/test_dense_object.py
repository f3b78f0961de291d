"""What DenseCache keeps and refuses: host checks, no GPU."""
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
