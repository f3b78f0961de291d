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
