"""Pieces that go as drafted trees do, at many rows: the sizes are such that they do."""
import pytest
import torch

import _prompt_oracle as po
from _gpu_common import assert_guards, out_buffer
from reference_residual_kv_gb300 import rkv
from test_gpu_prompt import BF16, MARK, cache_with, check_piece, held, i32, near, piece, randn, rows_kv
from test_prompt_ways import tree_bytes

pytestmark = pytest.mark.gpu
CASES = [(8, 2, 128, 33), (8, 2, 128, 64), (7, 1, 64, 40), (7, 1, 64, 64), (8, 1, 256, 5), (8, 1, 256, 8), (3, 3, 256, 60)]


def make(H, N, D, n, lens, bits=4):
    T = 20000
    gen = torch.Generator(device="cuda").manual_seed(n + D)
    c = cache_with(rows_kv(gen, len(lens), max(lens), N, D), lens, T, N, D, bits)
    assert rkv.rkv_chunk_attention_workspace(c.p, H, n) == tree_bytes(c.p, H, n)
    return c, randn(gen, len(lens), n, H, D).to(BF16), rows_kv(gen, len(lens), n, N, D)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("H,N,D,n", CASES)
def test_pieces_as_trees(H, N, D, n, bits):
    lens, new = [0, 31, 777, 2100], [n, n // 2, 0, n - 1]
    c, q, kv = make(H, N, D, n, lens, bits)
    for s in range(4):
        kv[s, new[s]:] = float("nan")                       # rows that are not there
        q[s, new[s]:] = float("nan")
    check_piece(c, H, q, torch.nan_to_num(kv, 0.0), lens, new, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("H,N,D,n", CASES)
def test_wrong_pieces_as_trees(H, N, D, n):
    good = [100, 300, 100, 200]
    c, q, kv = make(H, N, D, n, good)
    lens, new = [-1, 300, c.T - n + 1, 200], [n, n + 1, n, n]
    out = out_buffer(q.shape, BF16)
    out.fill_(MARK)
    c.chunk_attend(H, q, kv, i32(lens), out, n_new=i32(new))
    assert_guards(c)
    assert c.device_status() == rkv.RKV_ERR_INDEX
    assert bool((out[:3] == MARK).all())
    k0, v0 = held(c, good)
    x = kv[3].double().view(n, 2, N, D)
    near(out[3], *po.causal(q[3].double(), torch.cat([k0[3, :200], x[:, 0]]), torch.cat([v0[3, :200], x[:, 1]]), 200))
