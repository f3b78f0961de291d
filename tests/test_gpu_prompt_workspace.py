"""Pieces of more sequences than lie in the scratch as bf16 rows at a time: groups one after another."""
import pytest
import torch

import _prompt_oracle as po
from _gpu_common import assert_guards, out_buffer
from reference_residual_kv_gb300 import rkv
from test_gpu_prompt import BF16, MARK, cache_with, held, i32, near, randn, rows_kv

pytestmark = pytest.mark.gpu


# 11 x 512 MiB: six sequences and five; 5 x 1 GiB: three and two, the last without new rows
@pytest.mark.parametrize("S,T,N,H,D,bits", [(11, 131072, 8, 32, 128, 4), (5, 262144, 4, 4, 256, 2)])
def test_groups_of_sequences(S, T, N, H, D, bits):
    gen = torch.Generator(device="cuda").manual_seed(S)
    n = 150
    good = [(977 * s + 13) % 2500 for s in range(S)]
    new = [n - 20 * (s % 3) for s in range(S)]
    new[S - 1] = 0
    c = cache_with(rows_kv(gen, S, max(good), N, D), good, T, N, D, bits)
    assert rkv.rkv_chunk_attention_workspace(c.p, H, n) < 4.2 * 2 ** 30 < 4 * S * T * N * D
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    k0, v0 = held(c, good)
    x = kv.double().view(S, n, 2, N, D)
    for wrong in (None, S - 2):                              # a wrong length in the second group
        lens = list(good)
        if wrong is not None:
            lens[wrong] = T
        out = out_buffer(q.shape, BF16)
        out.fill_(MARK)
        c.chunk_attend(H, q, kv, i32(lens), out, n_new=i32(new))
        assert_guards(c)
        assert c.device_status() == (0 if wrong is None else rkv.RKV_ERR_INDEX)
        for s in range(S):
            m, a, g = good[s], 0 if s == wrong else new[s], H // N
            assert bool((out[s, a:] == MARK).all()), s
            for h in {0, (5 * s) % H, H - 1} if a else ():
                want = po.causal(q[s, :a, h: h + 1].double(), torch.cat([k0[s, :m], x[s, :a, 0]])[:, h // g: h // g + 1],
                                 torch.cat([v0[s, :m], x[s, :a, 1]])[:, h // g: h // g + 1], m)
                near(out[s, :a, h: h + 1], *want)
    # the first group's bits do not depend on the second one's lengths
    c.status.zero_()
    again = torch.full_like(q, MARK)
    c.chunk_attend(H, q, kv, i32(good), again, n_new=i32(new))
    assert c.device_status() == 0 and torch.equal(again[: (S + 1) // 2], out[: (S + 1) // 2])
