"""Pieces of 64 to 257 sequences: up to 256 of them the first CTA of the cache's way to bf16 works the items
out, 64 lengths at a time, beyond that a kernel of its own.  n > 64, so that none goes as a drafted tree."""
import pytest
import torch

from _gpu_common import assert_guards, out_buffer
from reference_residual_kv_gb300 import rkv
from test_gpu_prompt import MARK, cache_with, check_piece, held, i32, near, piece, randn, rows_kv
import _prompt_oracle as po

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
GROUPS = [64, 65, 130, 256, 257]


def make(S, n, T, H, N, D, lens, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = cache_with(rows_kv(gen, S, max(lens), N, D), lens, T, N, D, 4)
    return c, randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)


@pytest.mark.parametrize("S", GROUPS)
def test_empty_ones_among_them(S):
    n, T, H, N, D = 70, 200, 4, 1, 64
    lens, new = [(29 * s) % 131 for s in range(S)], [0 if s % 5 == 2 else (31 * s) % 71 for s in range(S)]
    c, q, kv = make(S, n, T, H, N, D, lens, S)
    check_piece(c, H, q, kv, lens, new, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("S", GROUPS)
def test_few_long_ones_are_split(S):
    # a few sequences of long text, the first and the last of a group of 64 among them: their items are split over the keys
    n, T, H, N, D = 70, 4000, 4, 1, 128
    live = sorted({x for x in (0, 5, 63, 64, 100, 127, 128, 191, 192, 255, S - 1) if x < S})[-7:]
    lens, new = [0] * S, [0] * S
    for i, s in enumerate(live):
        lens[s], new[s] = 3900 - 333 * i, n - i
    c, q, kv = make(S, n, T, H, N, D, lens, S + 1)
    out = piece(c, H, q, kv, lens, new)
    check_piece(c, H, q, kv, lens, new, out)
    assert torch.equal(out, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("S,n,T,H,past", [(65, 300, 500, 8, 130), (130, 200, 1700, 8, 1500), (256, 100, 300, 8, 100), (257, 100, 300, 8, 100)])
def test_more_than_512_tiles(S, n, T, H, past):
    # tiles of 32 tokens; the second set has more keys than stay in L2: its items go by sequence
    N, D = 1, 128
    lens, new = [past - s % 40 for s in range(S)], [n - (7 * s) % 50 for s in range(S)]
    assert sum((x + 31) // 32 for x in new) > 512
    c, q, kv = make(S, n, T, H, N, D, lens, S + 2)
    check_piece(c, H, q, kv, lens, new, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("S,wrong", [(64, 63), (65, 64), (130, 100), (130, 129), (256, 200), (257, 256)])
def test_a_wrong_one_in_a_later_group(S, wrong):
    n, T, H, N, D = 70, 200, 4, 1, 64
    good, new = [(29 * s) % 131 for s in range(S)], [(31 * s) % 71 for s in range(S)]
    c, q, kv = make(S, n, T, H, N, D, good, S + 3)
    lens = list(good)
    lens[wrong], new[wrong] = T - 9, 10
    out = out_buffer(q.shape, BF16)
    out.fill_(MARK)
    c.chunk_attend(H, q, kv, i32(lens), out, n_new=i32(new))
    assert_guards(c)
    assert c.device_status() == rkv.RKV_ERR_INDEX
    k0, v0 = held(c, good)
    x = kv.double().view(S, n, 2, N, D)
    for s in range(S):
        m, a = good[s], 0 if s == wrong else new[s]
        if a:
            near(out[s, :a], *po.causal(q[s, :a].double(), torch.cat([k0[s, :m], x[s, :a, 0]]), torch.cat([v0[s, :m], x[s, :a, 1]]), m))
        assert bool((out[s, a:] == MARK).all()), s


# rows that the capacity has room for, though not for as many as the call allows
@pytest.mark.parametrize("n", [40, 64, 65, 200])
def test_the_last_rows_of_the_capacity(n):
    S, T, H, N, D = 3, 500, 8, 2, 128
    lens, new = [T - 3, T - n + 1, T], [3, n - 1, 0]
    c, q, kv = make(S, n, T, H, N, D, lens, n)
    check_piece(c, H, q, kv, lens, new, piece(c, H, q, kv, lens, new))
