"""Scores that overflow to minus infinity: such keys count for nothing, and a row all of whose scores are minus
infinity gives zeros, whichever way its call goes."""
import pytest
import torch

import _prompt_oracle as po
from test_gpu_prompt import BF16, attend, cache_with, held, near, packed, piece, randn, rows_kv

pytestmark = pytest.mark.gpu
BIG = 2.0 ** 100                                             # its square is beyond fp32


def expect(got, q, k, v, before=0):
    want, mag = po.causal(q.double(), k.double(), v.double(), before)
    none = low_rows(q, k, before)
    # the products' fp32 sums overflow where 64-bit ones do not: weights of such keys are 0 there as well
    assert bool((got[none] == 0).all()) and bool(none.any()) and not bool(none.all())
    near(got[~none], want[~none], mag[~none])


def low_rows(q, k, before):
    """Rows [n][H] that see no key whose channel 0 is 0 and have -BIG there."""
    zero_seen = (k[:, :, 0] == 0).long().cumsum(0)[before:] > 0            # [n][N]
    return (q[:, :, 0].double() == -BIG) & ~zero_seen.repeat_interleave(q.shape[1] // k.shape[1], dim=1)


# whole items, items of the plan, items split over the keys
@pytest.mark.parametrize("lens,H,N,D", [([300], 8, 2, 64), ([300, 200], 8, 2, 128), ([300], 4, 1, 256), ([100] * 40, 4, 2, 128),
                                        ([2500], 1, 1, 64), ([3000], 2, 1, 128), ([2500], 1, 1, 256)])
def test_prompts(lens, H, N, D):
    gen = torch.Generator(device="cuda").manual_seed(41 + D)
    q, k, v, start = packed(gen, lens, H, N, D)
    q, k = q.clone(), k.clone()
    q[:, :, 0], k[:, :, 0] = 0.0, 0.0
    q[::3, :, 0] = -BIG
    for a, b in zip(start[:-1], start[1:]):
        k[a: a + (b - a) * 2 // 3, :, 0] = BIG               # the last third of each prompt sees keys that count
    out = attend(q, k, v, start)
    for a, b in zip(start[:-1], start[1:]):
        expect(out[a:b], q[a:b], k[a:b], v[a:b])


# as drafted trees of few rows and of many, and from bf16 rows; behind 300 tokens none of which counts
@pytest.mark.parametrize("n", [4, 40, 64, 100])
@pytest.mark.parametrize("H,N,D", [(8, 2, 64), (8, 2, 128), (4, 1, 256)])
def test_pieces(n, H, N, D):
    gen = torch.Generator(device="cuda").manual_seed(43 + D)
    lens, T = [300, 20], 500
    past, kv = rows_kv(gen, 2, 300, N, D), rows_kv(gen, 2, n, N, D)
    past.view(2, 300, 2, N, D)[:, :, 0, :, 0] = BIG
    x = kv.view(2, n, 2, N, D)
    x[:, :, 0, :, 0] = 0.0
    x[:, : n // 2, 0, :, 0] = BIG
    q = randn(gen, 2, n, H, D).to(BF16)
    q[:, :, :, 0] = 0.0
    q[:, ::3, :, 0] = -BIG
    c = cache_with(past, lens, T, N, D, 4)
    out = piece(c, H, q, kv, lens, None)
    k0, v0 = held(c, lens)
    for s, m in enumerate(lens):
        expect(out[s], q[s], torch.cat([k0[s, :m].to(BF16), x[s, :, 0]]), torch.cat([v0[s, :m].to(BF16), x[s, :, 1]]), m)
