"""How far the attention of prompts and of pieces is from its definition in 64 bits as a whole
(relative norms over the outputs).  The bounds of tests/test_gpu_prompt.py hold for the worst case of
every value and are too wide to tell how many parts the probabilities are held in; these are not.

The distance of a number y from the bf16 numbers, dist(y), moves by no more than y does, so an output
computed as x + d and rounded lies within dist(x + d) + |d| <= dist(x) + 2 |d| of x, and dist(x) is known
exactly (its norm is 1.5-1.7e-3 of the outputs').  |d|: below 2^-16 for probabilities in two parts (half a step
of the second one, which is below 2^-7), 2^-17 for scores and exponentials in fp32; and the accumulators cut each
product of 16 keys that they add, by less than a step of 2^-23, two parts of n keys: n / 8 such cuts.  Together
2 (2^-16 + 2^-17) + n / 4 x 2^-23.  Probabilities in one part have |d| = 0.9e-3 and more, which adds 0.25e-3 at
least; the bound adds 0.12e-3 for 2500 keys."""

import pytest
import torch

import _prompt_oracle as po
from test_gpu_prompt import attend, cache_with, held, packed, piece, randn, rows_kv

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def as_far_off_as_rounding(got, want, keys):
    norm = want.norm()
    off, rounding = float((got.double() - want).norm() / norm), float((want.to(BF16).double() - want).norm() / norm)
    most = rounding + 6 * 2.0 ** -17 + keys / 4 * 2.0 ** -23
    assert off <= most, "%.4e off, its rounding alone %.4e, at most %.4e" % (off, rounding, most)


# whole items of one sequence and of many, items split over the keys, items of the plan
@pytest.mark.parametrize("lens,H,N,D", [([1500], 8, 2, 128), ([1200, 0, 700, 1], 7, 1, 128), ([1100], 8, 2, 64), ([130] * 8, 28, 4, 64),
                                        ([900], 4, 1, 256), ([300] * 40, 4, 2, 128), ([2500], 1, 1, 64), ([2500], 2, 1, 128),
                                        ([2000], 1, 1, 256)])
def test_prompts_are_as_far_off_as_their_own_rounding(lens, H, N, D):
    gen = torch.Generator(device="cuda").manual_seed(31 + H + D)
    q, k, v, start = packed(gen, lens, H, N, D)
    out = attend(q, k, v, start)
    want = torch.cat([po.causal(q[a:b].double(), k[a:b].double(), v[a:b].double())[0] for a, b in zip(start[:-1], start[1:])])
    as_far_off_as_rounding(out, want, max(lens))


# as drafted trees, and from bf16 rows
@pytest.mark.parametrize("n", [3, 33, 64, 65, 300])
@pytest.mark.parametrize("H,N,D,bits", [(8, 2, 128, 4), (7, 1, 64, 2), (4, 1, 256, 4)])
def test_pieces_are_as_far_off_as_their_own_rounding(n, H, N, D, bits):
    gen = torch.Generator(device="cuda").manual_seed(n + D)
    lens, T = [1500, 33, 1131], 2000
    c = cache_with(rows_kv(gen, 3, 1500, N, D), lens, T, N, D, bits)
    q, kv = randn(gen, 3, n, H, D).to(BF16), rows_kv(gen, 3, n, N, D)
    out = piece(c, H, q, kv, lens, None)
    k0, v0 = held(c, lens)
    x = kv.double().view(3, n, 2, N, D)
    want = torch.stack([po.causal(q[s].double(), torch.cat([k0[s, :m], x[s, :, 0]]), torch.cat([v0[s, :m], x[s, :, 1]]), m)[0]
                        for s, m in enumerate(lens)])
    as_far_off_as_rounding(out, want, max(lens) + n)

