"""How far the dense cache's attention is from its definition in 64 bits as a whole (relative
norms over an output tensor).  The bounds of tests/_dense_oracle.py hold for the worst case of
every value and are too wide to tell how many parts the probabilities are held in; these are not.

bf16 outputs: the distance of a number y from the bf16 numbers, dist(y), moves by no more than y
does, so an output computed as x + d and rounded lies within dist(x + d) + |d| <= dist(x) + 2 |d|
of x.  dist(x) is known exactly (its norm is about 1.6e-3 of the outputs'); |d| is at most
2^-17 for the probabilities in two parts, and below 2^-17 for scores and sums in fp32 (5e-6
over the longest runs of blocks): 4 x 2^-17 together.  Probabilities in one part have
|d| = 0.9e-3 and more, which adds 0.2e-3.
"""
import numpy as np
import pytest
import torch

import _dense_oracle as do
from test_gpu_dense import Case, attend_gpu, make_rows, random_tree, tree_gpu

pytestmark = pytest.mark.gpu

BF16_MORE = 4 * 2.0 ** -17


def exact_tree(case, q, parent, draft):
    """[S][n][H][D] in 64 bits."""
    S, n, H, D = q.shape
    G = H // case.N
    out = np.zeros(q.shape)
    for s in range(S):
        K, V, _ = case.held(s)
        sees = np.zeros((n, n), bool)
        for j in range(n):
            line = do.line_of(parent[s], j)
            if line is not None:
                sees[j, line] = True
        for h in range(H):
            k = np.concatenate([K[:, h // G], draft[s, :, 0, h // G]])
            v = np.concatenate([V[:, h // G], draft[s, :, 1, h // G]])
            x = q[s, :, h] @ k.T / np.sqrt(D)
            x[:, len(K):][~sees] = -np.inf
            p = np.exp(x - x.max(axis=1, keepdims=True))
            out[s, :, h] = p / p.sum(axis=1, keepdims=True) @ v
        out[s, parent[s] == -2] = 0.0
    return out


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def tree_case(D, bits, N, G, n, lens):
    rng = np.random.default_rng(D + 10 * bits + n)
    case = Case(make_rows(rng, len(lens), max(lens), N, D), lens, bits)
    q = do.bf16(rng.normal(size=(len(lens), n, N * G, D)) * 1.5)
    draft, parent = make_rows(rng, len(lens), n, N, D), random_tree(rng, len(lens), n)
    return case, q, parent, draft


# up to 32 query rows to a KV head and more, one row tile and two, more than one of 256 rows
@pytest.mark.parametrize("D,bits,G,n", [(64, 4, 4, 8), (64, 2, 4, 9), (128, 4, 4, 8), (128, 4, 7, 24), (128, 2, 4, 64),
                                        (128, 4, 8, 40), (256, 4, 4, 12)])
def test_bf16_outputs_of_trees_are_as_far_off_as_their_own_rounding(D, bits, G, n):
    case, q, parent, draft = tree_case(D, bits, 2, G, n, [1500, 1131])
    want = exact_tree(case, q, parent, draft)
    got = tree_gpu(case, q, parent, draft, torch.bfloat16)
    case.done()
    assert off(got, want) <= off(do.bf16(want), want) + BF16_MORE


@pytest.mark.parametrize("D,bits,G", [(64, 4, 1), (128, 2, 4), (128, 4, 7), (256, 4, 8)])
def test_bf16_outputs_of_single_tokens_are_as_far_off_as_their_own_rounding(D, bits, G):
    rng = np.random.default_rng(D + G)
    lens = [1500, 1131, 2049, 700]
    case = Case(make_rows(rng, 4, 2049, 2, D), lens, bits)
    q = do.bf16(rng.normal(size=(4, 2 * G, D)) * 1.5)
    want = np.zeros(q.shape)
    for s in range(4):
        K, V, _ = case.held(s)
        for h in range(2 * G):
            x = K[:, h // G] @ q[s, h] / np.sqrt(D)
            p = np.exp(x - x.max())
            want[s, h] = p / p.sum() @ V[:, h // G]
    got = attend_gpu(case, q, dtype=torch.bfloat16)
    case.done()
    assert off(got, want) <= off(do.bf16(want), want) + BF16_MORE
