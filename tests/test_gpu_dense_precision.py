"""How far the dense cache's attention is from its definition in 64 bits as a whole (relative
norms over an output tensor).  The bounds of tests/_dense_oracle.py hold for the worst case of
every value and are too wide to tell how many parts the probabilities are held in; these are not.

bf16 outputs: the distance of a number y from the bf16 numbers, dist(y), moves by no more than y
does, so an output computed as x + d and rounded lies within dist(x + d) + |d| <= dist(x) + 2 |d|
of x.  dist(x) is known exactly (its norm is about 1.6e-3 of the outputs'); |d| is at most
2^-17 for the probabilities in two parts, and below 2^-17 for scores and sums in fp32 (5e-6
over the longest runs of blocks): 4 x 2^-17 together.  Probabilities in one part have
|d| = 0.9e-3 and more, which adds 0.2e-3.

fp32 outputs: probabilities in two parts alone are 1.7e-6 off and more on this data, those in three
2e-8, and scores summed in fp32 0.2-0.4e-6 (tests/test_dense_precision_limits.py): 1.2e-6 tells two
parts from three, and does not let sums grow long in accumulators that cut what they add.
"""
import numpy as np
import pytest
import torch

import _dense_oracle as do
from reference_residual_kv_gb300 import rkv
from test_gpu_dense import Case, attend_gpu, make_rows, random_tree, tree_gpu

pytestmark = pytest.mark.gpu

BF16_MORE = 4 * 2.0 ** -17
F32_OFF = 1.2e-6
TREES = [(64, 4, 4, 8), (64, 2, 4, 9), (128, 4, 4, 8), (128, 4, 7, 24), (128, 2, 4, 64), (128, 4, 8, 40), (256, 4, 4, 12)]
SINGLE = [(64, 4, 1), (128, 2, 4), (128, 4, 7), (256, 4, 8)]


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
@pytest.mark.parametrize("D,bits,G,n", TREES)
def test_bf16_outputs_of_trees_are_as_far_off_as_their_own_rounding(D, bits, G, n):
    case, q, parent, draft = tree_case(D, bits, 2, G, n, [1500, 1131])
    want = exact_tree(case, q, parent, draft)
    got = tree_gpu(case, q, parent, draft, torch.bfloat16)
    case.done()
    assert off(got, want) <= off(do.bf16(want), want) + BF16_MORE


@pytest.mark.parametrize("D,bits,G,n", TREES)
def test_fp32_outputs_of_trees(D, bits, G, n):
    case, q, parent, draft = tree_case(D, bits, 2, G, n, [1500, 1131])
    want = exact_tree(case, q, parent, draft)
    got = tree_gpu(case, q, parent, draft)
    case.done()
    assert off(got, want) <= F32_OFF


def single_case(D, bits, G):
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
    return case, q, want


@pytest.mark.parametrize("D,bits,G", SINGLE)
def test_bf16_outputs_of_single_tokens_are_as_far_off_as_their_own_rounding(D, bits, G):
    case, q, want = single_case(D, bits, G)
    got = attend_gpu(case, q, dtype=torch.bfloat16)
    case.done()
    assert off(got, want) <= off(do.bf16(want), want) + BF16_MORE


@pytest.mark.parametrize("D,bits,G", SINGLE)
def test_fp32_outputs_of_single_tokens(D, bits, G):
    case, q, want = single_case(D, bits, G)
    got = attend_gpu(case, q)
    case.done()
    assert off(got, want) <= F32_OFF


def test_fp32_outputs_over_131072_tokens():
    # 216 blocks to a CTA for the tree; keys and values in 64 bits are those that the cache reads back
    # (test_gpu_dense.py holds them against the definition)
    T, N, G, D, n = 131072, 8, 4, 128, 9
    H = N * G
    gen = torch.Generator("cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    c = rkv.DenseCache(rkv.make_dense_params(1, T, N, D))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c.write((rand(1, T, 2 * N * D) + rand(1, 1, 2 * N * D) * 0.7).bfloat16(), i32(0))
    k, v = torch.empty(1, T, N * D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, T, N * D, dtype=torch.bfloat16, device="cuda")
    c.read(i32(T), torch.arange(T, dtype=torch.int32, device="cuda")[None], k, v)
    q, draft = (rand(1, n, H, D) * 1.5).bfloat16(), rand(1, n, 2 * N * D).bfloat16()
    parent = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    out, one = torch.empty(1, n, H, D, device="cuda"), torch.empty(1, H, D, device="cuda")
    c.tree_attend(H, q, parent, draft, i32(T), out)
    c.attend(H, q[:, 0].contiguous(), i32(T), one)
    d = draft.double().view(n, 2, N, D)
    num, den = {"tree": 0.0, "one": 0.0}, {"tree": 0.0, "one": 0.0}
    for h in range(H):
        K, V = k.view(T, N, D)[:, h // G].double(), v.view(T, N, D)[:, h // G].double()
        x = torch.cat([q[0, :, h].double() @ K.T, (q[0, :, h].double() * d[:, 0, h // G]).sum(1, keepdim=True)], 1) / D ** 0.5
        p = torch.softmax(x, 1)
        want = p[:, :T] @ V + p[:, T:] * d[:, 1, h // G]
        alone = torch.softmax(x[:1, :T], 1) @ V
        for name, a, b in (("tree", out[0, :, h], want), ("one", one[0, h], alone[0])):
            num[name] += float((a.double() - b).square().sum())
            den[name] += float(b.square().sum())
    assert c.device_status() == 0
    assert (num["one"] / den["one"]) ** 0.5 <= F32_OFF
    assert (num["tree"] / den["tree"]) ** 0.5 <= F32_OFF


# the most rows that a call takes, as two tiles of 256, and two rows to a warp of the last pass at
# D = 256 (more CTAs than the GPU holds at a time)
@pytest.mark.parametrize("D,bits,S,G,n", [(128, 4, 3, 8, 64), (64, 2, 3, 8, 64), (256, 4, 40, 4, 32), (256, 2, 42, 2, 61)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_trees(D, bits, S, G, n, dtype):
    lens = [800, 32 * 17, 63] if S == 3 else [int(x) for x in np.random.default_rng(S).integers(0, 200, S)]
    case, q, parent, draft = tree_case(D, bits, 1, G, n, lens)
    want = exact_tree(case, q, parent, draft)
    got = tree_gpu(case, q, parent, draft, dtype)
    case.done()
    assert not got[parent == -2].any()
    limit = F32_OFF if dtype == torch.float32 else off(do.bf16(want), want) + BF16_MORE
    assert off(got, want) <= limit
    for s in range(S):                             # no row hides behind the others' norm
        for j in np.nonzero(parent[s] > -2)[0]:
            assert off(got[s, j], want[s, j]) <= 4 * limit, (s, j)


# sums that leave the accumulators several times in a share while the running maximum grows (one row
# tile whose last warp has four rows, two tiles, the second one of four rows and of 32, and 64 rows
# beyond 256)
@pytest.mark.parametrize("D,bits,G,n", [(128, 4, 4, 9), (64, 2, 4, 33), (128, 2, 8, 20), (128, 4, 8, 40)])
def test_joined_sums_follow_a_growing_maximum(D, bits, G, n):
    T, N = 20005, 8
    H = N * G
    gen = torch.Generator("cuda").manual_seed(n)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = rand(1, T, 2 * N * D)
    kv[:, :, : N * D] *= 0.2 + 4.0 * torch.arange(T, device="cuda")[:, None] / T
    c = rkv.DenseCache(rkv.make_dense_params(1, T, N, D, bits), guard=4096)
    c.write(kv.bfloat16(), i32(0))
    k, v = torch.empty(1, T, N * D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, T, N * D, dtype=torch.bfloat16, device="cuda")
    c.read(i32(T), torch.arange(T, dtype=torch.int32, device="cuda")[None], k, v)
    q, draft = (rand(1, n, H, D) * 1.5).bfloat16(), rand(1, n, 2 * N * D).bfloat16()
    parent = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    out = torch.full((1, n, H, D), float("nan"), device="cuda")
    c.tree_attend(H, q, parent, draft, i32(T), out)
    d = draft.double().view(n, 2, N, D)
    for h in range(H):
        own_k, own_v = d[:, 0, h // G], d[:, 1, h // G]
        K, V = k.view(T, N, D)[:, h // G].double(), v.view(T, N, D)[:, h // G].double()
        Q = q[0, :, h].double()
        x = torch.cat([Q @ K.T, (Q * own_k).sum(1, keepdim=True)], 1) / D ** 0.5
        p = torch.softmax(x, 1)
        want = p[:, :T] @ V + p[:, T:] * own_v
        # the bound of _dense_oracle.attend
        A = torch.maximum((Q.abs() @ K.abs().T).amax(1), (Q.abs() * own_k.abs()).sum(1)) / D ** 0.5
        r = D * 2.0 ** -22 * A + 2.0 ** -23 * x.abs().amax(1) + 2.0 ** -20
        tol = (2 * r + 2.0 ** -16)[:, None] * (p[:, :T] @ V.abs() + p[:, T:] * own_v.abs())
        assert bool(((out[0, :, h].double() - want).abs() <= tol).all()), h
    torch.cuda.synchronize()
    assert c.device_status() == 0 and not c.guard_violations()
