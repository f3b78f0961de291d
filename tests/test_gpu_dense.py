"""The dense cache on the GPU against its fp64 restatement: what is written reads back as
defined, bit for bit; block lists are equal; attention stays within a bound that is worked
out from the data (tests/_dense_oracle.py: attend)."""
import math

import numpy as np
import pytest
import torch

import _dense_oracle as do
from _gpu_common import GUARD, assert_guards, ensure_lib, out_buffer
from reference_residual_kv_gb300 import rkv

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8          # torch.finfo(torch.bfloat16).eps / 2


def make_rows(rng, S, T, N, D, kind="normal"):
    """float64 [S][T][2][N][D] of bf16 values."""
    x = rng.normal(size=(S, T, 2, N, D))
    if kind == "normal":
        x[:, :, 0] += rng.normal(size=(1, 1, N, D)) * np.where(rng.random((1, 1, N, D)) < 0.05, 6.0, 0.7)
    elif kind == "ties":            # small whole numbers: many exact half steps
        x = rng.integers(-15, 16, size=x.shape).astype(np.float64)
    elif kind == "grid":            # offsets, tiny values among large ones, zeros, coarse grids
        x = np.choose(rng.integers(0, 4, size=x.shape), [rng.integers(-200, 200, size=x.shape) / 8.0, x, x * 2.0 ** -10, 0.0])
        x = x + np.where(rng.random((S, 1, 2, N, D)) < 0.3, 100.0, 0.0)
    elif kind == "wide":            # exponents far apart: differences that fp32 rounds
        x = x * 2.0 ** rng.integers(-40, 41, size=x.shape)
    return do.bf16(x)


def to_bf16(x):
    return torch.from_numpy(do.bf16_bits(x).view(np.int16).copy()).view(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Case:
    """A cache on the GPU that holds rows[s][:lens[s]], written in one call."""

    def __init__(self, rows, lens, bits, T=None, write=True):
        ensure_lib()
        S, t, _, N, D = rows.shape
        self.rows, self.lens, self.bits = rows, list(lens), bits
        self.S, self.N, self.D, self.T = S, N, D, T or t
        self.c = rkv.DenseCache(rkv.make_dense_params(S, self.T, N, D, bits), guard=GUARD)
        for t_ in (self.c.codes, self.c.khdr, self.c.tail):
            t_.fill_(0xFF)                          # NaN everywhere that is not written
        self.len = i32(self.lens)
        if write and max(self.lens) > 0:
            m = max(self.lens)
            self.c.write(to_bf16(rows[:, :m].reshape(S, m, 2 * N * D)), i32([0] * S), self.len)

    def held(self, s):
        return do.held(self.rows[s], self.lens[s], self.bits)

    def read(self, sel):
        k = out_buffer((self.S, sel.shape[1], self.N * self.D), torch.bfloat16)
        v = out_buffer(k.shape, k.dtype)
        self.c.read(self.len, i32(sel), k, v)
        return [x.float().cpu().numpy().astype(np.float64).reshape(self.S, -1, self.N, self.D) for x in (k, v)]

    def check_all(self):
        """Every token, in a shuffled order with padding and repeats."""
        n = max(self.lens) + 5
        rng = np.random.default_rng(n)
        sel = np.full((self.S, n), -1, np.int32)
        for s in range(self.S):
            sel[s, : self.lens[s]] = rng.permutation(self.lens[s])
            if self.lens[s]:
                sel[s, -1] = sel[s, 0]
        k, v = self.read(sel)
        for s in range(self.S):
            K, V, _ = self.held(s)
            live = sel[s] >= 0
            assert np.array_equal(k[s][live], K[sel[s][live]], equal_nan=True), "keys of sequence %d" % s
            assert np.array_equal(v[s][live], V[sel[s][live]], equal_nan=True), "values of sequence %d" % s
            assert not k[s][~live].any() and not v[s][~live].any()
        self.done()

    def done(self, status=0):
        torch.cuda.synchronize()
        assert self.c.device_status() == status
        assert not self.c.guard_violations()
        assert_guards()


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("kind", ["normal", "ties", "wide", "grid"])
@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("N,D", [(1, 64), (3, 128), (2, 256)])
def test_written_rows_read_back_as_defined(N, D, bits, kind):
    rng = np.random.default_rng(D + bits)
    Case(make_rows(rng, 3, 101, N, D, kind), [101, 64, 7], bits).check_all()


def test_groups_at_the_ends_of_the_range():
    # constant groups, both zeros, the smallest and the largest numbers, a step that rounds to
    # zero, NaN, infinities and 2^126, each in a block of its own, in keys and in values
    rng = np.random.default_rng(1)
    rows = make_rows(rng, 1, 12 * 32 + 3, 1, 64)
    b = rows[0, :384].reshape(12, 32, 2, 1, 64)
    b[0] = 1.7109375
    b[1] = np.where(rng.random(b[1].shape) < 0.5, 0.0, -0.0)
    b[2] = do.bf16(rng.integers(-9, 10, b[2].shape) * 2.0 ** -133)       # subnormals
    b[3] = do.bf16(rng.normal(size=b[3].shape) * 2.0 ** -124)
    b[4] = do.bf16(rng.uniform(-1, 1, b[4].shape) * 2.0 ** 125.9)
    b[5, 3, :, :, 5] = np.nan
    b[6, 9, :, :, 9] = np.inf
    b[7, 11, :, :, 40] = -np.inf
    b[8, 30, :, :, 1] = 2.0 ** 126
    b[9, 30, :, :, 1] = -(2.0 ** 126)
    b[10] = do.bf16(rng.normal(size=b[10].shape) * 2.0 ** -110)          # no finite reciprocal of the step
    b[11] = np.where(rng.random(b[11].shape) < 0.5, 1.0, do.bf16(1.0 + 2.0 ** -7))
    rows[0, 384:] = np.nan                                               # the tail holds rows as they are
    for bits in (2, 4):
        Case(rows, [387], bits).check_all()


@pytest.mark.parametrize("f32", [False, True])
def test_a_prompt_then_pieces_then_single_tokens(f32):
    # the same cache as one write makes, whatever the pieces: a prompt, pieces that start and
    # end inside blocks, then one token at a time across block ends; uneven sequences
    rng = np.random.default_rng(3)
    S, N, D, T = 3, 2, 128, 260
    rows = make_rows(rng, S, T, N, D)
    raw = rows + (rng.normal(size=rows.shape) * 2.0 ** -12 * np.abs(rows) if f32 else 0.0)
    raw = raw.astype(np.float32)
    rows = do.bf16(raw.astype(np.float64)) if f32 else rows
    case = Case(rows, [0] * S, 4, write=False)
    have = [0] * S
    for piece in ([70, 33, 0], [1, 64, 5], [31, 3, 27], [0, 1, 90]) + tuple([1, 1, 1] for _ in range(70)):
        n = max(piece)
        kv = np.zeros((S, n, 2, N, D), np.float32)
        for s, m in enumerate(piece):
            kv[s, :m] = raw[s, have[s]: have[s] + m]
            kv[s, m:] = np.nan                      # rows behind n_new are not read
        kv = kv.reshape(S, n, -1)
        kv = torch.from_numpy(kv).cuda() if f32 else torch.from_numpy(kv).cuda().bfloat16()
        case.c.write(kv, i32(have), None if n == 1 else i32(piece))
        have = [h + m for h, m in zip(have, piece)]
    case.lens, case.len = have, i32(have)
    case.check_all()


def test_wrong_positions_and_counts_write_nothing():
    rng = np.random.default_rng(4)
    rows = make_rows(rng, 5, 96, 1, 64)
    case = Case(rows, [40] * 5, 4)
    torch.cuda.synchronize()
    before = [t.clone() for t in (case.c.codes, case.c.khdr, case.c.tail)]
    kv = to_bf16(make_rows(rng, 5, 40, 1, 64).reshape(5, 40, -1))
    case.c.write(kv, i32([-1, 90, 40, 40, 57]), i32([5, 7, 41, -1, 40]))
    case.done(rkv.RKV_ERR_INDEX)
    for a, b in zip(before, (case.c.codes, case.c.khdr, case.c.tail)):
        assert torch.equal(a, b)


def test_wrong_entries_and_lengths_read_zeros():
    rng = np.random.default_rng(5)
    case = Case(make_rows(rng, 2, 70, 2, 64), [70, 33], 4)
    k, v = case.read(np.array([[0, 70, -2], [33, 32, 2 ** 31 - 1]]))
    K, V, _ = case.held(0)
    assert np.array_equal(k[0, 0], K[0]) and not k[0, 1:].any() and not v[0, 1:].any()
    assert not k[1, 0].any() and not k[1, 2].any() and np.array_equal(v[1, 1], case.held(1)[1][32])
    case.done(rkv.RKV_ERR_INDEX)
    case.c.status.zero_()
    case.len = i32([71, -1])
    k, v = case.read(np.array([[0, 1], [0, 1]]))
    assert not k.any() and not v.any()
    case.done(rkv.RKV_ERR_INDEX)


# ------------------------------------------------------------------ attention of single tokens
def attend_gpu(case, q, blocks=None, dtype=torch.float32):
    out = out_buffer((case.S, q.shape[1], case.D), dtype)
    out.fill_(float("nan"))
    case.c.attend(q.shape[1], to_bf16(q), case.len, out, blocks=None if blocks is None else i32(blocks))
    return out.double().cpu().numpy()


def check_attend(case, q, got, blocks=None, bf16=False):
    H, G = q.shape[1], q.shape[1] // case.N
    for s in range(case.S):
        K, V, _ = case.held(s)
        full = case.lens[s] // 32
        for h in range(H):
            n = h // G
            at = np.arange(case.lens[s])
            if blocks is not None:
                pick = [b for b in blocks[s, n if blocks.shape[1] > 1 else 0] if 0 <= b < full]
                at = np.concatenate([np.arange(32 * b, 32 * b + 32) for b in pick] + [np.arange(32 * full, case.lens[s])]).astype(int)
            want, tol = do.attend(q[s, h], K[at, n], V[at, n])
            if bf16:
                tol = tol + HALF_BF16 * np.abs(want)
            assert np.all(np.abs(got[s, h] - want) <= tol), (s, h, np.abs(got[s, h] - want).max(), tol.min())


@pytest.mark.parametrize("D,bits,N,G", [
    (64, 4, 2, 1), (64, 2, 1, 8), (128, 4, 2, 4), (128, 2, 3, 3), (128, 4, 1, 7), (128, 4, 1, 8),
    (256, 4, 1, 2), (256, 2, 2, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_over_whole_caches(D, bits, N, G, dtype):
    # lengths: nothing, one token, one short of a block, a block, one more, ragged, many blocks
    rng = np.random.default_rng(D + G)
    lens = [0, 1, 31, 32, 33, 64, 257, 1000]
    case = Case(make_rows(rng, len(lens), 1003, N, D), lens, bits)
    q = do.bf16(rng.normal(size=(len(lens), N * G, D)) * 1.5)
    got = attend_gpu(case, q, dtype=dtype)
    check_attend(case, q, got, bf16=dtype == torch.bfloat16)
    assert not got[0].any()
    case.done()


def test_attention_over_listed_blocks():
    rng = np.random.default_rng(11)
    lens = [20, 32, 331, 640]
    case = Case(make_rows(rng, 4, 640, 2, 128), lens, 4)
    q = do.bf16(rng.normal(size=(4, 6, 128)) * 1.5)
    for lists in (1, 2):
        blocks = np.full((4, lists, 19), -1, np.int32)
        for s in range(4):
            for l in range(lists):
                n = lens[s] // 32
                m = int(rng.integers(0, n + 1))
                blocks[s, l, rng.permutation(19)[:m]] = rng.permutation(n)[:m]      # any order, -1 between
        blocks[3, 0, :4] = 7                                                         # a block several times
        got = attend_gpu(case, q, blocks)
        check_attend(case, q, got, blocks)
        case.done()
    # entries outside the finished blocks are left out and reported
    blocks = np.array([[[0, -1]], [[1, 0]], [[10, 3]], [[-5, 4]]], np.int32)
    got = attend_gpu(case, q, blocks)
    check_attend(case, q, got, blocks)
    case.done(rkv.RKV_ERR_INDEX)


def test_scores_far_apart_and_infinite_rows():
    # scores in the thousands (one token takes all), and a block whose values are NaN: seen
    # without a list, unseen where the list leaves it out
    rng = np.random.default_rng(12)
    rows = make_rows(rng, 1, 200, 1, 128)
    rows[0, :, 0] *= 64.0
    case = Case(rows, [200], 4)
    q = do.bf16(rng.normal(size=(1, 4, 128)) * 16)
    check_attend(case, q, attend_gpu(case, q))
    rows[0, 70, 1] = np.nan
    rows[0, 130, 0] = np.inf
    case = Case(rows, [200], 4)
    assert np.isnan(attend_gpu(case, q)).all()
    blocks = np.array([[[0, 1, 3, 5]]])
    check_attend(case, q, attend_gpu(case, q, blocks), blocks)
    case.done()


# ------------------------------------------------------------------ selection
def select_gpu(case, q, lists, n, first, last):
    blocks = out_buffer((case.S, lists, n), torch.int32)
    blocks.fill_(-9)
    case.c.select(q.shape[1], to_bf16(q), case.len, blocks, keep_first=first, keep_last=last)
    return blocks.cpu().numpy()


@pytest.mark.parametrize("D,bits,N,G", [(64, 4, 2, 1), (128, 4, 2, 4), (128, 2, 3, 7), (256, 4, 1, 8)])
def test_selected_blocks_are_those_of_the_exact_scores(D, bits, N, G):
    rng = np.random.default_rng(D + N)
    lens = [0, 40, 32 * 21, 32 * 40 + 9, 1311]
    rows = make_rows(rng, 5, 1311, N, D)
    rows[3, 320:640] = rows[3, 640:960]                 # ten blocks twice: equal scores
    case = Case(rows, lens, bits)
    q = do.bf16(rng.normal(size=(5, N * G, D)))
    for lists in {1, N}:
        for n, first, last in ((1, 0, 0), (1, 0, 1), (7, 1, 1), (20, 3, 0), (39, 0, 0), (64, 2, 5)):
            got = select_gpu(case, q, lists, n, first, last)
            for s in range(5):
                want = do.select(q[s], case.held(s)[2], n, first, last, lists == 1 and N > 1)
                assert np.array_equal(got[s], want), (s, lists, n, got[s], want)
    case.done()


def test_selection_among_equal_scores_and_not_numbers():
    # zero queries: every score is equal, the lowest indexes win, with more candidates than
    # one pass ranks (1200 blocks); then a query that sees only the sign bit of two blocks
    rng = np.random.default_rng(21)
    rows = make_rows(rng, 1, 1200 * 32, 1, 64)
    rows[0, 999 * 32 + 4, 0, 0, 3] = np.nan             # ranks above every number
    case = Case(rows, [1200 * 32], 4)
    q = np.zeros((1, 2, 64))
    got = select_gpu(case, q, 1, 50, 2, 3)[0, 0]
    # 0 * NaN is NaN: block 999 first, then the kept ends and the lowest of the others
    assert list(got) == list(range(46)) + [999, 1197, 1198, 1199]
    q[0, 0, 0] = 1.0
    want = do.select(q[0], case.held(0)[2], 300, 0, 0, False)
    assert np.array_equal(select_gpu(case, q, 1, 300, 0, 0)[0], want)
    # near ties: keys whose bounds differ in the last bits of a long sum
    rows = np.repeat(make_rows(rng, 1, 32, 1, 64), 400, axis=1).reshape(1, 12800, 2, 1, 64)
    rows[0, :, 0, 0, 5] = np.repeat(do.bf16(1.0 + rng.integers(0, 40, 400) * 2.0 ** -7), 32)
    case = Case(rows, [12800], 4)
    q = do.bf16(rng.normal(size=(1, 2, 64)) * 100)
    q[0, :, 5] = do.bf16(2.0 ** -9)
    want = do.select(q[0], case.held(0)[2], 111, 0, 0, False)
    assert np.array_equal(select_gpu(case, q, 1, 111, 0, 0)[0], want)
    case.done()


# ------------------------------------------------------------------ trees of drafted tokens
def tree_gpu(case, q, parent, draft, dtype=torch.float32):
    S, n, H, D = q.shape
    out = out_buffer((S, n, H, D), dtype)
    out.fill_(float("nan"))
    case.c.tree_attend(H, to_bf16(q), i32(parent), to_bf16(draft.reshape(S, n, -1)), case.len, out)
    return out.double().cpu().numpy()


def check_tree(case, q, parent, draft, got, bf16=False):
    S, n, H, D = q.shape
    G = H // case.N
    for s in range(S):
        K, V, _ = case.held(s)
        for j in range(n):
            line = do.line_of(parent[s], j)
            if line is None or line == "bad":
                assert not got[s, j].any()
                continue
            line = sorted(line)
            for h in range(H):
                kh = np.concatenate([K[:, h // G], draft[s, line, 0, h // G]])
                vh = np.concatenate([V[:, h // G], draft[s, line, 1, h // G]])
                # many rows with bf16 outputs: probabilities in bf16 (include/rkv.h)
                want, tol = do.attend(q[s, j, h], kh, vh, 2.0 ** -8 if bf16 and n * G > 32 and D <= 128 else 2.0 ** -16)
                if bf16:
                    tol = tol + HALF_BF16 * np.abs(want)
                assert np.all(np.abs(got[s, j, h] - want) <= tol), (s, j, h, np.abs(got[s, j, h] - want).max(), tol.min())


def random_tree(rng, S, n):
    parent = np.full((S, n), -2, np.int32)
    for s in range(S):
        m = n if s == 0 else int(rng.integers(1, n + 1))
        for j in range(m):
            parent[s, j] = -1 if j == 0 or rng.random() < 0.1 else rng.integers(max(0, j - 5), j)
    return parent


@pytest.mark.parametrize("D,bits,N,G,n", [
    (64, 4, 1, 8, 1), (64, 2, 2, 3, 5), (128, 4, 2, 4, 2), (128, 4, 1, 4, 4), (128, 2, 1, 7, 24),
    (128, 4, 2, 1, 64), (128, 4, 1, 8, 33), (256, 4, 1, 2, 9), (256, 2, 1, 4, 32)])
def test_tree_attention(D, bits, N, G, n):
    rng = np.random.default_rng(D + n)
    lens = [500, 0, 1, 32, 95]
    case = Case(make_rows(rng, 5, 515, N, D), lens, bits)
    q = do.bf16(rng.normal(size=(5, n, N * G, D)) * 1.5)
    draft = make_rows(rng, 5, n, N, D)
    parent = random_tree(rng, 5, n)
    for dtype in (torch.float32, torch.bfloat16):
        got = tree_gpu(case, q, parent, draft, dtype)
        check_tree(case, q, parent, draft, got, dtype == torch.bfloat16)
    case.done()


@pytest.mark.parametrize("D,bits,G,n", [(128, 4, 4, 64), (128, 2, 5, 20), (64, 4, 8, 40), (64, 2, 3, 12), (128, 4, 8, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_trees_over_long_caches(D, bits, G, n, dtype):
    # many tiles and several runs of blocks; keys grow along the cache, so that the maximum of
    # a row moves again and again (and by more than any fixed reference allows); the other
    # sequence ends inside a tile
    rng = np.random.default_rng(D * n)
    rows = make_rows(rng, 2, 4500, 1, D)
    rows[:, :, 0] = do.bf16(rows[:, :, 0] * (0.2 + 4.0 * np.arange(4500)[None, :, None, None] / 4500))
    case = Case(rows, [4500, 2085], bits)
    q = do.bf16(rng.normal(size=(2, n, G, D)) * 1.5)
    draft = make_rows(rng, 2, n, 1, D)
    parent = random_tree(rng, 2, n)
    check_tree(case, q, parent, draft, tree_gpu(case, q, parent, draft, dtype), dtype == torch.bfloat16)
    case.done()


def test_chains_roots_and_wrong_parents():
    rng = np.random.default_rng(31)
    n = 40
    case = Case(make_rows(rng, 4, 70, 1, 128), [70, 64, 3, 0], 4)
    q = do.bf16(rng.normal(size=(4, n, 2, 128)))
    draft = make_rows(rng, 4, n, 1, 128)
    parent = np.stack([np.arange(n) - 1, np.full(n, -1), np.full(n, -1), np.arange(n) - 1]).astype(np.int32)
    got = tree_gpu(case, q, parent, draft)
    check_tree(case, q, parent, draft, got)
    case.done()
    parent[0, 5] = 5                                   # itself
    parent[1, 7] = 39                                  # a later one
    parent[2, 3], parent[2, 4] = -2, 3                 # a child of padding
    parent[3, 9] = -3
    got = tree_gpu(case, q, parent, draft)
    check_tree(case, q, parent, draft, got)
    case.done(rkv.RKV_ERR_INDEX)


def test_what_a_drafted_token_does_not_see_does_not_reach_it():
    rng = np.random.default_rng(32)
    case = Case(make_rows(rng, 1, 100, 1, 128), [100], 4)
    q = do.bf16(rng.normal(size=(1, 6, 4, 128)))
    draft = make_rows(rng, 1, 6, 1, 128)
    parent = np.array([[-1, 0, 0, 1, -2, -1]], np.int32)
    draft[0, 2, 0] = np.inf                            # seen by itself alone
    draft[0, 2, 1] = np.nan
    draft[0, 4] = np.nan                               # padding
    got = tree_gpu(case, q, parent, draft)
    assert np.isnan(got[0, 2]).all() and not got[0, 4].any()
    parent[0, 2] = -2
    got[0, 2] = 0.0
    check_tree(case, q, parent, draft, got)
    case.done()


# ------------------------------------------------------------------ together
def test_decode_with_selection_drafts_and_the_sparse_read():
    """A prompt, then steps: the full-attention layer selects blocks, attends them, verifies a
    tree of drafted tokens, writes the accepted line, and its tokens go through the sparse
    layers' attention as rows."""
    rng = np.random.default_rng(41)
    S, N, G, D, T = 2, 2, 4, 128, 420
    H = N * G
    rows = make_rows(rng, S, T, N, D)
    case = Case(rows, [300, 251], 4)
    for step in range(4):
        q = do.bf16(rng.normal(size=(S, H, D)))
        blocks = select_gpu(case, q, 1, 5, 1, 1)
        for s in range(S):
            assert np.array_equal(blocks[s], do.select(q[s], case.held(s)[2], 5, 1, 1, True))
        check_attend(case, q, attend_gpu(case, q, blocks), blocks)
        n = 12
        parent = random_tree(rng, S, n)
        draft = make_rows(rng, S, n, N, D)
        qt = do.bf16(rng.normal(size=(S, n, H, D)))
        check_tree(case, qt, parent, draft, tree_gpu(case, qt, parent, draft))
        lines = [sorted(do.line_of(parent[s], int(max(np.nonzero(parent[s] > -2)[0])))) for s in range(S)]
        m = max(map(len, lines))
        kv = np.zeros((S, m, 2, N, D))
        for s in range(S):
            kv[s, : len(lines[s])] = draft[s, lines[s]]
            rows[s, case.lens[s]: case.lens[s] + len(lines[s])] = draft[s, lines[s]]
        case.c.write(to_bf16(kv.reshape(S, m, -1)), case.len, i32([len(x) for x in lines]))
        case.lens = [a + len(x) for a, x in zip(case.lens, lines)]
        case.len = i32(case.lens)
        case.check_all()
    # the last selection's tokens as the sparse layers' index set
    sel = np.full((S, 32 * 5), -1, np.int32)
    for s in range(S):
        t = [32 * b + i for b in blocks[s, 0] if b >= 0 for i in range(32)]
        sel[s, : len(t)] = t
    k = out_buffer((S, sel.shape[1], N * D), torch.bfloat16)
    v = out_buffer(k.shape, k.dtype)
    case.c.read(case.len, i32(sel), k, v)
    p = rkv.make_params(1, S, T, N, D, 256, 256)
    out = out_buffer((S, H, D), torch.float32)
    ws = out_buffer((max(rkv.rkv_attention_workspace(p, H, sel.shape[1]), 256),), torch.uint8)
    rkv.rkv_sparse_attention(p, H, to_bf16(q), k, v, i32(sel), sel.shape[1], out, ws, ws.numel())
    out = out.double().cpu().numpy()
    for s in range(S):
        K, V, _ = case.held(s)
        t = sel[s][sel[s] >= 0]
        for h in range(H):
            want, tol = do.attend(q[s, h], K[t, h // G], V[t, h // G])
            assert np.all(np.abs(out[s, h] - want) <= tol)
    case.done()


def test_captured_steps_replay_on_new_lengths_and_other_streams():
    """A decode step (write, select, attend, tree) in a graph: replays follow pos and len, two
    graphs of one cache share no scratch, and a stream of the caller's gives the same bits."""
    rng = np.random.default_rng(51)
    S, N, G, D, T = 2, 2, 4, 128, 2100
    H, n = N * G, 6
    rows = make_rows(rng, S, T, N, D)
    start = [2050, 1000]
    case = Case(rows, start, 4, T=T)
    q, qt = do.bf16(rng.normal(size=(S, H, D))), do.bf16(rng.normal(size=(S, n, H, D)))
    draft, parent = make_rows(rng, S, n, N, D), random_tree(rng, S, n)
    kv_d, pos, length = torch.empty(S, 1, 2 * N * D, dtype=torch.bfloat16, device="cuda"), i32(start), i32(start)
    q_d, qt_d, dr_d, pa_d = to_bf16(q), to_bf16(qt), to_bf16(draft.reshape(S, n, -1)), i32(parent)

    def outputs():
        return [torch.empty(S, N, 9, dtype=torch.int32, device="cuda"), torch.empty(S, H, D, device="cuda"),
                torch.empty(S, n, H, D, device="cuda")]

    def step(o, stream=None):
        case.c.write(kv_d, pos, stream=stream)
        case.c.select(H, q_d, length, o[0], 1, 1, stream=stream)
        case.c.attend(H, q_d, length, o[1], blocks=o[0], stream=stream)
        case.c.tree_attend(H, qt_d, pa_d, dr_d, length, o[2], stream=stream)

    def put(i):
        kv_d.copy_(to_bf16(np.stack([rows[s, start[s] + i] for s in range(S)]).reshape(S, 1, -1)))
        pos.copy_(i32([a + i for a in start]))
        length.copy_(i32([a + i + 1 for a in start]))

    put(0)
    o = [outputs() for _ in range(3)]
    step(o[0])
    torch.cuda.synchronize()
    graphs = []
    for k in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o[k])
        graphs.append(g)
    side = torch.cuda.Stream()
    for i in range(34):
        put(i)
        step(o[0])
        want = [t.clone() for t in o[0]]
        torch.cuda.synchronize()
        # both graphs at once on two streams: they write the same rows with the same values
        with torch.cuda.stream(side):
            graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        for k in (1, 2):
            for a, b in zip(want, o[k]):
                assert torch.equal(a, b), (i, k)
    for t in o[0]:
        t.zero_()
    torch.cuda.synchronize()
    step(o[0], stream=side)
    side.synchronize()
    for a, b in zip(want, o[0]):
        assert torch.equal(a, b)
    case.lens = [a + 34 for a in start]
    case.len = i32(case.lens)
    case.check_all()


def test_many_sequences_of_all_lengths():
    # more sequences than a warp has lanes, empty ones among them, one far longer than the rest:
    # single tokens, lists and trees, for both ways of cutting the blocks into runs (fewer
    # sequences than runs, and more)
    rng = np.random.default_rng(71)
    for S, N, G, n in ((35, 8, 1, 6), (70, 1, 2, 20)):
        lens = [int(x) for x in rng.integers(0, 130, S)]
        lens[0], lens[7], lens[33], lens[S - 1] = 0, 1600, 64, 1
        case = Case(make_rows(rng, S, 1600, N, 64), lens, 4)
        q = do.bf16(rng.normal(size=(S, N * G, 64)))
        check_attend(case, q, attend_gpu(case, q))
        blocks = select_gpu(case, q, N, 3, 1, 0)
        for s in range(S):
            assert np.array_equal(blocks[s], do.select(q[s], case.held(s)[2], 3, 1, 0, False))
        check_attend(case, q, attend_gpu(case, q, blocks), blocks)
        qt, draft, parent = do.bf16(rng.normal(size=(S, n, N * G, 64))), make_rows(rng, S, n, N, 64), random_tree(rng, S, n)
        check_tree(case, qt, parent, draft, tree_gpu(case, qt, parent, draft))
        case.done()


@pytest.mark.parametrize("D,bits,G,n", [(64, 4, 2, 17), (128, 4, 4, 10), (128, 2, 4, 33), (64, 2, 4, 40)])
def test_trees_over_many_short_sequences_among_long_ones(D, bits, G, n):
    # 16 blocks at least go to one CTA: a dozen sequences of one block, in which half of the CTA
    # has nothing to do, then sequences of more, and a long one that several share
    rng = np.random.default_rng(n)
    lens = [32 + i % 32 for i in range(23)] + [31, 0, 70, 96, 129, 700] + [33] * 7 + [224, 64, 5] + [40] * 6 + [600, 32]
    S = len(lens)
    case = Case(make_rows(rng, S, 705, 1, D), lens, bits)
    q = do.bf16(rng.normal(size=(S, n, G, D)) * 1.5)
    draft = make_rows(rng, S, n, 1, D)
    parent = random_tree(rng, S, n)
    for dtype in (torch.float32, torch.bfloat16):
        got = tree_gpu(case, q, parent, draft, dtype)
        again = tree_gpu(case, q, parent, draft, dtype)
        assert np.array_equal(got, again)
        check_tree(case, q, parent, draft, got, dtype == torch.bfloat16)
    case.done()


def test_hundreds_of_sequences():
    # more than 256, which are passed over at once where none of them is a CTA's; empty ones, and
    # one long one beyond the first 256
    rng = np.random.default_rng(5)
    S = 601
    lens = [int(x) for x in rng.integers(0, 100, S)]
    lens[0], lens[255], lens[256], lens[511], lens[580] = 31, 0, 64, 1, 640
    case = Case(make_rows(rng, S, 650, 1, 64), lens, 4)
    q = do.bf16(rng.normal(size=(S, 2, 64)))
    check_attend(case, q, attend_gpu(case, q))
    blocks = rng.integers(-1, 3, (S, 1, 4)).astype(np.int32)
    blocks[(blocks >= np.array(lens)[:, None, None] // 32)] = -1
    check_attend(case, q, attend_gpu(case, q, blocks), blocks)
    for n in (3, 17):
        qt, draft, parent = do.bf16(rng.normal(size=(S, n, 2, 64))), make_rows(rng, S, n, 1, 64), random_tree(rng, S, n)
        check_tree(case, qt, parent, draft, tree_gpu(case, qt, parent, draft))
    case.done()


def test_selection_over_more_blocks_than_shared_memory_holds():
    # 42000 blocks of one head; all keys equal but for nine blocks that stand out: those, the
    # kept ends, and the lowest of the others
    ensure_lib()
    T = 42000 * 32 + 5
    c = rkv.DenseCache(rkv.make_dense_params(1, T, 1, 64, 2), guard=GUARD)
    kv = torch.full((1, T, 128), 0.5, dtype=torch.bfloat16, device="cuda")
    high = [3, 40959, 40960, 40961, 41000, 20000, 20001, 77, 39999]
    for b in high:
        kv[0, 32 * b + b % 32, 9] = 2.0
    c.write(kv, i32([0]))
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for n, first, last in ((9, 0, 0), (40, 1, 2), (5000, 3, 0), (5, 0, 0)):
        blocks = out_buffer((1, 1, n), torch.int32)
        c.select(1, q, i32([T]), blocks, keep_first=first, keep_last=last)
        want = set(range(first)) | set(range(42000 - last, 42000))
        for b in sorted(high) + list(range(42000)):
            if len(want) < n:
                want.add(b)
        assert blocks[0, 0].tolist() == sorted(want), n
    torch.cuda.synchronize()
    assert c.device_status() == 0 and not c.guard_violations()
    assert_guards()


def test_a_sequence_is_cut_back_or_begun_anew_at_a_block():
    rng = np.random.default_rng(81)
    rows = make_rows(rng, 2, 200, 2, 64)
    case = Case(rows, [200, 150], 4)
    new = make_rows(rng, 2, 75, 2, 64)
    case.c.write(to_bf16(new.reshape(2, 75, -1)), i32([96, 0]), i32([75, 50]))
    rows[0, 96:171], rows[1, :50] = new[0], new[1, :50]
    case.lens = [171, 50]
    case.len = i32(case.lens)
    case.check_all()


def test_readers_of_one_cache_at_once():
    # single tokens and a tree on two streams, over and over: each with scratch of its own
    rng = np.random.default_rng(91)
    case = Case(make_rows(rng, 2, 3000, 2, 128), [3000, 1700], 4)
    q, qt = to_bf16(rng.normal(size=(2, 8, 128))), to_bf16(rng.normal(size=(2, 16, 8, 128)))
    dr, pa = to_bf16(rng.normal(size=(2, 16, 512))), i32(random_tree(rng, 2, 16))
    outs = [torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 16, 8, 128, device="cuda")]
    c = rkv.DenseCache(case.c.p)
    c.write(to_bf16(case.rows.reshape(2, 3000, -1)), i32([0, 0]), case.len)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = None
    for i in range(30):
        outs[0].zero_(), outs[1].zero_()
        torch.cuda.synchronize()
        c.attend(8, q, case.len, outs[0], stream=streams[0])
        c.tree_attend(8, qt, pa, dr, case.len, outs[1], stream=streams[1].cuda_stream)
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        if want is None:
            want = got
            assert all(o.isfinite().all() for o in outs)
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i


def test_offsets_past_32_bits():
    # 2000 sequences: codes, input rows and outputs pass 2^32 bytes; the last one is checked
    S, N, D, T = 2000, 8, 128, 1920
    p = rkv.make_dense_params(S, T, N, D, 4)
    ensure_lib()
    assert rkv.rkv_dense_sizes(p)[0] > 2 ** 32
    c = rkv.DenseCache(p)
    rng = np.random.default_rng(61)
    rows = make_rows(rng, 1, T, N, D)
    kv = torch.zeros(S, T, 2 * N * D, dtype=torch.bfloat16, device="cuda")
    kv[-1] = to_bf16(rows.reshape(T, -1))
    counts = torch.zeros(S, dtype=torch.int32, device="cuda")
    counts[-1] = T
    c.write(kv, torch.zeros_like(counts), counts)
    sel = torch.full((S, 3), -1, dtype=torch.int32, device="cuda")
    sel[-1] = torch.tensor([0, 1000, T - 1], dtype=torch.int32)
    k = torch.empty(S, 3, N * D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c.read(counts, sel, k, v)
    K, V, _ = do.held(rows[0], T, 4)
    assert np.array_equal(k[-1].double().cpu().numpy().reshape(3, N, D), K[[0, 1000, T - 1]])
    assert np.array_equal(v[-1].double().cpu().numpy().reshape(3, N, D), V[[0, 1000, T - 1]])
    q = np.zeros((S, N, D))
    q[-1] = do.bf16(rng.normal(size=(N, D)))
    out = torch.empty(S, N, D, device="cuda")
    c.attend(N, to_bf16(q), counts, out)
    out = out.double().cpu().numpy()
    assert not out[:-1].any() and c.device_status() == 0
    for h in range(N):
        want, tol = do.attend(q[-1, h], K[:, h], V[:, h])
        assert np.all(np.abs(out[-1, h] - want) <= tol)
