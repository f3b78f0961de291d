"""Block selection against rankings in exact rational numbers: scores that 53 bits do not tell apart,
and products far below what fp32 holds."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import _dense_oracle as do
from test_gpu_dense import Case, make_rows, select_gpu

pytestmark = pytest.mark.gpu


def exact_scores(q, ends):
    """[N][blocks] as Fractions; q [H][D]."""
    lo, hi = ends
    nb, N, D = lo.shape
    G = q.shape[0] // N
    fq = [[Fraction(float(x)) for x in row] for row in q]
    out = []
    for n in range(N):
        row = []
        for b in range(nb):
            fl, fh = [Fraction(float(x)) for x in lo[b, n]], [Fraction(float(x)) for x in hi[b, n]]
            row.append(max(sum(max(x * l, x * h) for x, l, h in zip(fq[n * G + g], fl, fh)) for g in range(G)))
        out.append(row)
    return out


def exact_select(scores, n_blocks):
    return [sorted(sorted(range(len(r)), key=lambda b: (-r[b], b))[:n_blocks]) for r in scores]


def check(case, q, sizes=(1, 7, 20, 41)):
    scores = exact_scores(q, case.held(0)[2])
    shared = [[max(x) for x in zip(*scores)]]
    for n in sizes:
        for lists, s in ((case.N, scores), (1, shared)):
            got = select_gpu(case, q[None], lists, n, 0, 0)[0]
            assert np.array_equal(got, exact_select(s, n)), (lists, n)
    case.done()


@pytest.mark.parametrize("D,N,G", [(64, 2, 2), (128, 1, 4), (256, 3, 5)])
def test_scores_that_differ_beyond_53_bits(D, N, G):
    # one channel of 2^40 in every block, one of 1 .. 2 times 2^-21 that differs: constant groups are
    # held exactly, and the sums differ from their 62nd bit on
    rng = np.random.default_rng(D)
    nb = 60
    rows = np.zeros((1, nb, 32, 2, N, D))
    rows[..., 0, :, 3] = 2.0 ** 40
    rows[0, :, :, 0, :, D - 5] = (1 + rng.integers(0, 128, (nb, 1, N)) / 128) * 2.0 ** (-21 + rng.integers(0, 2, (nb, 1, N)))
    case = Case(do.bf16(rows.reshape(1, nb * 32, 2, N, D)), [nb * 32], 4)
    q = np.zeros((N * G, D))
    q[:, 3] = q[:, D - 5] = 1.0
    q[1::G, 3] = 0.5
    check(case, q)


@pytest.mark.parametrize("D,bits", [(64, 2), (128, 4)])
def test_products_below_the_range_of_fp32(D, bits):
    # queries and keys of about 2^-70, a few products of them in reach of fp32's smallest numbers
    rng = np.random.default_rng(D + bits)
    rows = make_rows(rng, 1, 50 * 32, 2, D) * 2.0 ** -70
    case = Case(rows, [50 * 32], bits)
    q = do.bf16(rng.normal(size=(4, D)) * 2.0 ** rng.integers(-80, -60, (4, D)))
    check(case, q)


def test_scores_beyond_the_range_of_fp32():
    # sums of magnitudes that fp32 does not hold: ranked by what a double tells apart
    rng = np.random.default_rng(7)
    rows = make_rows(rng, 1, 45 * 32, 2, 64) * 2.0 ** 90
    case = Case(rows, [45 * 32], 4)
    check(case, do.bf16(rng.normal(size=(4, 64)) * 2.0 ** 60))


def test_ordinary_scores_against_rational_numbers():
    rng = np.random.default_rng(8)
    case = Case(make_rows(rng, 1, 50 * 32, 2, 64), [50 * 32], 4)
    check(case, do.bf16(rng.normal(size=(6, 64))))
