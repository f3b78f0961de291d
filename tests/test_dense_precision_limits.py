"""What the limits of test_gpu_dense_precision.py can tell apart, worked out on the host from the same
data: probabilities in one, two and three bf16 parts, and scores summed in fp32, each alone."""
import numpy as np
import pytest

import _dense_oracle as do
from test_gpu_dense import make_rows
from test_gpu_dense_precision import BF16_MORE, F32_OFF, SINGLE, TREES, off


def in_parts(p, parts):
    p = p.astype(np.float32).astype(np.float64)
    out = np.zeros_like(p)
    for _ in range(parts):
        out += do.bf16(p - out)
    return out


@pytest.mark.parametrize("D,bits,G,n", TREES + [(D, bits, G, 1) for D, bits, G in SINGLE])
def test_fewer_parts_of_the_probabilities_pass_the_limits(D, bits, G, n):
    rng = np.random.default_rng(D + 10 * bits + n)
    K, V, _ = do.held(make_rows(rng, 1, 1500, 1, D)[0], 1500, bits)
    q = do.bf16(rng.normal(size=(n * G, D)) * 1.5)
    x = q @ K[:, 0].T / np.sqrt(D)
    p = np.exp(x - x.max(axis=1, keepdims=True))
    total, v = p.sum(axis=1, keepdims=True), V[:, 0]
    want = p / total @ v
    one, two, three = (in_parts(p, k) / total @ v for k in (1, 2, 3))
    x32 = (q.astype(np.float32) @ K[:, 0].T.astype(np.float32)).astype(np.float64) / np.sqrt(D)
    p32 = np.exp(x32 - x32.max(axis=1, keepdims=True))
    scores = p32 / p32.sum(axis=1, keepdims=True) @ v
    # fp32 outputs: two parts fail, three leave room for all else that is fp32
    assert off(two, want) > 1.2 * F32_OFF
    assert off(three, want) + off(scores, want) < F32_OFF / 2
    # bf16 outputs: one part fails, two do not
    rounding = off(do.bf16(want), want)
    assert off(do.bf16(one), want) > rounding + 3 * BF16_MORE
    assert off(do.bf16(two), want) <= rounding + BF16_MORE / 2
