"""What include/rkv.h says of the probabilities of rkv_prompt_attention, by arithmetic on the CPU."""
import os
import re

import numpy as np
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "rkv.h")


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


def parts(p):
    """The two bf16 parts of fp32 probabilities: p cut off, and the rest with 2^-24 of the first, rounded."""
    hi = (p.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    rest = (p.astype(np.float64) - hi.astype(np.float64) * (1 - 2.0 ** -24)).astype(np.float32)     # one rounding, as a fused product
    return hi, bf16(rest)


def probabilities():
    rng = np.random.default_rng(5)
    # every number of 12 bits and its neighbours next to a border of the first part's and of the rest's, at random for the others
    m = np.arange(1 << 12, dtype=np.uint32) << 11
    edge = np.concatenate([m + d for d in (0, 1, 2, 127, 128, 129, 255, 256, 257, 2047)])
    p = np.concatenate([edge, rng.integers(0, 1 << 23, size=1 << 20, dtype=np.uint32)]) & np.uint32(0x7FFFFF)
    return np.concatenate([(p | np.uint32((127 + e) << 23)).view(np.float32) for e in (0, -1, -60, 10)])


def test_the_header_states_the_bound():
    with open(HEADER) as f:
        src = f.read()
    said = re.search(r"Causal attention of whole prompts.*?in two parts \(relative error 2\^-(\d+)\)", src, re.S)
    assert said
    p = probabilities()
    hi, lo = parts(p)
    worst = float((np.abs(p.astype(np.float64) - hi - lo) / p).max())
    assert 2.0 ** -(int(said.group(1)) + 1) < worst <= 2.0 ** -int(said.group(1)), worst


def test_one_part_is_off_by_half_a_step():
    # 1 + 2^-8 lies half way: 2^-8 of it, not 2^-9, and as much for the outputs' rounding
    p = probabilities()
    worst = float((np.abs(p.astype(np.float64) - bf16(p)) / p).max())
    assert 2.0 ** -8 * (1 - 2.0 ** -7) < worst <= 2.0 ** -8


def test_both_parts_are_above_zero():
    # infinities that a row sees stay infinite in the sum of both products
    hi, lo = parts(probabilities())
    assert (hi > 0).all() and (lo > 0).all()
    zero = np.zeros(1, np.float32)
    assert all(float(x[0]) == 0.0 for x in parts(zero))
