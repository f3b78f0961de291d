"""How far fp32 rotations are from their definition in 64 bits as a whole (relative norms over the outputs),
against the plain form in fp32 whose angles are exact: cosines and sines rounded once, products and their sum
rounded one after another.  The bounds of tests/test_gpu_rotate.py hold for the worst case of every value and do
not tell how an angle was rounded.

What the kernel rounds beside that: the rest of an angle to 24 bits, 2^-28 of a turn or 2.3e-8 at most, as a uniform error
1.4e-8 / 1.5 in the mean over rests of all sizes; what it rounds less: one of the products, which is fused.  Next to
the plain form's 4.2e-8, in quadrature, that is below a tenth; an angle rounded to 24 bits as a whole, 2^-26 of a
turn or 9.4e-8 at most, adds a third."""
import numpy as np
import pytest
import torch

import _prompt_oracle as po
from _gpu_common import GUARD, assert_guards, ensure_lib
from reference_residual_kv_gb300 import rkv

pytestmark = pytest.mark.gpu
F32 = torch.float32


def off(got, want):
    return float(np.linalg.norm(got.astype(np.float64) - want) / np.linalg.norm(want))


@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_fp32_rotations_are_as_far_off_as_fp32_arithmetic(D, R, layout):
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(D)
    rows, H, N = 700, 4, 2
    q, k = (torch.randn(rows, h, D, generator=gen, device="cuda") for h in (H, N))
    pos = torch.randint(0, 131072, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    heads = rkv.PromptHeads(H, N, D, guard=GUARD)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    heads.rotate(rkv.make_rope(D, R, layout), q, k, pos, qo, ko)
    assert_guards(heads)
    assert heads.device_status() == 0
    th, _ = po.theta(R, 10000.0)
    at = pos.cpu().numpy()
    ang = np.outer(at.astype(np.float64), th)[:, None]
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if layout == "pairs" else (slice(0, R // 2), slice(R // 2, R))
    for x, got in ((q, qo), (k, ko)):
        x = x.cpu().numpy()
        want, _ = po.rotate(x.astype(np.float64), at, th, 1.0, layout)
        plain = x.copy()
        plain[..., a], plain[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        assert off(got.cpu().numpy(), want) <= 1.1 * off(plain, want)


def test_quarter_and_eighth_turns():
    # angles on and next to the borders between quarters, by frequencies of the caller's own: the nearest fp32 cosine and
    # sine to two units of their last place
    ensure_lib()
    D = 64
    rope = rkv.make_rope(D, D, "pairs")
    turns = [f % 2 ** 64 for e in range(0, 8) for f in ((e << 61), (e << 61) + 2 ** 32, (e << 61) - 2 ** 32, (e << 61) + 12345678901234567)]
    assert len(turns) == D // 2
    for i, t in enumerate(turns):
        rope.turn[i] = t
    x = torch.zeros(3, 1, D, device="cuda")
    x[..., 0::2] = 1.0
    pos = torch.tensor([1, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    heads, out = rkv.PromptHeads(1, 1, D, guard=GUARD), torch.empty_like(x)
    heads.rotate(rope, x, None, pos, out, None)
    assert_guards(heads)
    got = out.cpu().numpy().astype(np.float64)[:, 0]
    for r, p in enumerate((1, 3, 2 ** 31 - 1)):
        for i, t in enumerate(turns):
            w = (t * p) % 2 ** 64
            w = w - 2 ** 64 if w >= 2 ** 63 else w
            ang = 2 * np.pi * (w / 2.0 ** 64)
            # 32 bits of the angle are kept, 24 of its rest
            tol = 2 * np.pi * (2.0 ** -32 + 2.0 ** -28) + 2 * 2.0 ** -24
            assert abs(got[r, 2 * i] - np.cos(ang)) <= tol and abs(got[r, 2 * i + 1] - np.sin(ang)) <= tol, (p, i)
            if w % 2 ** 62 == 0:
                exact = {0: (1, 0), 1: (0, 1), 2: (-1, 0), 3: (0, -1)}[(w >> 62) % 4]
                assert (got[r, 2 * i], got[r, 2 * i + 1]) == exact
