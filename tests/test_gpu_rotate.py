"""Norm and rotation of queries and keys on the GPU against their fp64 restatement."""
import numpy as np
import pytest
import torch

import _prompt_oracle as po
import oracle
from _gpu_common import GUARD, assert_guards, ensure_lib, out_buffer
from reference_residual_kv_gb300 import rkv

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def rows_of(gen, rows, heads, D, dt, wide=0):
    """[rows][heads][D], rows `wide` further elements apart."""
    x = torch.randn(rows, heads * D + wide, generator=gen, device="cuda", dtype=F32).mul_(1.5).to(dt)
    return x[:, : heads * D].view(rows, heads, D) if wide == 0 else x[:, : heads * D].unflatten(1, (heads, D))


def tolerance(want, mag, dt, normed):
    """Half a step of the type, and fp32 errors in units of 2^-24 of the pair's magnitude: the angle
    (half a turn to 24 bits: pi), sine and cosine (2 each), the gain (2), products and their sum (3);
    with a norm 16 + log2(D) roundings of the sum of squares, halved by the root, the root's 2 ulp
    and two products."""
    return torch.finfo(dt).eps / 2 * np.abs(want) + (12 + (18 if normed else 0)) * 2.0 ** -24 * mag + 1e-37


def check(got, x, pos, th, gain, layout, w, dt):
    want, mag = po.rotate(x.double().cpu().numpy(), pos, th, gain, layout, None if w is None else w.double().cpu().numpy())
    err = np.abs(got.double().cpu().numpy() - want)
    tol = tolerance(want, mag, dt, w is not None)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48), (256, 256), (256, 128), (128, 0)])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("normed", [False, True])
def test_heads_and_types(D, R, layout, dt, normed):
    ensure_lib()
    for rows, H, N, wide in ((1, 1, 1, 0), (5, 7, 1, 16), (67, 28, 4, 0), (33, 6, 3, 8)):
        gen = torch.Generator(device="cuda").manual_seed(rows * 1000 + D)
        q, k = rows_of(gen, rows, H, D, dt, wide), rows_of(gen, rows, N, D, dt, wide)
        pos = torch.randint(0, 131072, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        w = [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) if normed else None for _ in range(2)]
        h = rkv.PromptHeads(H, N, D, guard=GUARD)
        rope = rkv.make_rope(D, R, layout, 10000.0)
        qo, ko = out_buffer((rows, H, D), dt), out_buffer((rows, N, D), dt)
        h.rotate(rope, q, k, pos, qo, ko, *w)
        assert_guards(h)
        assert h.device_status() == 0
        th, gain = po.theta(R, 10000.0)
        for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
            check(got, x, pos.cpu().numpy(), th, gain, layout, wt, dt)


@pytest.mark.parametrize("scaling", [("linear", 4.0), ("bands", 8.0, 8192, 1.0, 4.0), ("yarn", 8.0, 8192, 32.0, 1.0)])
def test_scaled_and_far_positions(scaling):
    ensure_lib()
    rows, H, N, D = 40, 4, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = rows_of(gen, rows, H, D, F32), rows_of(gen, rows, N, D, F32)
    # the last ones lie where fp32 angles would be off by whole radians; fp64's own are off by
    # 2^31 2^-53 in the oracle
    pos = torch.tensor([0, 1, 2, 3] + [7919 * i for i in range(30)] + [2 ** 24 + 1, 2 ** 27, 10 ** 9, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1],
                       dtype=torch.int32, device="cuda")
    h = rkv.PromptHeads(H, N, D)
    for layout in ("pairs", "halves"):
        qo, ko = out_buffer((rows, H, D), F32), out_buffer((rows, N, D), F32)
        h.rotate(rkv.make_rope(D, None, layout, 500000.0, scaling), q, k, pos, qo, ko)
        assert_guards()
        th, gain = po.theta(D, 500000.0, scaling)
        p = pos.cpu().numpy().astype(np.float64)
        for got, x in ((qo, q), (ko, k)):
            want, mag = po.rotate(x.double().cpu().numpy(), p, th, gain, layout)
            # the frequency itself: a few 2^-53, times the position
            tol = tolerance(want, mag, F32, False) + (p * 2.0 ** -49)[:, None, None] * mag
            assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def test_in_place_padding_and_one_side():
    ensure_lib()
    rows, H, N, D = 50, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    p = torch.randn(rows, (H + 2 * N) * D, generator=gen, device="cuda").to(BF16)
    q, k = p[:, : H * D].unflatten(1, (H, D)), p[:, H * D: (H + N) * D].unflatten(1, (N, D))
    before = p.clone()
    pos = torch.randint(0, 9000, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    pos[::7] = -1
    h = rkv.PromptHeads(H, N, D)
    rope = rkv.make_rope(D, 64, "halves")
    qo, ko = out_buffer((rows, H, D), BF16), out_buffer((rows, N, D), BF16)
    qo.fill_(7.0)
    ko.fill_(7.0)
    h.rotate(rope, q, k, pos, qo, ko)
    assert_guards()
    assert bool((qo[::7] == 7.0).all()) and bool((ko[::7] == 7.0).all())
    assert torch.equal(p, before)
    # in place, queries and keys by themselves: the same bits, padding rows and V untouched
    h.rotate(rope, q, None, pos, q, None)
    h.rotate(rope, None, k, pos, None, k)
    live = pos >= 0
    assert torch.equal(q[live], qo[live]) and torch.equal(k[live], ko[live])
    assert torch.equal(p[::7], before[::7]) and torch.equal(p[:, (H + N) * D:], before[:, (H + N) * D:])
    assert h.device_status() == 0
    # a position below -1 is an error, its row is left alone, the others are done
    pos[3] = -5
    qo.fill_(7.0)
    h.rotate(rope, qo.clone(), None, pos, qo, None)
    assert h.device_status() == rkv.RKV_ERR_INDEX
    assert bool((qo[3] == 7.0).all()) and not bool((qo[4] == 7.0).all())


def test_values_that_are_not_finite_stay_in_their_head():
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = rows_of(gen, 4, 8, 128, BF16).clone()
    k = rows_of(gen, 4, 2, 128, BF16).clone()
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    w = torch.ones(128, device="cuda", dtype=BF16)
    h, rope = rkv.PromptHeads(8, 2, 128), rkv.make_rope(128)
    clean = torch.empty_like(q), torch.empty_like(k)
    h.rotate(rope, q, k, pos, *clean, w, w)
    q[1, 3, 5], q[2, 7, 100], k[0, 1, 0] = float("nan"), float("inf"), -float("inf")
    got = torch.empty_like(q), torch.empty_like(k)
    h.rotate(rope, q, k, pos, *got, w, w)
    for a, b, hurt in ((got[0], clean[0], [(1, 3), (2, 7)]), (got[1], clean[1], [(0, 1)])):
        same = (a == b).all(-1)
        for at in hurt:
            assert not bool(same[at])
            same[at] = True
        assert bool(same.all())


def test_rotation_is_that_of_restored_keys():
    # rkv_restore_kv's rotation, as the oracle of the restore defines it
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(8)
    k = rows_of(gen, 6, 2, 128, F32)
    pos = torch.tensor([0, 1, 17, 4095, 100000, 131071], dtype=torch.int32, device="cuda")
    ko = torch.empty_like(k)
    rkv.PromptHeads(8, 2, 128).rotate(rkv.make_rope(128), None, k, pos, None, ko)
    for i, p in enumerate(pos.tolist()):
        for n in range(2):
            x = k[i, n].double().cpu().numpy()
            want = oracle.rope(x, p, 10000.0)
            mag = np.repeat(np.hypot(x[0::2], x[1::2]), 2)
            assert np.all(np.abs(ko[i, n].double().cpu().numpy() - want) <= tolerance(want, mag, F32, False))


def test_streams_and_graphs():
    ensure_lib()
    rows, H, N, D = 300, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(9)
    q, k = rows_of(gen, rows, H, D, BF16), rows_of(gen, rows, N, D, BF16)
    pos = torch.arange(rows, device="cuda", dtype=torch.int32)
    h, rope = rkv.PromptHeads(H, N, D), rkv.make_rope(D, layout="halves")
    want = torch.empty_like(q), torch.empty_like(k)
    h.rotate(rope, q, k, pos, *want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = torch.zeros_like(q), torch.zeros_like(k)
    torch.cuda.synchronize()
    h.rotate(rope, q, k, pos, *got, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        h.rotate(rope, q, k, pos, *got)
    # the rotation goes with the captured call: changing it afterwards changes nothing there
    rope.gain = 3.0
    q.mul_(-1.0)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], -want[0]) and torch.equal(got[1], want[1])
