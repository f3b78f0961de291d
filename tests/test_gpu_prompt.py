"""Attention of packed prompts and of pieces behind their cached text, on the GPU against fp64.

Tolerance, for each value: half a step of bf16 of the result, and for the probabilities (rounded
to bf16, half a step of 2^-8 each) 2^-8 of sum(weight |v|).  Scores in fp32 with sums that the
products cut: a relative error below 2^-17 of sum |q_d k_d| scale log2(e), at most 2^5 here, and the
exponential's 2^-22: together below 2^-11 of sum(weight |v|)."""
import math

import numpy as np
import pytest
import torch

import _prompt_oracle as po
from _gpu_common import GUARD, assert_guards, ensure_lib, out_buffer
from reference_residual_kv_gb300 import rkv

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
MARK = 77.0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def near(got, want, mag):
    err, tol = (got.double() - want).abs(), HALF * want.abs() + (HALF + 2.0 ** -11) * mag + 1e-30
    assert not bool(got.isnan().any()), "NaN"
    assert bool((err <= tol).all()), "%.3g of the tolerance" % float((err / tol).max())


def packed(gen, lens, H, N, D, behind=0, fused=False):
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    rows = start[-1] + behind
    if fused:
        p = randn(gen, rows, (H + 2 * N) * D).to(BF16)
        q, k, v = (p[:, a * D: b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + N), (H + N, H + 2 * N)))
    else:
        q, k, v = randn(gen, rows, H, D).to(BF16), randn(gen, rows, N, D).to(BF16), randn(gen, rows, N, D).to(BF16)
    return q, k, v, start


def attend(q, k, v, start, h=None, out=None):
    ensure_lib()
    h = h or rkv.PromptHeads(q.shape[1], k.shape[1], q.shape[2], guard=GUARD)
    if out is None:
        out = out_buffer(q.shape, BF16)
        out.fill_(MARK)
    h.attend(q, k, v, i32(start), out)
    assert_guards(h)
    assert h.device_status() == 0
    return out


def check(q, k, v, start, out):
    rows = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for a, b in zip(start[:-1], start[1:]):
        if b > a:
            want, mag = po.causal(q[a:b].double(), k[a:b].double(), v[a:b].double())
            near(out[a:b], want, mag)
            rows[a:b] = True
    assert bool((out[~rows] == MARK).all()), "rows of no prompt were written"


EDGES = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,N", [(1, 1), (2, 1), (6, 2), (8, 2), (7, 1), (16, 2), (3, 3)])
def test_lengths_at_the_tiles_edges(D, H, N):
    gen = torch.Generator(device="cuda").manual_seed(D + H)
    q, k, v, start = packed(gen, EDGES + [0, 0, 5, 0], H, N, D, behind=9)
    check(q, k, v, start, attend(q, k, v, start))


@pytest.mark.parametrize("lens,H,N,D,fused", [
    ([700], 8, 2, 128, True), ([1500, 0, 1, 37], 28, 4, 128, False), ([2000], 4, 4, 64, True), ([900, 900], 8, 1, 256, True),
    ([4096], 2, 1, 128, False), ([5000], 1, 1, 64, False), ([3000, 2999], 2, 2, 128, True), ([2500], 1, 1, 256, False)])
def test_longer_prompts(lens, H, N, D, fused):
    # the last ones have few items, which are split over the keys
    gen = torch.Generator(device="cuda").manual_seed(len(lens) + H)
    q, k, v, start = packed(gen, lens, H, N, D, behind=3, fused=fused)
    check(q, k, v, start, attend(q, k, v, start))


def test_more_keys_than_stay_in_l2():
    # items go by sequence and KV head there
    gen = torch.Generator(device="cuda").manual_seed(11)
    q, k, v, start = packed(gen, [9000, 4, 16000, 700], 8, 8, 128)
    out = attend(q, k, v, start)
    for a, b in zip(start[:-1], start[1:]):
        for h in (0, 7):
            want, mag = po.causal(q[a:b, h: h + 1].double(), k[a:b, h: h + 1].double(), v[a:b, h: h + 1].double())
            near(out[a:b, h: h + 1], want, mag)
    # every head and row by itself: each must be what the same call gives for that sequence alone
    alone = attend(q[start[1]: start[2]].contiguous(), k[start[1]: start[2]].contiguous(), v[start[1]: start[2]].contiguous(), [0, 4])
    near(out[start[1]: start[2]], *po.causal(q[start[1]: start[2]].double(), k[start[1]: start[2]].double(), v[start[1]: start[2]].double()))
    assert bool(((out[start[1]: start[2]].double() - alone.double()).abs() <= 2 * HALF * alone.double().abs() + 1e-3).all())


def test_many_heads_of_more_keys_than_stay_in_l2():
    # items by sequence and KV head
    gen = torch.Generator(device="cuda").manual_seed(19)
    q, k, v, start = packed(gen, [9000, 4, 8000, 0, 700, 5000, 3000], 32, 8, 128, behind=5)
    out = attend(q, k, v, start)
    for a, b in zip(start[:-1], start[1:]):
        for h in (0, 13, 31):
            if b > a:
                want, mag = po.causal(q[a:b, h: h + 1].double(), k[a:b, h // 4: h // 4 + 1].double(), v[a:b, h // 4: h // 4 + 1].double())
                near(out[a:b, h: h + 1], want, mag)
    assert bool((out[start[-1]:] == MARK).all()) and not bool((out[: start[-1]] == MARK).all(-1).any())


@pytest.mark.parametrize("S", [2, 31, 32, 33])
def test_items_worked_out_by_the_producers(S):
    # up to 32 sequences whatever their lengths, the empty ones among them; one more goes by the plan
    gen = torch.Generator(device="cuda").manual_seed(S)
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.integers(0, 150, size=S - 1)] + [700]
    q, k, v, start = packed(gen, lens, 8, 2, 128, behind=2)
    check(q, k, v, start, attend(q, k, v, start))


def test_thousands_of_short_prompts():
    gen = torch.Generator(device="cuda").manual_seed(12)
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 12, size=2500)]
    q, k, v, start = packed(gen, lens, 4, 2, 64, behind=1)
    check(q, k, v, start, attend(q, k, v, start))


def test_scores_far_apart():
    # maxima that grow along the keys (the reference moves again and again) and fall; ties; huge and tiny scores
    gen = torch.Generator(device="cuda").manual_seed(13)
    n, H, D = 900, 4, 128
    q, k, v, start = packed(gen, [n], H, 1, D)
    q = q.clone()
    q[:, :, 0] = 8.0
    k[:, 0, 0] = torch.linspace(-60, 60, n, device="cuda").to(BF16)
    q[:, 1, 0] = -8.0
    q[:, 2] = 0.0
    q[:, 3] = (q[:, 3].float() * 20).to(BF16)
    out = attend(q, k, v, start)
    want, mag = po.causal(q.double(), k.double(), v.double())
    # sums |q k| scale log2(e) reach 8 60 / 11.3 1.44 = 61 here, 20 times the usual 12 in head 3: 2^-17 2^8 of the weights
    err, tol = (out.double() - want).abs(), HALF * want.abs() + (HALF + 2.0 ** -9) * mag + 1e-30
    assert bool((err <= tol).all())
    # equal scores: the mean of what is seen
    mean = v[:, 0].double().cumsum(0) / torch.arange(1, n + 1, device="cuda")[:, None]
    assert bool(((out[:, 2].double() - mean).abs() <= HALF * mean.abs() + 2.0 ** -11 * mag[:, 2] + HALF * mag[:, 2]).all())


@pytest.mark.parametrize("D,H,N", [(64, 4, 1), (128, 8, 2), (128, 2, 2), (256, 4, 1)])
def test_what_is_not_seen_has_no_effect(D, H, N):
    # NaN and infinities in V and K of later tokens, of the next prompt and behind the last: the rows
    # before them keep their bits
    gen = torch.Generator(device="cuda").manual_seed(14)
    lens = [200, 77, 140]
    q, k, v, start = packed(gen, lens, H, N, D, behind=20)
    clean = attend(q, k, v, start).clone()
    for at, bad in ((150, float("nan")), (277, float("inf")), (330, -float("inf")), (420, float("nan"))):
        k2, v2 = k.clone(), v.clone()
        v2[at, :, 3] = bad
        k2[at, :, 5] = bad
        v2[at + 1:] = v2[at + 1:] if at != 420 else float("nan")
        q2 = q.clone()
        if at == 420:
            q2[417:] = float("nan")
            k2[417:] = float("nan")
            v2[417:] = float("nan")
        out = attend(q2, k2, v2, start)
        for a, b in zip(start[:-1], start[1:]):
            stop = at if a <= at < b else b
            assert torch.equal(out[a:stop], clean[a:stop]), (at, a)
        assert bool((out[417:] == MARK).all())


@pytest.mark.parametrize("D,H,N", [(64, 4, 1), (128, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("n", [300, 3000])
def test_values_that_are_not_finite_are_seen_by_later_rows(D, H, N, n):
    # 3000 rows of few heads: split over the keys
    gen = torch.Generator(device="cuda").manual_seed(15)
    q, k, v, start = packed(gen, [n], H, N, D)
    clean = attend(q, k, v, start).clone()
    nan, inf = float("nan"), float("inf")
    marks = [(n - 100, 0, nan), (n - 90, 1, inf), (n - 60, 2, -inf), (n - 50, 4, inf), (n - 40, 4, -inf), (n - 30, D - 1, inf),
             (n - 20, D - 1, nan), (7, 5, inf)]
    v2 = v.clone()
    for t, d, x in marks:
        v2[t, 0, d] = x
    out = attend(q, k, v2, start)
    G = H // N
    want = torch.zeros(n, D, dtype=torch.float64, device="cuda")
    for t, d, x in marks:
        want[t:, d] += x                                    # inf - inf is NaN
    for h in range(H):
        if h >= G:
            assert torch.equal(out[:, h], clean[:, h])
            continue
        fine = want == 0
        assert torch.equal(out[:, h][fine], clean[:, h][fine])
        o = out[:, h].double()
        assert torch.equal(o[~fine].isnan(), want[~fine].isnan())
        assert torch.equal(o[~fine].nan_to_num(1.0), want[~fine].nan_to_num(1.0))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [300, 3000])
def test_a_row_leaves_its_neighbours_bits_alone(D, n):
    # maxima that grow along the keys: each row moves its reference by its own scores, whatever the rows beside it hold
    gen = torch.Generator(device="cuda").manual_seed(26)
    q, k, v, start = packed(gen, [n], 4, 1, D, behind=10)
    q = q.clone()
    q[:, :, 0] = 8.0
    k[:, 0, 0] = torch.linspace(-60, 60, n + 10, device="cuda").to(BF16)
    clean = attend(q, k, v, start).clone()
    q2 = q.clone()
    q2[77, 1] = float("nan")
    q2[n - 3, 2] = float("inf")
    q2[n:] = float("nan")
    out = attend(q2, k, v, start)
    others = torch.ones(n, 4, dtype=torch.bool, device="cuda")
    others[77, 1] = others[n - 3, 2] = False
    assert torch.equal(out[:n][others], clean[:n][others])
    assert bool(out[77, 1].isnan().all()) and bool(out[n - 3, 2].isnan().all())
    assert bool((out[n:] == MARK).all())


@pytest.mark.parametrize("lens,H,N,D,fused", [([1], 8, 2, 128, True), ([1], 1, 1, 64, False), ([300, 5, 1000], 8, 2, 128, True),
                                              ([2500], 1, 1, 256, False), ([100] * 40, 7, 1, 64, True), ([3500], 2, 1, 128, True)])
def test_outputs_over_the_queries(lens, H, N, D, fused):
    # one row; whole items, items split over the keys, items of the plan
    gen = torch.Generator(device="cuda").manual_seed(27)
    q, k, v, start = packed(gen, lens, H, N, D, fused=fused)
    want = attend(q, k, v, start).clone()
    check(q, k, v, start, want)
    before = k.clone(), v.clone()
    assert attend(q, k, v, start, out=q).data_ptr() == q.data_ptr()
    assert torch.equal(q, want) and torch.equal(k, before[0]) and torch.equal(v, before[1])


def test_bad_starts_write_nothing():
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(16)
    q, k, v, _ = packed(gen, [100], 8, 2, 128)
    for start in ([0, 50, 40, 100], [-1, 100], [0, 101], [0, 100, 0, 100, 0, 100], [60, 100, 2 ** 31 - 1]):
        h = rkv.PromptHeads(8, 2, 128, guard=GUARD)
        out = out_buffer(q.shape, BF16)
        out.fill_(MARK)
        h.attend(q, k, v, i32(start), out)
        assert_guards(h)
        assert h.device_status() == rkv.RKV_ERR_INDEX and bool((out == MARK).all())
    # a first prompt that begins later, and no prompt at all
    out = attend(q, k, v, [30, 90])
    near(out[30:90], *po.causal(q[30:90].double(), k[30:90].double(), v[30:90].double()))
    assert bool((out[:30] == MARK).all()) and bool((out[90:] == MARK).all())
    assert bool((attend(q, k, v, [0]) == MARK).all())
    assert bool((attend(q, k, v, [20, 20, 20]) == MARK).all())
    assert attend(q[:0], k[:0], v[:0], [0, 0]).shape[0] == 0


def test_strided_outputs_and_views():
    gen = torch.Generator(device="cuda").manual_seed(17)
    q, k, v, start = packed(gen, [130, 70], 8, 2, 128, fused=True)
    wide = torch.full((200, 12, 128), MARK, dtype=BF16, device="cuda")
    attend(q, k, v, start, out=wide[:, 2:10])
    check(q, k, v, start, wide[:, 2:10].contiguous())
    assert bool((wide[:, :2] == MARK).all()) and bool((wide[:, 10:] == MARK).all())


def test_the_same_bits_again_on_streams_and_in_graphs():
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(18)
    # the second one is split over the keys
    cases = [packed(gen, [500, 20, 90], 8, 2, 128), packed(gen, [3500], 2, 1, 128)]
    want = [attend(*c).clone() for c in cases]
    heads = [rkv.PromptHeads(c[0].shape[1], c[1].shape[1], 128) for c in cases]
    starts = [i32(c[3]) for c in cases]
    outs = [torch.zeros_like(c[0]) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):                                     # two calls at once, each with its own scratch
        for c, h, st, o, s in zip(cases, heads, starts, outs, streams):
            h.attend(c[0], c[1], c[2], st, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for c, h, st, o in zip(cases, heads, starts, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h.attend(c[0], c[1], c[2], st, o)
        graphs.append(g)
        o.zero_()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # the captured call reads its starts when it runs
    starts[0].copy_(i32([0, 250, 400, 610]))
    outs[0].fill_(MARK)
    graphs[0].replay()
    torch.cuda.synchronize()
    q, k, v, _ = cases[0]
    check(q, k, v, [0, 250, 400, 610], outs[0])
    assert all(h.device_status() == 0 for h in heads)


# ------------------------------------------------------------------ pieces behind their cached text
def rows_kv(gen, S, n, N, D):
    return randn(gen, S, n, 2 * N * D).to(BF16)


def cache_with(kv, lens, T, N, D, bits):
    ensure_lib()
    S = kv.shape[0]
    c = rkv.DenseCache(rkv.make_dense_params(S, T, N, D, bits), guard=GUARD)
    for t in (c.codes, c.khdr, c.tail):
        t.fill_(0xFF)                                       # NaN everywhere that is not written
    if kv.shape[1]:
        c.write(kv, i32([0] * S), i32(lens))
    return c


def held(c, lens):
    """K and V [S][T][N][D] float64 of the cached tokens, as they are read back."""
    S, N, D, m = c.S, c.N, c.D, max(lens)
    sel = torch.arange(m, device="cuda", dtype=torch.int32).expand(S, m)
    sel = torch.where(sel < i32(lens)[:, None], sel, -1).contiguous()
    k, v = torch.zeros(S, m, N * D, dtype=BF16, device="cuda"), torch.zeros(S, m, N * D, dtype=BF16, device="cuda")
    if m:
        c.read(i32(lens), sel, k, v)
    return k.double().view(S, m, N, D), v.double().view(S, m, N, D)


def piece(c, H, q, kv, lens, new):
    out = out_buffer(q.shape, BF16)
    out.fill_(MARK)
    c.chunk_attend(H, q, kv, i32(lens), out, n_new=None if new is None else i32(new))
    assert_guards(c)
    assert c.device_status() == 0
    return out


def check_piece(c, H, q, kv, lens, new, out):
    S, n = q.shape[:2]
    k0, v0 = held(c, lens)
    x = kv.double().view(S, n, 2, c.N, c.D)
    for s in range(S):
        m, a = lens[s], n if new is None else new[s]
        if a:
            want, mag = po.causal(q[s, :a].double(), torch.cat([k0[s, :m], x[s, :a, 0]]), torch.cat([v0[s, :m], x[s, :a, 1]]), m)
            near(out[s, :a], want, mag)
        assert bool((out[s, a:] == MARK).all()), "rows behind the piece were written"


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("H,N,D", [(8, 2, 128), (7, 1, 64), (3, 3, 128), (8, 1, 256)])
@pytest.mark.parametrize("n", [1, 33, 64, 65, 200])
def test_pieces(bits, H, N, D, n):
    # short pieces go as drafted trees do
    gen = torch.Generator(device="cuda").manual_seed(n + D)
    lens = [0, 1, 31, 32, 33, 64, 500, 777]
    new = [n, max(1, n - 1), n, 0, n // 2, 1, n, max(1, n - 7)]
    c = cache_with(rows_kv(gen, 8, 777, N, D), lens, 1000, N, D, bits)
    q, kv = randn(gen, 8, n, H, D).to(BF16), rows_kv(gen, 8, n, N, D)
    for s in range(8):
        kv[s, new[s]:] = float("nan")                       # rows that are not there
        q[s, new[s]:] = float("nan")
    check_piece(c, H, q, torch.nan_to_num(kv, 0.0), lens, new, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("S,n,T,H,N,D", [(1, 300, 20000, 4, 2, 128), (3, 130, 6000, 7, 1, 128), (1, 700, 9000, 2, 2, 64),
                                         (2, 100, 7000, 8, 2, 256), (1, 2048, 2048, 8, 2, 128)])
def test_pieces_behind_long_text(S, n, T, H, N, D):
    # few items: split over the keys; the last one has no text before it
    gen = torch.Generator(device="cuda").manual_seed(T)
    lens = [T - n] + [max(0, T - n - 1000 * (s + 1)) for s in range(S - 1)]
    c = cache_with(rows_kv(gen, S, T - n, N, D), lens, T, N, D, 4)
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    out = piece(c, H, q, kv, lens, None)
    check_piece(c, H, q, kv, lens, None, out)
    again = piece(c, H, q, kv, lens, None)
    assert torch.equal(out, again)


def test_a_sequence_alone_and_in_a_batch():
    # small and large pieces side by side with sequences that have none
    gen = torch.Generator(device="cuda").manual_seed(21)
    S, n, T, H, N, D = 40, 90, 400, 4, 1, 64
    lens = [(37 * s) % 310 for s in range(S)]
    new = [(53 * s) % 91 for s in range(S)]
    c = cache_with(rows_kv(gen, S, 310, N, D), lens, T, N, D, 4)
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    check_piece(c, H, q, kv, lens, new, piece(c, H, q, kv, lens, new))


def test_pieces_of_more_keys_than_stay_in_l2():
    # items by sequence and KV head
    gen = torch.Generator(device="cuda").manual_seed(28)
    S, n, T, H, N, D = 12, 1100, 5000, 32, 4, 128
    lens = [3900 - 100 * s for s in range(S)]
    new = [n - 7 * s for s in range(S)]
    c = cache_with(rows_kv(gen, S, 3900, N, D), lens, T, N, D, 4)
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    out = piece(c, H, q, kv, lens, new)
    k0, v0 = held(c, lens)
    x = kv.double().view(S, n, 2, N, D)
    for s in range(S):
        m, a, h = lens[s], new[s], (5 * s) % H
        want, mag = po.causal(q[s, :a, h: h + 1].double(), torch.cat([k0[s, :m], x[s, :a, 0]])[:, h // 8: h // 8 + 1],
                              torch.cat([v0[s, :m], x[s, :a, 1]])[:, h // 8: h // 8 + 1], m)
        near(out[s, :a, h: h + 1], want, mag)
        assert bool((out[s, a:] == MARK).all()) and not bool((out[s, :a] == MARK).all(-1).any())


def test_hundreds_of_sequences_pieces():
    # more than the cache's way to bf16 works the items out for
    gen = torch.Generator(device="cuda").manual_seed(25)
    S, n, T, H, N, D = 300, 70, 200, 4, 2, 64
    lens = [(29 * s) % 131 for s in range(S)]
    new = [(31 * s) % 71 for s in range(S)]
    c = cache_with(rows_kv(gen, S, 130, N, D), lens, T, N, D, 2)
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    check_piece(c, H, q, kv, lens, new, piece(c, H, q, kv, lens, new))


@pytest.mark.parametrize("n", [40, 100])
def test_wrong_pieces_are_left_alone(n):
    gen = torch.Generator(device="cuda").manual_seed(22)
    S, T, H, N, D = 6, 300, 8, 2, 128
    good = [200, 0, 200, 100, 200, 150]
    c = cache_with(rows_kv(gen, S, 200, N, D), good, T, N, D, 4)
    lens, new = [200, -1, 200, 100, 301, 150], [n, n, n + 1, -2, 0, n]
    if n == 100:
        lens[5], new[5] = 201, n                            # beyond the capacity
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    out = out_buffer(q.shape, BF16)
    out.fill_(MARK)
    c.chunk_attend(H, q, kv, i32(lens), out, n_new=i32(new))
    assert_guards(c)
    assert c.device_status() == rkv.RKV_ERR_INDEX
    live = [0] if n == 100 else [0, 5]
    k0, v0 = held(c, good)
    for s in range(S):
        if s in live:
            x = kv[s].double().view(n, 2, N, D)
            near(out[s], *po.causal(q[s].double(), torch.cat([k0[s, :lens[s]], x[:, 0]]), torch.cat([v0[s, :lens[s]], x[:, 1]]), lens[s]))
        else:
            assert bool((out[s] == MARK).all()), s


def test_pieces_on_streams_and_in_graphs():
    gen = torch.Generator(device="cuda").manual_seed(23)
    S, T, H, N, D = 2, 1500, 8, 2, 128
    lens = [1200, 40]
    c = cache_with(rows_kv(gen, S, 1200, N, D), lens, T, N, D, 4)
    ln = i32(lens)
    jobs = []
    for n in (30, 200):
        q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
        jobs.append((q, kv, piece(c, H, q, kv, lens, None).clone(), torch.zeros_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, kv, _, out, s in jobs:
            c.chunk_attend(H, q, kv, ln, out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, _, want, out, _ in jobs)
    graphs = []
    for q, kv, _, out, _ in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.chunk_attend(H, q, kv, ln, out)
        graphs.append(g)
        out.zero_()
    for _ in range(3):
        for g, (_, _, _, _, s) in zip(graphs, jobs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, _, want, out, _ in jobs)


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_a_prompt_from_its_projection_to_the_next_token(layout):
    """A layer's way through a text: rows q | k | v of one projection normed and rotated in place, a
    first piece that attends over itself and is written, a second and a third piece behind it, and a
    single token over the whole cache."""
    gen = torch.Generator(device="cuda").manual_seed(24)
    H, N, D, T, bits = 8, 2, 128, 700, 4
    cuts = [0, 333, 333 + 150, 333 + 150 + 40, 333 + 150 + 41]
    n = cuts[-1]
    p = randn(gen, n, (H + 2 * N) * D).to(BF16)
    raw = p.clone()
    wq, wk = ((1 + 0.1 * randn(gen, D)).to(BF16) for _ in range(2))
    q, k, v = p[:, : H * D].unflatten(1, (H, D)), p[:, H * D: (H + N) * D].unflatten(1, (N, D)), p[:, (H + N) * D:].unflatten(1, (N, D))
    heads = rkv.PromptHeads(H, N, D, guard=GUARD)
    rope = rkv.make_rope(D, layout=layout)
    c = rkv.DenseCache(rkv.make_dense_params(1, T, N, D, bits), guard=GUARD)
    out = torch.empty(n, H, D, dtype=BF16, device="cuda")
    ensure_lib()
    heads.rotate(rope, q, k, torch.arange(n, device="cuda", dtype=torch.int32), q, k, wq, wk)
    th, _ = po.theta(D, 10000.0)
    for got, x, w in ((q, raw[:, : H * D].unflatten(1, (H, D)), wq), (k, raw[:, H * D: (H + N) * D].unflatten(1, (N, D)), wk)):
        want, mag = po.rotate(x.double().cpu().numpy(), np.arange(n), th, 1.0, layout, w.double().cpu().numpy())
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= HALF * np.abs(want) + 30 * 2.0 ** -24 * mag)
    for i, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
        kv = p[None, a:b, H * D:].contiguous()
        if i == 0:
            heads.attend(q[a:b], k[a:b], v[a:b], i32([0, b - a]), out[a:b])
            before_k, before_v = k[:0].double(), v[:0].double()
        elif b - a > 1:
            before_k, before_v = (x[0] for x in held(c, [a]))
            o = torch.empty(1, b - a, H, D, dtype=BF16, device="cuda")
            c.chunk_attend(H, q[a:b][None].contiguous(), kv, i32([a]), o)
            out[a:b] = o[0]
        c.write(kv, i32([a]))
        if b - a > 1:
            want, mag = po.causal(q[a:b].double(), torch.cat([before_k, k[a:b].double()]), torch.cat([before_v, v[a:b].double()]), a)
            near(out[a:b], want, mag)
        else:
            before_k, before_v = (x[0] for x in held(c, [b]))
            o = torch.empty(1, H, D, dtype=BF16, device="cuda")
            c.attend(H, q[a:b].contiguous(), i32([b]), o)
            near(o, *po.causal(q[a:b].double(), before_k, before_v, a))
    assert heads.device_status() == 0 and c.device_status() == 0
    assert_guards(heads, c)
