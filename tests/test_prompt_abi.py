"""Refusals, sizes and frequencies of the prompt's operators: host checks, no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import _prompt_oracle as po
from reference_residual_kv_gb300 import build, rkv

INVALID, UNSUPPORTED = rkv.RKV_ERR_INVALID_ARG, rkv.RKV_ERR_UNSUPPORTED
ALIGN, WORKSPACE = rkv.RKV_ERR_ALIGNMENT, rkv.RKV_ERR_WORKSPACE
B = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rkv.lib()


@pytest.mark.parametrize("R,base,scaling", [
    (128, 10000.0, None), (64, 500000.0, None), (16, 1e6, ("linear", 4.0)), (128, 500000.0, ("bands", 8.0, 8192, 1.0, 4.0)),
    (256, 10000.0, ("yarn", 8.0, 8192, 32.0, 1.0)), (64, 10000.0, ("yarn", 0.5, 4096, 32.0, 1.0)),
    (32, 10000.0, ("yarn", 40.0, 16, 32.0, 1.0)), (0, 10000.0, None)])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_frequencies(lib, R, base, scaling, layout):
    r = rkv.make_rope(256, R, layout, base, scaling)
    th, gain = po.theta(R, base, scaling)
    assert (r.D, r.R, r.layout) == (256, R, 0 if layout == "pairs" else 1)
    assert r.gain == np.float32(gain)
    got = np.array([r.turn[i] / 2.0 ** 64 for i in range(R // 2)])
    # a power, a quotient by 2 pi and up to five more roundings of 2^-53 each
    want = (th / (2 * math.pi)) % 1.0
    assert np.all(np.abs(got - want) <= 2.0 ** -49 * want + 2.0 ** -60)
    assert all(r.turn[i] == 0 for i in range(R // 2, 128))


def test_rope_refuses(lib):
    r, sc = rkv.rkv_rope(), rkv.rkv_rope_scaling

    def init(D=128, R=128, layout=0, base=10000.0, s=None, r=r):
        return lib.rkv_rope_init(None if r is None else B(r), D, R, layout, base, None if s is None else B(s))

    assert init() == 0
    nan = float("nan")
    for kw, code in ((dict(r=None), INVALID), (dict(R=130), INVALID), (dict(R=24), INVALID), (dict(R=-16), INVALID),
                     (dict(R=144), INVALID), (dict(layout=2), INVALID), (dict(base=1.0), INVALID), (dict(base=nan), INVALID),
                     (dict(base=math.inf), INVALID), (dict(D=512), UNSUPPORTED), (dict(s=sc(4, 0, 2, 8192, 1, 4)), INVALID),
                     (dict(s=sc(1, 0, 5e-324, 0, 0, 0)), INVALID),
                     (dict(s=sc(1, 1, 2, 0, 0, 0)), INVALID), (dict(s=sc(1, 0, 0, 0, 0, 0)), INVALID),
                     (dict(s=sc(2, 0, 8, 0, 1, 4)), INVALID), (dict(s=sc(2, 0, 8, 8192, 4, 4)), INVALID),
                     (dict(s=sc(3, 0, nan, 8192, 32, 1)), INVALID), (dict(s=sc(3, 0, 8, 8192, 32, 0)), INVALID)):
        assert init(**kw) == code, kw


def test_rotate_refuses(lib):
    rope = rkv.make_rope(128)

    def rotate(p=(8, 2, 128, 0), rope=rope, rows=4, dt=1, q=16, qs=1024, k=16, ks=256, pos=16, qw=None, kw=None, eps=1e-6,
               qo=16, qos=1024, ko=16, kos=256, st=16):
        p = rkv.rkv_head_params(*p)
        return lib.rkv_qk_rotate(B(p), None if rope is None else B(rope), rows, dt, q, qs, k, ks, pos, qw, kw, eps, qo, qos,
                                 ko, kos, st, None)

    assert rotate(rows=0) == 0
    bent = rkv.make_rope(128)
    bent.R = 24
    loud = rkv.make_rope(128)
    loud.gain = math.inf
    for kw, code in ((dict(p=(0, 2, 128, 0)), INVALID), (dict(p=(8, 3, 128, 0)), UNSUPPORTED), (dict(p=(8, 2, 96, 0)), UNSUPPORTED),
                     (dict(p=(8, 2, 128, 1)), INVALID), (dict(rope=None), INVALID), (dict(rope=rkv.make_rope(64)), INVALID),
                     (dict(rope=bent), INVALID), (dict(rope=loud), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 28), UNSUPPORTED), (dict(dt=2), INVALID),
                     (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(q=None, qo=None, k=None, ko=None), INVALID),
                     (dict(qs=1023), INVALID), (dict(qs=1028), ALIGN), (dict(kos=260), ALIGN), (dict(pos=None), INVALID),
                     (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(st=None), INVALID),
                     (dict(qos=1032), INVALID), (dict(q=24), ALIGN), (dict(kw=20), ALIGN)):
        assert rotate(**kw) == code, kw


def test_prompt_attention_refuses(lib):
    def attend(p=(8, 2, 128, 0), S=2, start=16, rows=40, q=16, qs=1024, k=16, ks=256, v=16, vs=256, o=16, os=1024, ws=256,
               nb=1 << 40, st=16):
        p = rkv.rkv_head_params(*p)
        return lib.rkv_prompt_attention(B(p), S, start, rows, q, qs, k, ks, v, vs, o, os, ws, nb, st, None)

    assert attend(S=0) == 0 and attend(rows=0) == 0
    for kw, code in ((dict(p=(9, 1, 128, 0)), UNSUPPORTED), (dict(p=(8, 2, 32, 0)), UNSUPPORTED), (dict(p=(8, 0, 128, 0)), INVALID),
                     (dict(S=-1), INVALID), (dict(rows=-1), INVALID), (dict(S=1 << 30), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(start=None), INVALID),
                     (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(st=None), INVALID),
                     (dict(qs=1000), INVALID), (dict(ks=260), ALIGN), (dict(os=1028), ALIGN), (dict(k=24), ALIGN),
                     (dict(S=40, nb=64), WORKSPACE), (dict(S=40, ws=None), WORKSPACE), (dict(S=40, ws=128), ALIGN),
                     (dict(ws=128), ALIGN)):
        assert attend(**kw) == code, kw
    p = rkv.rkv_head_params(8, 2, 128, 0)
    assert rkv.rkv_prompt_attention_workspace(p, 0, 40) == 0 and rkv.rkv_prompt_attention_workspace(p, 40, 0) == 0
    assert rkv.rkv_prompt_attention_workspace(p, 2, 40) == 0 and rkv.rkv_prompt_attention_workspace(p, 40, 40) > 64
    with pytest.raises(rkv.RkvError):
        rkv.rkv_prompt_attention_workspace(p, -1, 40)


def test_the_workspace_does_not_grow_with_the_rows_squared(lib):
    # items of 32 bytes for each tile of 256 rows, and at most 608 partials of 256 rows
    p = rkv.rkv_head_params(32, 8, 128, 0)
    for rows in (1, 500, 8192, 131072, 1 << 20):
        need = rkv.rkv_prompt_attention_workspace(p, 3, rows)
        assert need <= 608 * 256 * (128 * 4 + 8) + 64 * (rows // 64 + 3 + 76) + 4096


def test_chunk_attention_refuses(lib):
    ok = rkv.rkv_dense_cache(16, 16, 16)

    def chunk(p=(2, 1000, 4, 128, 4, 0), H=8, q=16, n=100, nn=16, kv=16, c=ok, ln=16, o=16, ws=256, nb=1 << 40, st=16):
        return lib.rkv_chunk_attention(B(rkv.rkv_dense_params(*p)), H, q, n, nn, kv, B(c), ln, o, ws, nb, st, None)

    for n in (1, 64, 65, 1000):
        for kw, code in ((dict(p=(0, 1000, 4, 128, 4, 0)), INVALID), (dict(p=(2, 1000, 4, 96, 4, 0)), UNSUPPORTED),
                         (dict(H=0), INVALID), (dict(H=6), UNSUPPORTED), (dict(H=36), UNSUPPORTED), (dict(q=None), INVALID),
                         (dict(kv=None), INVALID), (dict(ln=None), INVALID), (dict(o=None), INVALID), (dict(st=None), INVALID),
                         (dict(q=24), ALIGN), (dict(nn=4), ALIGN), (dict(nb=100), WORKSPACE), (dict(ws=None), WORKSPACE),
                         (dict(ws=16), ALIGN), (dict(c=rkv.rkv_dense_cache(None, 16, 16)), INVALID),
                         (dict(c=rkv.rkv_dense_cache(16, 16, 8)), ALIGN)):
            assert chunk(n=n, **kw) == code, kw
    for n in (0, -1, 1001):
        assert chunk(n=n) == INVALID
        with pytest.raises(rkv.RkvError):
            rkv.rkv_chunk_attention_workspace(rkv.make_dense_params(2, 1000, 4, 128), 8, n)
    p = rkv.make_dense_params(2, 1000, 4, 128)
    for n in (64, 65):
        need = rkv.rkv_chunk_attention_workspace(p, 8, n)
        assert chunk(n=n, nb=need - 1) == WORKSPACE and chunk(n=n, nb=need, ws=16) == ALIGN


def test_the_heads_object_checks_its_tensors(lib):
    h = rkv.PromptHeads(8, 2, 128, device="cpu")
    rope = rkv.make_rope(128)
    q, k = torch.zeros(6, 8, 128, dtype=torch.bfloat16), torch.zeros(6, 2, 128, dtype=torch.bfloat16)
    pos, w = torch.zeros(6, dtype=torch.int32), torch.ones(128, dtype=torch.bfloat16)
    start = torch.tensor([0, 6], dtype=torch.int32)
    bad = [
        lambda: h.rotate(rope, q.half(), k, pos, q, k), lambda: h.rotate(rope, q, k.float(), pos, q, k),
        lambda: h.rotate(rope, q[:, :4], k, pos, q, k), lambda: h.rotate(rope, q, k[:5], pos, q, k),
        lambda: h.rotate(rope, q, k, pos.long(), q, k), lambda: h.rotate(rope, q, k, pos[:5], q, k),
        lambda: h.rotate(rope, q, k, pos, q, None), lambda: h.rotate(rope, None, None, pos, None, None),
        lambda: h.rotate(rope, q, None, pos, q, None, k_weight=w), lambda: h.rotate(rope, q, k, pos, q, k, w.float()),
        lambda: h.rotate(rope, q, k, pos, q, k, w[:64]), lambda: h.rotate(rkv.make_rope(64), q, k, pos, q, k),
        lambda: h.rotate(rope, q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, q, k),
        lambda: h.rotate(rope, q[:1].expand(6, 8, 128), k, pos, q, k), lambda: h.rotate(rope, q.to("meta"), k, pos, q, k),
        lambda: h.attend(q.float(), k, k, start, q), lambda: h.attend(q, k, k[:5], start, q),
        lambda: h.attend(q, k, k, start.long(), q), lambda: h.attend(q, k, k, start[None], q),
        lambda: h.attend(q, k, k, start, q.float()), lambda: h.attend(q, k, k, start[:0], q),
        lambda: h.attend(q[0], k, k, start, q),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: h.rotate(rope, q, k, pos, q, k), lambda: h.attend(q, k, k, start, q)):
        with pytest.raises(ValueError, match="not on a GPU"):
            f()
    for H, N, D in ((8, 3, 128), (8, 2, 100), (0, 1, 128), (8, 0, 128)):
        with pytest.raises(rkv.RkvError):
            rkv.PromptHeads(H, N, D, device="cpu")


def test_pieces_are_checked(lib):
    c = rkv.DenseCache(rkv.make_dense_params(2, 100, 4, 128), device="cpu")
    q, kv = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 3, 1024, dtype=torch.bfloat16)
    ln = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: c.chunk_attend(8, q.float(), kv, ln, q), lambda: c.chunk_attend(8, q, kv[:, :2], ln, q),
              lambda: c.chunk_attend(8, q, kv, ln.long(), q), lambda: c.chunk_attend(8, q, kv, ln, q.float()),
              lambda: c.chunk_attend(8, q, kv, ln, q, n_new=ln[:1]), lambda: c.chunk_attend(4, q, kv, ln, q),
              lambda: c.chunk_attend(8, q.transpose(0, 1), kv, ln, q)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError, match="not on a GPU"):
        c.chunk_attend(8, q, kv, ln, torch.zeros_like(q))


def test_the_restatement_of_rotation():
    # closed forms: position 0 keeps everything, a quarter turn of the first pair, the norm of a constant head
    x = np.arange(1.0, 33.0).reshape(1, 1, 32)
    th, _ = po.theta(16, 10000.0)
    assert np.array_equal(po.rotate(x, [0], th, 1.0, "pairs")[0], x)
    one = np.zeros(8)
    one[0] = math.pi / 2
    y, _ = po.rotate(x, [1], one, 2.0, "pairs")
    assert np.allclose(y[0, 0, :4], [-4.0, 2.0, 6.0, 8.0]) and np.array_equal(y[0, 0, 16:], x[0, 0, 16:])
    y, _ = po.rotate(x, [1], one, 1.0, "halves")
    assert np.allclose(y[0, 0, [0, 8]], [-9.0, 1.0]) and y[0, 0, 1] == 2.0
    assert np.allclose(po.rotate(np.full((1, 1, 32), 3.0), [5], th[:0], 1.0, "pairs", weight=np.full(32, 0.5), eps=0.0)[0], 0.5)


def test_the_restatement_of_attention():
    import oracle
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(9, 4, 64)), rng.normal(size=(14, 2, 64)), rng.normal(size=(14, 2, 64))
    out, _ = po.causal(torch.tensor(q), torch.tensor(k), torch.tensor(v), before=5)
    for i in range(9):
        want = oracle.attention(q[i], k[: 6 + i].reshape(-1, 128), v[: 6 + i].reshape(-1, 128), 2)
        assert np.allclose(out[i].numpy(), want, rtol=1e-12, atol=1e-13)
