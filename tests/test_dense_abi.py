"""Refusals and sizes of the dense cache's entry points: host checks, no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import _dense_oracle as do
from reference_residual_kv_gb300 import build, rkv, storage

INVALID, UNSUPPORTED = rkv.RKV_ERR_INVALID_ARG, rkv.RKV_ERR_UNSUPPORTED
ALIGN, WORKSPACE = rkv.RKV_ERR_ALIGNMENT, rkv.RKV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rkv.lib()


def params(S=2, T=1000, N=4, D=128, bits=4, reserved=0):
    return rkv.rkv_dense_params(S, T, N, D, bits, reserved)


def test_sizes(lib):
    # 5 bits a value at 4 bits a code: 8 D 4 / 8 ... per block and head D (8 bits + 4) + 4 D bytes
    codes, khdr, tail = rkv.rkv_dense_sizes(params())
    assert codes == 2 * 4 * 31 * 128 * 36 and khdr == 2 * 4 * 31 * 512 and tail == 2 * 4 * 2 * 32 * 128 * 2
    assert rkv.rkv_dense_sizes(params(T=31, bits=2))[:2] == (0, 0)
    assert codes + khdr == 2 * 4 * 31 * 32 * 2 * 128 * 5 // 8


def test_stored_bytes_are_the_paper_s_share(lib):
    # a layer-sequence of whole blocks: the accounting's bytes, and q_b of the fp16 cache's
    for D, bits in ((64, 2), (128, 4), (256, 2), (256, 4)):
        codes, khdr, _ = rkv.rkv_dense_sizes(params(S=1, T=640, N=3, D=D, bits=bits))
        per_token = storage.dense_layer_bytes_per_token(3, D, bits)
        assert (codes + khdr) / 640 == per_token == storage.q_b(bits) * 2 * 3 * D * 2


@pytest.mark.parametrize("field,value,code", [
    ("S", 0, INVALID), ("T", 0, INVALID), ("N", 0, INVALID), ("D", 0, INVALID), ("bits", 3, INVALID),
    ("bits", 8, INVALID), ("reserved", 1, INVALID), ("D", 96, UNSUPPORTED), ("D", 512, UNSUPPORTED),
    ("N", 1025, UNSUPPORTED), ("T", 2 ** 31 - 1, UNSUPPORTED)])
def test_wrong_params(lib, field, value, code):
    p = params()
    setattr(p, field, value)
    a = ctypes.c_size_t()
    assert lib.rkv_dense_sizes(ctypes.byref(p), ctypes.byref(a), None, None) == code
    c = rkv.rkv_dense_cache(16, 16, 16)
    B = ctypes.byref
    assert lib.rkv_dense_write(B(p), 16, 1, 1, 16, None, B(c), 16, None) == code
    assert lib.rkv_dense_read(B(p), B(c), 16, 16, 1, 16, 16, 16, None) == code
    assert lib.rkv_block_select(B(p), 8, 16, B(c), 16, 1, 4, 0, 0, 16, 256, 1 << 40, 16, None) == code
    assert lib.rkv_dense_attention(B(p), 8, 16, B(c), 16, None, 1, 0, 16, 0, 256, 1 << 40, 16, None) == code
    assert lib.rkv_tree_attention(B(p), 8, 16, 4, 16, 16, B(c), 16, 16, 0, 256, 1 << 40, 16, None) == code


def test_write_and_read_refuse(lib):
    p, B = params(), ctypes.byref
    ok = rkv.rkv_dense_cache(16, 16, 16)

    def write(kv=16, dt=1, n=4, pos=16, nn=16, c=ok, st=16):
        return lib.rkv_dense_write(B(p), kv, dt, n, pos, nn, B(c), st, None)

    assert write(n=0) == rkv.RKV_OK
    for kw, code in ((dict(kv=None), INVALID), (dict(dt=2), INVALID), (dict(n=-1), INVALID), (dict(n=1001), INVALID),
                     (dict(pos=None), INVALID), (dict(st=None), INVALID), (dict(kv=24), ALIGN), (dict(nn=20), ALIGN),
                     (dict(c=rkv.rkv_dense_cache(None, 16, 16)), INVALID),
                     (dict(c=rkv.rkv_dense_cache(16, 16, None)), INVALID),
                     (dict(c=rkv.rkv_dense_cache(16, 8, 16)), ALIGN)):
        assert write(**kw) == code, kw

    def read(ln=16, sel=16, n=4, k=16, v=16, st=16):
        return lib.rkv_dense_read(B(p), B(ok), ln, sel, n, k, v, st, None)

    assert read(n=0) == rkv.RKV_OK
    for kw, code in ((dict(n=-1), INVALID), (dict(ln=None), INVALID), (dict(sel=None), INVALID), (dict(k=None), INVALID),
                     (dict(v=8), ALIGN), (dict(st=None), INVALID), (dict(n=2 ** 29), UNSUPPORTED)):
        assert read(**kw) == code, kw


def test_selection_and_attention_refuse(lib):
    p, B = params(), ctypes.byref
    ok = rkv.rkv_dense_cache(16, 16, 16)

    def select(H=8, q=16, ln=16, lists=4, n=6, first=1, last=1, out=16, ws=256, nb=1 << 40, st=16, p=p):
        return lib.rkv_block_select(B(p), H, q, B(ok), ln, lists, n, first, last, out, ws, nb, st, None)

    for kw, code in ((dict(H=0), INVALID), (dict(H=6), UNSUPPORTED), (dict(H=36), UNSUPPORTED), (dict(lists=2), INVALID),
                     (dict(n=0), INVALID), (dict(first=-1), INVALID), (dict(first=4, last=3), INVALID),
                     (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID), (dict(q=None), INVALID),
                     (dict(out=8), ALIGN), (dict(nb=10), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=128), ALIGN),
                     (dict(p=params(T=1 << 23)), UNSUPPORTED)):
        assert select(**kw) == code, kw
    with pytest.raises(rkv.RkvError):
        rkv.rkv_block_select_workspace(p, 3)

    def attend(H=8, q=16, ln=16, blocks=16, lists=4, n=6, out=16, dt=0, ws=256, nb=1 << 40, st=16):
        return lib.rkv_dense_attention(B(p), H, q, B(ok), ln, blocks, lists, n, out, dt, ws, nb, st, None)

    for kw, code in ((dict(H=-4), INVALID), (dict(H=40), UNSUPPORTED), (dict(lists=3), INVALID), (dict(n=0), INVALID),
                     (dict(dt=2), INVALID), (dict(ln=None), INVALID), (dict(out=None), INVALID), (dict(blocks=4), ALIGN),
                     (dict(nb=100), WORKSPACE), (dict(ws=16), ALIGN), (dict(st=None), INVALID)):
        assert attend(**kw) == code, kw

    def tree(H=8, q=16, n=4, par=16, kv=16, ln=16, out=16, dt=1, ws=256, nb=1 << 40, st=16):
        return lib.rkv_tree_attention(B(p), H, q, n, par, kv, B(ok), ln, out, dt, ws, nb, st, None)

    for kw, code in ((dict(n=0), INVALID), (dict(n=65), INVALID), (dict(par=None), INVALID), (dict(kv=None), INVALID),
                     (dict(kv=8), ALIGN), (dict(H=9), UNSUPPORTED), (dict(dt=7), INVALID), (dict(nb=0), WORKSPACE)):
        assert tree(**kw) == code, kw
    for nq in (0, 65):
        with pytest.raises(rkv.RkvError):
            rkv.rkv_dense_attention_workspace(p, 8, nq)


def test_the_cache_object_checks_its_tensors(lib):
    c = rkv.DenseCache(rkv.make_dense_params(2, 100, 4, 128), device="cpu")
    pos = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros(2, 3, 1024, dtype=torch.bfloat16)
    q, out = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 128)
    bad = [
        lambda: c.write(kv.half(), pos), lambda: c.write(kv[:, :, :1000], pos), lambda: c.write(kv[:, ::2], pos),
        lambda: c.write(kv[0], pos), lambda: c.write(kv, pos.long()), lambda: c.write(kv, pos[:1]),
        lambda: c.write(kv, pos, pos[:1]), lambda: c.write(kv.to("meta"), pos),
        lambda: c.read(pos, pos, kv, kv), lambda: c.read(pos, torch.zeros(2, 3, dtype=torch.int32), kv[..., :512], kv),
        lambda: c.select(8, q, pos, torch.zeros(2, 4, dtype=torch.int32)),
        lambda: c.attend(8, q, pos, out.double()), lambda: c.attend(4, q, pos, out),
        lambda: c.attend(8, q, pos, out, blocks=torch.zeros(2, 1, 0, dtype=torch.int32)),
        lambda: c.attend(8, q.transpose(0, 1), pos, out),
        lambda: c.tree_attend(8, q, pos, kv, pos, out),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_a_cache_off_the_gpu_is_refused(lib):
    c = rkv.DenseCache(rkv.make_dense_params(2, 100, 4, 128), device="cpu")
    pos = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros(2, 3, 1024, dtype=torch.bfloat16)
    q, out = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 128)
    rows, blocks = torch.zeros(2, 3, 512, dtype=torch.bfloat16), torch.zeros(2, 4, 2, dtype=torch.int32)
    qt, parent = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32)
    for f in (lambda s: c.write(kv, pos, stream=s), lambda s: c.read(pos, parent, rows, rows, stream=s),
              lambda s: c.select(8, q, pos, blocks, stream=s), lambda s: c.attend(8, q, pos, out, stream=s),
              lambda s: c.tree_attend(8, qt, parent, kv, pos, torch.zeros(2, 3, 8, 128), stream=s)):
        for stream in (None, 1):
            with pytest.raises(ValueError, match="not on a GPU"):
                f(stream)


def test_oracle_rounding_and_codes():
    # bf16 rounding with one rounding: ties to even, and a border that fp32 alone would hit
    assert list(do.bf16([1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, 1.0 + 2.0 ** -8 + 2.0 ** -40, -(1.0 + 2.0 ** -8 - 2.0 ** -40)]) ) \
        == [1.0, 1.0 + 2.0 ** -6, 1.0 + 2.0 ** -7, -1.0]
    assert do.bf16(2.0 ** -133) == 2.0 ** -133 and do.bf16(2.0 ** -134) == 0.0 and do.bf16(1.5 * 2.0 ** -134) == 2.0 ** -133
    code, lo, step = do.quantise(np.array([0.0, 1.0, 3.0, 5.0, 30.0]), 0, 4)
    assert step[0] == 2.0 and list(code) == [0, 0, 2, 2, 15] and lo[0] == 0.0
    code, lo, step = do.quantise(np.array([2.5, 2.5]), 0, 2)
    assert not code.any() and step[0] == 0.0 and lo[0] == 2.5
    code, lo, step = do.quantise(np.array([1.0, np.inf]), 0, 2)
    assert np.isnan(lo[0]) and np.isnan(step[0])
