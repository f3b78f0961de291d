"""Python binding of librkv: the same entry points as include/rkv.h, argument
marshalling only.  Every step of the path runs in the library's CUDA kernels; torch
only allocates device memory and supplies streams.  There is no fallback: if
librkv.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "librkv.so")
_lib = None

RKV_F32, RKV_BF16, RKV_FP8_E4M3 = 0, 1, 2
RKV_OK, RKV_ERR_INVALID_ARG, RKV_ERR_UNSUPPORTED, RKV_ERR_ALIGNMENT = 0, 1, 2, 3
RKV_ERR_CUDA, RKV_ERR_INDEX, RKV_ERR_DEVICE_TIMEOUT, RKV_ERR_WORKSPACE = 4, 5, 6, 7
EXPORTED = ("rkv_n_ref", "rkv_query_sizes", "rkv_build_ref_pool", "rkv_compress",
            "rkv_gather_dequant", "rkv_restore_kv", "rkv_attention_workspace", "rkv_sparse_attention",
            "rkv_append_token", "rkv_compress_noalloc", "rkv_profile_enable", "rkv_profile_collect",
            "rkv_debug_wait_fault", "rkv_status_string",
            "rkv_dense_sizes", "rkv_dense_write", "rkv_dense_read", "rkv_block_select_workspace",
            "rkv_block_select", "rkv_dense_attention_workspace", "rkv_dense_attention",
            "rkv_tree_attention")
_DTYPES = {"f32": RKV_F32, "bf16": RKV_BF16, "fp8": RKV_FP8_E4M3}


class rkv_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "L", "B", "T", "N", "D", "d_ff", "d_c", "k", "group", "bits", "kv_dtype", "ref_dtype",
        "stride", "first")] + [("alpha", ctypes.c_double), ("n_sink", ctypes.c_int32),
                               ("reserved", ctypes.c_int32)]


class rkv_ref_pool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("ref_pos", "ref_slot", "pool_size", "ref_vec",
                                               "ref_sqnorm")]


class rkv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "hdr", "ref_idx")]


class rkv_dense_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("S", "T", "N", "D", "bits", "reserved")]


class rkv_dense_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "khdr", "tail")]


class RkvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (status %d)" % (where, rkv_status_string(code), code))


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load librkv.so (raises if it is absent: there is no other implementation)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("librkv.so is not built (%s); run "
                               "reference_residual_kv_gb300.build.build()" % _LIB_PATH)
        L = ctypes.CDLL(_LIB_PATH)
        P, V, I32 = ctypes.POINTER(rkv_params), ctypes.c_void_p, ctypes.c_int32
        sz = ctypes.POINTER(ctypes.c_size_t)
        L.rkv_n_ref.argtypes = [P]
        L.rkv_n_ref.restype = I32
        L.rkv_query_sizes.argtypes = [P, sz, sz, sz]
        L.rkv_query_sizes.restype = I32
        L.rkv_build_ref_pool.argtypes = [P, V, ctypes.POINTER(rkv_ref_pool), V]
        L.rkv_build_ref_pool.restype = I32
        L.rkv_compress.argtypes = [P, V, ctypes.POINTER(rkv_ref_pool), V, V, V,
                                   ctypes.POINTER(rkv_cache), V, ctypes.c_size_t, V, V, V]
        L.rkv_compress.restype = I32
        L.rkv_compress_noalloc.argtypes = [P, V, ctypes.POINTER(rkv_ref_pool), V, V, V,
                                           ctypes.POINTER(rkv_cache), V, V, V]
        L.rkv_compress_noalloc.restype = I32
        L.rkv_gather_dequant.argtypes = [P, ctypes.POINTER(rkv_ref_pool), ctypes.POINTER(rkv_cache),
                                         V, I32, V, V, I32, V, V]
        L.rkv_gather_dequant.restype = I32
        L.rkv_restore_kv.argtypes = [P, ctypes.POINTER(rkv_ref_pool), ctypes.POINTER(rkv_cache),
                                     V, V, I32, ctypes.c_double, V, V, V, V]
        L.rkv_restore_kv.restype = I32
        L.rkv_append_token.argtypes = [P, V, I32, ctypes.POINTER(rkv_ref_pool), V, V, V,
                                       ctypes.POINTER(rkv_cache), V, ctypes.c_size_t, V, V]
        L.rkv_append_token.restype = I32
        L.rkv_attention_workspace.argtypes = [P, I32, I32, sz]
        L.rkv_attention_workspace.restype = I32
        L.rkv_sparse_attention.argtypes = [P, I32, V, V, V, V, I32, V, V, ctypes.c_size_t, V]
        L.rkv_sparse_attention.restype = I32
        DP, DC, Z = ctypes.POINTER(rkv_dense_params), ctypes.POINTER(rkv_dense_cache), ctypes.c_size_t
        for name, args in (
                ("rkv_dense_sizes", [DP, sz, sz, sz]),
                ("rkv_dense_write", [DP, V, I32, I32, V, V, DC, V, V]),
                ("rkv_dense_read", [DP, DC, V, V, I32, V, V, V, V]),
                ("rkv_block_select_workspace", [DP, I32, sz]),
                ("rkv_block_select", [DP, I32, V, DC, V, I32, I32, I32, I32, V, V, Z, V, V]),
                ("rkv_dense_attention_workspace", [DP, I32, I32, sz]),
                ("rkv_dense_attention", [DP, I32, V, DC, V, V, I32, I32, V, I32, V, Z, V, V]),
                ("rkv_tree_attention", [DP, I32, V, I32, V, V, DC, V, V, I32, V, Z, V, V])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, I32
        L.rkv_profile_enable.argtypes = [I32]
        L.rkv_profile_enable.restype = I32
        L.rkv_profile_collect.argtypes = [ctypes.c_char_p, I32, ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(I32), I32]
        L.rkv_profile_collect.restype = I32
        L.rkv_debug_wait_fault.argtypes = [ctypes.c_int64, I32]
        L.rkv_debug_wait_fault.restype = I32
        L.rkv_status_string.argtypes = [I32]
        L.rkv_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_params(L, B, T, N, D, d_ff, d_c, k=4, group=32, bits=4, kv_dtype="bf16",
                ref_dtype=None, stride=8, first=0, alpha=0.0, n_sink=0) -> rkv_params:
    kd = _DTYPES[kv_dtype] if isinstance(kv_dtype, str) else kv_dtype
    rd = kd if ref_dtype is None else (_DTYPES[ref_dtype] if isinstance(ref_dtype, str) else ref_dtype)
    return rkv_params(L, B, T, N, D, d_ff, d_c, k, group, bits, kd, rd, stride, first, float(alpha),
                      n_sink, 0)


def params_from_config(cfg) -> rkv_params:
    """rkv_params from a workload description with the same field names."""
    return make_params(cfg.L, cfg.B, cfg.T, cfg.N, cfg.D, cfg.d_ff, cfg.d_c, cfg.k, cfg.group,
                       cfg.bits, cfg.kv_dtype, cfg.ref_dtype, cfg.stride, cfg.first,
                       getattr(cfg, "alpha", 0.0), getattr(cfg, "n_sink", 0))


# ---- entry points (same names as the C ABI) -------------------------------------------
def rkv_status_string(code: int) -> str:
    return lib().rkv_status_string(int(code)).decode()


def rkv_n_ref(p: rkv_params) -> int:
    return lib().rkv_n_ref(ctypes.byref(p))


def rkv_query_sizes(p: rkv_params):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    st = lib().rkv_query_sizes(ctypes.byref(p), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    if st:
        raise RkvError(st, "rkv_query_sizes")
    return a.value, b.value, c.value


def rkv_build_ref_pool(p: rkv_params, kv, pool: rkv_ref_pool, stream=None) -> None:
    st = lib().rkv_build_ref_pool(ctypes.byref(p), _ptr(kv), ctypes.byref(pool), _stream(stream))
    if st:
        raise RkvError(st, "rkv_build_ref_pool")


def rkv_compress(p: rkv_params, kv, pool: rkv_ref_pool, W1t, W2t, W3t, cache: rkv_cache,
                 workspace, workspace_bytes: int, z_out, dev_status, stream=None) -> None:
    st = lib().rkv_compress(ctypes.byref(p), _ptr(kv), ctypes.byref(pool), _ptr(W1t), _ptr(W2t),
                            _ptr(W3t), ctypes.byref(cache), _ptr(workspace), int(workspace_bytes),
                            _ptr(z_out), _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_compress")


def rkv_compress_noalloc(p: rkv_params, kv, pool: rkv_ref_pool, W1t, W2t, W3t, cache: rkv_cache,
                         z_out, dev_status, stream=None) -> None:
    """rkv_compress with the library's built-in 64 MiB scratch instead of a workspace
    (for callers that cannot allocate device memory at the call)."""
    st = lib().rkv_compress_noalloc(ctypes.byref(p), _ptr(kv), ctypes.byref(pool), _ptr(W1t),
                                    _ptr(W2t), _ptr(W3t), ctypes.byref(cache), _ptr(z_out),
                                    _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_compress_noalloc")


def rkv_gather_dequant(p: rkv_params, pool: rkv_ref_pool, cache: rkv_cache, sel, n_sel: int,
                       out_z, out_mean, out_dtype: int, dev_status, stream=None) -> None:
    st = lib().rkv_gather_dequant(ctypes.byref(p), ctypes.byref(pool), ctypes.byref(cache),
                                  _ptr(sel), int(n_sel), _ptr(out_z), _ptr(out_mean),
                                  int(out_dtype), _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_gather_dequant")


def rkv_restore_kv(p: rkv_params, pool: rkv_ref_pool, cache: rkv_cache, Wd, sel, n_sel: int,
                   rope_base: float, out_k, out_v, dev_status, stream=None) -> None:
    st = lib().rkv_restore_kv(ctypes.byref(p), ctypes.byref(pool), ctypes.byref(cache), _ptr(Wd),
                              _ptr(sel), int(n_sel), float(rope_base), _ptr(out_k), _ptr(out_v),
                              _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_restore_kv")


def rkv_append_token(p: rkv_params, kv_new, t: int, pool: rkv_ref_pool, W1t, W2t, W3t,
                     cache: rkv_cache, workspace, workspace_bytes: int, dev_status, stream=None) -> None:
    st = lib().rkv_append_token(ctypes.byref(p), _ptr(kv_new), int(t), ctypes.byref(pool), _ptr(W1t),
                                _ptr(W2t), _ptr(W3t), ctypes.byref(cache), _ptr(workspace),
                                int(workspace_bytes), _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_append_token")


def rkv_attention_workspace(p: rkv_params, H: int, n_sel: int) -> int:
    b = ctypes.c_size_t()
    st = lib().rkv_attention_workspace(ctypes.byref(p), int(H), int(n_sel), ctypes.byref(b))
    if st:
        raise RkvError(st, "rkv_attention_workspace")
    return b.value


def rkv_sparse_attention(p: rkv_params, H: int, q, k_hat, v_hat, sel, n_sel: int, out, workspace,
                         workspace_bytes: int, stream=None) -> None:
    st = lib().rkv_sparse_attention(ctypes.byref(p), int(H), _ptr(q), _ptr(k_hat), _ptr(v_hat),
                                    _ptr(sel), int(n_sel), _ptr(out), _ptr(workspace),
                                    int(workspace_bytes), _stream(stream))
    if st:
        raise RkvError(st, "rkv_sparse_attention")


def make_dense_params(S, T, N, D, bits=4) -> rkv_dense_params:
    return rkv_dense_params(S, T, N, D, bits, 0)


def rkv_dense_sizes(p: rkv_dense_params):
    """(codes, khdr, tail) bytes."""
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    st = lib().rkv_dense_sizes(ctypes.byref(p), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    if st:
        raise RkvError(st, "rkv_dense_sizes")
    return a.value, b.value, c.value


def rkv_dense_write(p: rkv_dense_params, kv, kv_dtype: int, n: int, pos, n_new, cache: rkv_dense_cache,
                    dev_status, stream=None) -> None:
    st = lib().rkv_dense_write(ctypes.byref(p), _ptr(kv), kv_dtype, n, _ptr(pos), _ptr(n_new),
                               ctypes.byref(cache), _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_dense_write")


def rkv_dense_read(p: rkv_dense_params, cache: rkv_dense_cache, length, sel, n_sel: int, out_k, out_v,
                   dev_status, stream=None) -> None:
    st = lib().rkv_dense_read(ctypes.byref(p), ctypes.byref(cache), _ptr(length), _ptr(sel), n_sel,
                              _ptr(out_k), _ptr(out_v), _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_dense_read")


def rkv_block_select_workspace(p: rkv_dense_params, lists: int) -> int:
    b = ctypes.c_size_t()
    st = lib().rkv_block_select_workspace(ctypes.byref(p), lists, ctypes.byref(b))
    if st:
        raise RkvError(st, "rkv_block_select_workspace")
    return b.value


def rkv_block_select(p: rkv_dense_params, H: int, q, cache: rkv_dense_cache, length, lists: int,
                     n_blocks: int, keep_first: int, keep_last: int, blocks, workspace,
                     workspace_bytes: int, dev_status, stream=None) -> None:
    st = lib().rkv_block_select(ctypes.byref(p), H, _ptr(q), ctypes.byref(cache), _ptr(length), lists,
                                n_blocks, keep_first, keep_last, _ptr(blocks), _ptr(workspace),
                                workspace_bytes, _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_block_select")


def rkv_dense_attention_workspace(p: rkv_dense_params, H: int, n_query: int = 1) -> int:
    b = ctypes.c_size_t()
    st = lib().rkv_dense_attention_workspace(ctypes.byref(p), H, n_query, ctypes.byref(b))
    if st:
        raise RkvError(st, "rkv_dense_attention_workspace")
    return b.value


def rkv_dense_attention(p: rkv_dense_params, H: int, q, cache: rkv_dense_cache, length, blocks, lists: int,
                        n_blocks: int, out, out_dtype: int, workspace, workspace_bytes: int, dev_status,
                        stream=None) -> None:
    st = lib().rkv_dense_attention(ctypes.byref(p), H, _ptr(q), ctypes.byref(cache), _ptr(length),
                                   _ptr(blocks), lists, n_blocks, _ptr(out), out_dtype, _ptr(workspace),
                                   workspace_bytes, _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_dense_attention")


def rkv_tree_attention(p: rkv_dense_params, H: int, q, n_draft: int, parent, draft_kv,
                       cache: rkv_dense_cache, length, out, out_dtype: int, workspace, workspace_bytes: int,
                       dev_status, stream=None) -> None:
    st = lib().rkv_tree_attention(ctypes.byref(p), H, _ptr(q), n_draft, _ptr(parent), _ptr(draft_kv),
                                  ctypes.byref(cache), _ptr(length), _ptr(out), out_dtype, _ptr(workspace),
                                  workspace_bytes, _ptr(dev_status), _stream(stream))
    if st:
        raise RkvError(st, "rkv_tree_attention")


def rkv_debug_wait_fault(wait_cycles: int, skip_use: int) -> None:
    st = lib().rkv_debug_wait_fault(int(wait_cycles), int(skip_use))
    if st:
        raise RkvError(st, "rkv_debug_wait_fault")


def rkv_profile_enable(on: bool) -> None:
    lib().rkv_profile_enable(1 if on else 0)


def rkv_profile_collect(max_entries: int = 64, name_len: int = 48):
    """{kernel name: (total ms, launches)} since the last rkv_profile_enable(True)."""
    names = ctypes.create_string_buffer(max_entries * name_len)
    ms = (ctypes.c_float * max_entries)()
    cnt = (ctypes.c_int32 * max_entries)()
    n = lib().rkv_profile_collect(names, name_len, ms, cnt, max_entries)
    if n < 0:
        raise RkvError(RKV_ERR_CUDA, "rkv_profile_collect")
    raw = names.raw
    out = {}
    for i in range(n):
        nm = raw[i * name_len:(i + 1) * name_len].split(b"\0", 1)[0].decode()
        out[nm] = (float(ms[i]), int(cnt[i]))
    return out


# ---- device buffers ----------------------------------------------------------------
_TORCH_REF = {RKV_F32: torch.float32, RKV_BF16: torch.bfloat16, RKV_FP8_E4M3: torch.uint8}


GUARD_BYTE = 0xA5


def guarded_empty(shape, dtype, device, guard: int, fill=None):
    """(tensor, raw): an uninitialised tensor of `shape` that is the head of a byte
    allocation followed by `guard` bytes of GUARD_BYTE (guard = 0: a plain allocation,
    raw is None).  A write past the tensor's end changes the tail (see guard_intact)."""
    if guard <= 0:
        t = torch.empty(shape, dtype=dtype, device=device)
        if fill is not None:
            t.fill_(fill)
        return t, None
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    raw = torch.empty(n + guard, dtype=torch.uint8, device=device)
    raw[n:].fill_(GUARD_BYTE)
    t = raw[:n].view(dtype).view(shape)
    if fill is not None:
        t.fill_(fill)
    return t, raw


def guard_intact(t, raw) -> bool:
    if raw is None:
        return True
    n = t.numel() * t.element_size()
    return bool((raw[n:] == GUARD_BYTE).all().item())


class Buffers:
    """Caller-owned device buffers for one rkv_params: pool, cache, workspace, status.
    guard > 0 puts that many guard bytes after every buffer (test support: the tails are
    checked by guard_violations())."""

    def __init__(self, p: rkv_params, device="cuda", want_z: bool = False, guard: int = 0):
        self.p = p
        LB, T, W = p.L * p.B, p.T, 2 * p.N * p.D
        R = rkv_n_ref(p)
        if R < 0:
            raise RkvError(RKV_ERR_INVALID_ARG, "Buffers")
        self.n_ref = R
        _, _, ws = rkv_query_sizes(p)
        self.guard = guard
        self._raw = {}

        def alloc(name, shape, dtype, fill=None):
            t, raw = guarded_empty(shape, dtype, device, guard, fill)
            self._raw[name] = raw
            return t

        i32 = torch.int32
        self.ref_pos = alloc("ref_pos", (max(R, 1),), i32)
        self.ref_slot = alloc("ref_slot", (T,), i32)
        self.pool_size = alloc("pool_size", (T,), i32)
        self.ref_vec = alloc("ref_vec", (LB, max(R, 1), W), _TORCH_REF[p.ref_dtype])
        self.ref_sqnorm = alloc("ref_sqnorm", (LB, max(R, 1)), torch.float32)
        self.codes = alloc("codes", (LB, T, p.d_c * p.bits // 8), torch.uint8)
        self.hdr = alloc("hdr", (LB, T, p.d_c // 32, 2), torch.float32)
        self.ref_idx = alloc("ref_idx", (LB, T, 4), i32)
        self.workspace_bytes = ws
        self.workspace = alloc("workspace", (max(ws, 256),), torch.uint8)
        self.status = alloc("status", (4,), i32, fill=0)
        self.z = alloc("z", (LB, T, p.d_c), torch.float32) if want_z else None
        self.pool = rkv_ref_pool(_ptr(self.ref_pos), _ptr(self.ref_slot), _ptr(self.pool_size),
                                 _ptr(self.ref_vec), _ptr(self.ref_sqnorm))
        self.cache = rkv_cache(_ptr(self.codes), _ptr(self.hdr), _ptr(self.ref_idx))

    def build_ref_pool(self, kv, stream=None):
        rkv_build_ref_pool(self.p, kv, self.pool, stream)

    def compress(self, kv, W1t, W2t, W3t, stream=None):
        rkv_compress(self.p, kv, self.pool, W1t, W2t, W3t, self.cache, self.workspace,
                     self.workspace_bytes, self.z, self.status, stream)

    def gather(self, sel, out_z, out_mean, out_dtype=None, stream=None):
        n_sel = sel.shape[-1]
        if out_dtype is None:
            out_dtype = RKV_F32 if out_z.dtype == torch.float32 else RKV_BF16
        rkv_gather_dequant(self.p, self.pool, self.cache, sel, n_sel, out_z, out_mean, out_dtype,
                           self.status, stream)

    def restore(self, Wd, sel, out_k, out_v, rope_base: float, stream=None):
        rkv_restore_kv(self.p, self.pool, self.cache, Wd, sel, sel.shape[-1], rope_base, out_k,
                       out_v, self.status, stream)

    def append(self, kv_new, t: int, W1t, W2t, W3t, stream=None):
        rkv_append_token(self.p, kv_new, t, self.pool, W1t, W2t, W3t, self.cache, self.workspace,
                         self.workspace_bytes, self.status, stream)

    def attend(self, H: int, q, k_hat, v_hat, sel, out, stream=None):
        n_sel = sel.shape[-1]
        need = rkv_attention_workspace(self.p, H, n_sel)
        if getattr(self, "_attn_ws", None) is None or self._attn_ws.numel() < need:
            self._attn_ws, self._raw["attention_workspace"] = guarded_empty(
                (max(need, 256),), torch.uint8, self.status.device, self.guard)
        rkv_sparse_attention(self.p, H, q, k_hat, v_hat, sel, n_sel, out, self._attn_ws,
                             self._attn_ws.numel(), stream)

    def device_status(self) -> int:
        return int(self.status[0].item())

    def guard_violations(self):
        """Names of the buffers whose guard bytes changed (empty without guards)."""
        bad = []
        for name, raw in self._raw.items():
            t = self._attn_ws if name == "attention_workspace" else getattr(self, name)
            if raw is not None and t is not None and not guard_intact(t, raw):
                bad.append(name)
        return bad


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# the raw handle of a device's current stream, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class DenseCache:
    """The dense cache of one rkv_dense_params on one device: its three buffers, the device
    status, and its operators with their tensors checked (type, shape, contiguity, device).
    Scratch is taken from torch's allocator for each call, on the stream that the call runs on,
    so that calls on several streams, and captured graphs, share none of it.  Calls that write
    the cache and calls that read it are ordered by the caller, as for any tensor.
    guard > 0 puts that many guard bytes behind every buffer, scratch included (test support)."""

    def __init__(self, p: rkv_dense_params, device="cuda", guard: int = 0):
        p = rkv_dense_params.from_buffer_copy(p)           # the buffers' own: later changes to the caller's do not reach it
        codes, khdr, tail = rkv_dense_sizes(p)
        self.p = p
        self.S, self.T, self.N, self.D = p.S, p.T, p.N, p.D
        self.guard = guard
        self._raw = {}
        for name, n, fill in (("codes", codes, None), ("khdr", khdr, None), ("tail", tail, None), ("status", 16, 0)):
            t, raw = guarded_empty((n,), torch.uint8, device, guard, fill)
            setattr(self, name, t)
            self._raw[name] = (t, raw)
        self.status = self.status.view(torch.int32)
        self.device = self.status.device
        self.cache = rkv_dense_cache(_ptr(self.codes), _ptr(self.khdr), _ptr(self.tail))
        self._sizes = {}
        self._p_ref, self._cache_ref = ctypes.byref(self.p), ctypes.byref(self.cache)
        self._status_ptr = self.status.data_ptr()

    def _refuse(self, name, t, dtypes, shape):
        """Says what is wrong with an argument, if anything is."""
        if t.dtype not in dtypes:
            raise ValueError("%s: %s, expected %s" % (name, t.dtype, " or ".join(map(str, dtypes))))
        if tuple(t.shape) != shape:
            raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), shape))
        if not t.is_contiguous():
            raise ValueError("%s is not contiguous" % name)
        if t.device != self.device:
            raise ValueError("%s is on %s, the cache on %s" % (name, t.device, self.device))

    def _check(self, name, t, dtypes, shape):
        if not (t.dtype in dtypes and t.shape == shape and t.device == self.device and t.is_contiguous()):
            self._refuse(name, t, dtypes, shape)

    def _call(self, name, stream, need, *args):
        """The entry point `name` with (params, *args, [workspace, bytes,] status, stream): the
        cache's device current, scratch of `need` bytes (None: it takes none) from the pool of the
        stream that the call runs on."""
        dev = self.device.index
        if dev is None:
            raise ValueError("%s: the cache is on %s, not on a GPU" % (name, self.device))
        if stream is not None and not isinstance(stream, int) and stream.device != self.device:
            raise ValueError("%s: the stream is on %s, the cache on %s" % (name, stream.device, self.device))
        if stream is None and torch.cuda.current_device() == dev:
            st = self._enter(name, need, args, _raw_stream(dev))
        else:
            with torch.cuda.device(dev):
                if stream is None:
                    st = self._enter(name, need, args, _raw_stream(dev))
                else:
                    if isinstance(stream, int):
                        stream = torch.cuda.ExternalStream(stream, device=self.device)
                    with torch.cuda.stream(stream):
                        st = self._enter(name, need, args, stream.cuda_stream)
        if st:
            raise RkvError(st, name)

    def _enter(self, name, need, args, stream):
        f = getattr(lib(), name)
        if need is None:
            return f(self._p_ref, *args, self._status_ptr, stream)
        ws = self._scratch(need)
        return f(self._p_ref, *args, ws.data_ptr(), need, self._status_ptr, stream)

    def _scratch(self, need):
        if not self.guard:
            return torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)
        t, raw = guarded_empty((max(need, 1),), torch.uint8, self.device, self.guard)
        self._raw["scratch %d" % len(self._raw)] = (t, raw)
        return t

    def _size(self, *key):
        """Bytes of scratch: ("select", lists) or ("attend", H, n_query)."""
        need = self._sizes.get(key)
        if need is None:
            f = rkv_block_select_workspace if key[0] == "select" else rkv_dense_attention_workspace
            need = self._sizes[key] = f(self.p, *key[1:])
        return need

    def write(self, kv, pos, n_new=None, stream=None):
        """kv [S][n][2ND] (bf16 or fp32) as tokens pos[s] .. of each sequence; n_new[s] of its n
        rows (all of them where n_new is None)."""
        n = kv.shape[1] if kv.dim() == 3 else -1
        self._check("kv", kv, (_BF16, _F32), (self.S, n, 2 * self.N * self.D))
        self._check("pos", pos, (_I32,), (self.S,))
        if n_new is not None:
            self._check("n_new", n_new, (_I32,), (self.S,))
        dt = RKV_F32 if kv.dtype is _F32 else RKV_BF16
        self._call("rkv_dense_write", stream, None, kv.data_ptr(), dt, n, pos.data_ptr(),
                   None if n_new is None else n_new.data_ptr(), self._cache_ref)

    def read(self, length, sel, out_k, out_v, stream=None):
        """K and V of tokens sel [S][n_sel] (-1: zero rows) to out_k, out_v bf16 [S][n_sel][ND]."""
        n = sel.shape[1] if sel.dim() == 2 else -1
        rows = (self.S, n, self.N * self.D)
        self._check("length", length, (_I32,), (self.S,))
        self._check("sel", sel, (_I32,), (self.S, n))
        self._check("out_k", out_k, (_BF16,), rows)
        self._check("out_v", out_v, (_BF16,), rows)
        self._call("rkv_dense_read", stream, None, self._cache_ref, length.data_ptr(), sel.data_ptr(), n,
                   out_k.data_ptr(), out_v.data_ptr())

    def select(self, H: int, q, length, blocks, keep_first: int = 0, keep_last: int = 0, stream=None):
        """The blocks [S][N or 1][n_blocks] (output) with the largest score bounds for q [S][H][D]."""
        lists, n = blocks.shape[1:] if blocks.dim() == 3 else (-1, -1)
        self._check("q", q, (_BF16,), (self.S, H, self.D))
        self._check("length", length, (_I32,), (self.S,))
        self._check("blocks", blocks, (_I32,), (self.S, lists, n))
        self._call("rkv_block_select", stream, self._size("select", lists), H, q.data_ptr(), self._cache_ref,
                   length.data_ptr(), lists, n, keep_first, keep_last, blocks.data_ptr())

    def attend(self, H: int, q, length, out, blocks=None, stream=None):
        """out [S][H][D] (fp32 or bf16): attention of q [S][H][D] over the cache, or over the
        listed blocks [S][N or 1][n_blocks] and the unfinished one."""
        self._check("q", q, (_BF16,), (self.S, H, self.D))
        self._check("length", length, (_I32,), (self.S,))
        self._check("out", out, (_F32, _BF16), (self.S, H, self.D))
        lists, n, listed = 1, 0, None
        if blocks is not None:
            lists, n = blocks.shape[1:] if blocks.dim() == 3 else (-1, -1)
            self._check("blocks", blocks, (_I32,), (self.S, lists, n))
            if n < 1:
                raise ValueError("blocks: an empty list")
            listed = blocks.data_ptr()
        dt = RKV_F32 if out.dtype is _F32 else RKV_BF16
        self._call("rkv_dense_attention", stream, self._size("attend", H, 1), H, q.data_ptr(), self._cache_ref,
                   length.data_ptr(), listed, lists, n, out.data_ptr(), dt)

    def tree_attend(self, H: int, q, parent, draft_kv, length, out, stream=None):
        """out [S][n][H][D] (fp32 or bf16): attention of the drafted tokens' q [S][n][H][D] over
        the cache and their own line of parents; draft_kv bf16 [S][n][2ND], parent [S][n]."""
        n = q.shape[1] if q.dim() == 4 else -1
        self._check("q", q, (_BF16,), (self.S, n, H, self.D))
        self._check("parent", parent, (_I32,), (self.S, n))
        self._check("draft_kv", draft_kv, (_BF16,), (self.S, n, 2 * self.N * self.D))
        self._check("length", length, (_I32,), (self.S,))
        self._check("out", out, (_F32, _BF16), (self.S, n, H, self.D))
        dt = RKV_F32 if out.dtype is _F32 else RKV_BF16
        self._call("rkv_tree_attention", stream, self._size("attend", H, n), H, q.data_ptr(), n, parent.data_ptr(),
                   draft_kv.data_ptr(), self._cache_ref, length.data_ptr(), out.data_ptr(), dt)

    def device_status(self) -> int:
        return int(self.status[0].item())

    def guard_violations(self):
        """Names of the buffers whose guard bytes changed (empty without guards)."""
        return [k for k, (t, raw) in self._raw.items() if raw is not None and not guard_intact(t, raw)]
