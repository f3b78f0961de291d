"""fp64 restatement of the dense cache on the host (numpy), for its tests.  Written from
the definition in include/rkv.h; shares no code with the library."""
import math

import numpy as np

BLK = 32


def bf16_bits(x, rest=0.0):
    """Nearest bf16 (ties to even) of x + rest with one rounding, as uint16 bits; x in float64,
    |rest| below x's last bit (what x lost to its own rounding).  The float32 neighbour of x
    towards zero and what was cut from it decide (magnitudes < 2^127)."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        f = x.astype(np.float32)
        over = np.abs(f.astype(np.float64)) > np.abs(x)
        u = f.view(np.uint32)
        u = np.where(over, u - np.uint32(1), u)                   # truncated towards zero
        cut = np.abs(x) - np.abs(u.view(np.float32).astype(np.float64))
        cut = np.where(cut != 0, cut, rest * np.sign(x))          # beyond the truncated value, or short of it
    low = u & np.uint32(0xFFFF)
    odd = ((u >> np.uint32(16)) & np.uint32(1)).astype(bool)
    up = (low > 0x8000) | ((low == 0x8000) & ((cut > 0) | ((cut == 0) & odd)))
    out = ((u >> np.uint32(16)) + up.astype(np.uint32)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), out)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def bf16(x, rest=0.0):
    return bf16_value(bf16_bits(x, rest))


def two_sum(a, b):
    """a + b = s + e exactly (s the rounded sum)."""
    s = a + b
    t = s - a
    return s, (a - (s - t)) + (b - t)


def quantise(x, axis, bits):
    """Groups along `axis`: (codes, min, step) of float64 values that bf16 holds.  Differences
    carry what float64 cuts from them (exponents may lie far apart)."""
    q = 2 ** bits - 1
    lo, hi = x.min(axis=axis, keepdims=True), x.max(axis=axis, keepdims=True)
    bad = ~(np.maximum(np.abs(lo), np.abs(hi)) < 2.0 ** 126)
    lo0, hi0 = np.where(bad, 0.0, lo), np.where(bad, 0.0, hi)
    span, rest = two_sum(hi0, -lo0)
    step = span / q
    left = (span - step * q) + rest                               # exact where step has few bits: on a border
    step = bf16(step, left)
    code = np.zeros_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        d, e = two_sum(x, -lo0)
        for j in range(q):                                        # half steps passed; on one: the even code
            edge = (2 * j + 1) * step
            past, on = (2.0 * d > edge) | ((2.0 * d == edge) & (e > 0)), (2.0 * d == edge) & (e == 0)
            code += past if j % 2 == 0 else past | on
    code = np.where((step > 0) & ~bad, code, 0.0)
    return code, np.where(bad, np.nan, lo0), np.where(bad, np.nan, step)


def value_of(lo, code, step):
    return bf16(*two_sum(lo, code * step))


def held(rows, length, bits):
    """rows [T][2][N][D] (float64 of bf16 values): (K, V) [length][N][D] as the cache reads,
    and the keys' (min, value of the largest code) [blocks][N][D]."""
    rows = np.asarray(rows, np.float64)
    N, D = rows.shape[2:]
    full = length // BLK * BLK
    out = rows[:length].copy()
    kb = rows[:full, 0].reshape(-1, BLK, N, D)
    code, lo, step = quantise(kb, 1, bits)
    out[:full, 0] = value_of(lo, code, step).reshape(full, N, D)
    ends = (lo[:, 0], value_of(lo, 2.0 ** bits - 1, step)[:, 0])
    vb = rows[:full, 1].reshape(full, N, D // BLK, BLK)
    code, lo, step = quantise(vb, 3, bits)
    out[:full, 1] = value_of(lo, code, step).reshape(full, N, D)
    return out[:, 0], out[:, 1], ends


def scores(q, ends):
    """[N][blocks] bounds of q [H][D]."""
    lo, hi = ends
    nb, N, D = lo.shape
    G = q.shape[0] // N
    qq = q.reshape(N, G, 1, D)
    with np.errstate(invalid="ignore"):
        s = (np.maximum(qq, 0) * hi.transpose(1, 0, 2)[:, None] + np.minimum(qq, 0) * lo.transpose(1, 0, 2)[:, None]).sum(-1)
    return s.max(axis=1)


def select(q, ends, n_blocks, keep_first, keep_last, shared):
    s = scores(q, ends)
    if shared:
        s = s.max(axis=0, keepdims=True)
    nb = s.shape[1]
    out = np.full((s.shape[0], n_blocks), -1, np.int32)
    for i, row in enumerate(s):
        rank = [(0 if b < keep_first or b >= nb - keep_last else 1 if math.isnan(v) else 2,
                 0.0 if math.isnan(v) else -v, b) for b, v in enumerate(row)]
        got = sorted(b for _, _, b in sorted(rank)[:n_blocks])
        out[i, : len(got)] = got
    return out


def attend(q, k, v, p_err=2.0 ** -16):
    """softmax(q K^T / sqrt(D)) V for one row q [D] over k, v [n][D], and an error bound of a
    pass whose scores are fp32 sums of exact products: (out, bound).
      scores: D products added in fp32, each addition off by at most 2^-22 of the sum of the
      magnitudes so far (tensor cores may cut instead of round): |ds| <= D 2^-22 A / sqrt(D),
      A = max_n sum |q k|; the exponent's argument adds 2^-23 |s|; sums of p and of p v in
      fp32: 2^-20 together.  A relative error r of every p, in numerator and denominator,
      moves the output by at most 2 r sum(p |v|) / sum(p).  The probabilities that meet the
      values, but not their sum, are rounded further by p_err: 2^-16 as bf16 hi + lo, 2^-8
      (half a step of bf16) as bf16; that moves the output by p_err sum(p |v|) / sum(p)."""
    D = q.shape[0]
    if len(k) == 0:
        return np.zeros(D), np.zeros(D)
    s = k @ q / math.sqrt(D)
    p = np.exp(s - s.max())
    p /= p.sum()
    A = (np.abs(k) @ np.abs(q)).max() / math.sqrt(D)
    r = D * 2.0 ** -22 * A + 2.0 ** -23 * np.abs(s).max() + 2.0 ** -20
    return p @ v, (2 * r + p_err) * (p @ np.abs(v)) + 1e-30


def line_of(parent, j):
    """Drafted tokens that j sees (itself first), None for padding, "bad" for a wrong line."""
    if parent[j] == -2:
        return None
    seen, p = [], j
    while p >= 0:
        seen.append(p)
        up = int(parent[p])
        if up >= p or up < -1:
            return "bad"
        p = up
    return seen
