"""Cases of a prompt's way through a full-attention layer: queries and keys are normed by
head and rotated to their positions, packed prompts attend over themselves, and pieces of a
prompt attend over the quantised cache that holds what came before.

Rotation of the first R of D channels of a head x at position t, after an optional norm by
head, x / sqrt(mean(x^2) + eps) * weight:
    (a, b) -> gain (a cos - b sin, a sin + b cos),   angle = t theta_i
with (a, b) channels (2i, 2i + 1) ("pairs") or (i, i + R/2) ("halves").
Attention: out_i = softmax(q_i K^T / sqrt(D)) V over the tokens that token i sees: those of
its sequence up to itself, and the cached ones before.  The cache holds blocks of 32 tokens in
b bits (keys per channel of a block, values per token and 32 channels), the tokens of the last,
unfinished block as they are:
    step = bf16((max - min) / (2^b - 1)),  code = min(2^b - 1, rint((x - min) / step)),
    value = bf16(min + code step).

Plain forms compute in 32 bits; angles, codes and steps in 64.
"""
import math
import random

import torch

own = False

G = 32          # tokens of a block, channels of a value group
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 sequences at far positions: the smallest call, latency counts
        dict(name="rotate-step", op="rotate", rows=32, H=32, N=8, D=128, R=128, layout="pairs", scaling="plain", base=10000.0, norm=False, f32=False, fused=False),
        # one prompt, heads normed and rotated where the layer's one projection left q | k | v
        dict(name="rotate-prompt", op="rotate", rows=8192, H=32, N=8, D=128, R=128, layout="halves", scaling="bands", base=500000.0, norm=True, f32=False, fused=True),
        # fp32 rows, half of each head rotates, an odd number of rows
        dict(name="rotate-f32-part", op="rotate", rows=4001, H=28, N=4, D=128, R=64, layout="halves", scaling="yarn", base=10000.0, norm=True, f32=True, fused=False),
        # a batch of long prompts at once
        dict(name="rotate-batch", op="rotate", rows=65536, H=28, N=4, D=128, R=128, layout="pairs", scaling="linear", base=10000.0, norm=False, f32=False, fused=False),
        # eight short questions: latency counts
        dict(name="prompt-short", op="prompt", S=8, T=130, H=32, N=8, D=128, fused=False, behind=0),
        # sixteen prompts of uneven lengths (some empty or of one token), rows left over behind them
        dict(name="prompt-ragged", op="prompt", S=16, T=4096, H=28, N=4, D=128, fused=False, behind=37),
        # small heads, read from the projection's rows
        dict(name="prompt-d64", op="prompt", S=2, T=4096, H=32, N=8, D=64, fused=True, behind=0),
        # one ordinary long prompt
        dict(name="prompt-8k", op="prompt", S=1, T=8192, H=32, N=8, D=128, fused=True, behind=0),
        # twice that: the largest prompt
        dict(name="prompt-16k", op="prompt", S=1, T=16384, H=32, N=8, D=128, fused=False, behind=0),
        # the last few tokens of four prompts, uneven
        dict(name="chunk-small", op="chunk", S=4, T=8192, n=48, H=32, N=8, D=128, bits=4),
        # pieces of eight prompts of uneven lengths
        dict(name="chunk-batch", op="chunk", S=8, T=16384, n=512, H=28, N=4, D=128, bits=4),
        # the last piece of a very long prompt: the largest work
        dict(name="chunk-long", op="chunk", S=1, T=131072, n=2048, H=32, N=8, D=128, bits=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "prompt", "prompt", "prompt", "chunk", "chunk", "chunk"])
    D = rng.choice([64, 128, 128, 128, 256])
    N = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rotate":
        rows = _log(rng, 1, 65536 * 32 * 128 // ((N * g + N) * D))
        return dict(op=op, rows=min(rows, 65536), H=N * g, N=N, D=D, R=rng.choice([D, D, D // 2, 16]), layout=rng.choice(["pairs", "halves"]),
                    scaling=rng.choice(["plain", "linear", "bands", "yarn"]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    norm=rng.random() < 0.5, f32=rng.random() < 0.3, fused=rng.random() < 0.4)
    S = _log(rng, 1, 24)
    if op == "prompt":
        # scores of the plain form: half as many as the largest listed case's
        most = int(math.sqrt(16384.0 * 16384.0 * 32 * 128 / (2.0 * S * N * g * max(D, 128))))
        return dict(op=op, S=S, T=_log(rng, 1, min(most, 16384)), H=N * g, N=N, D=D, fused=rng.random() < 0.4, behind=rng.choice([0, 0, 1, 50]))
    n = _log(rng, 1, 2048)
    cap = min(131072.0 * 1024 / (S * N * D), 2048.0 * 131072 * 32 * 128 / (S * n * N * g * max(D, 128))) / 2
    T = _log(rng, 257, max(300, min(131072, int(cap))))
    return dict(op=op, S=S, T=T, n=max(1, min(n, T // 2)), H=N * g, N=N, D=D, bits=rng.choice([2, 4, 4]))


# ------------------------------------------------------------------ inputs
ORIGINAL, FACTOR, LOW, HIGH, FAST, SLOW = 8192, 8.0, 1.0, 4.0, 32.0, 1.0


def _theta(c):
    """(theta_i, gain) of a case's rotation, as Python floats."""
    R, base, f = c["R"], c["base"], FACTOR
    th = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if c["scaling"] == "linear":
        return [t / f for t in th], 1.0
    if c["scaling"] == "bands":
        # wavelengths beyond ORIGINAL / LOW are stretched, those below ORIGINAL / HIGH stay
        smooth = [min(1.0, max(0.0, (ORIGINAL * t / (2 * math.pi) - LOW) / (HIGH - LOW))) for t in th]
        return [t * s + t / f * (1 - s) for t, s in zip(th, smooth)], 1.0
    if c["scaling"] == "yarn":
        at = lambda turns: R * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(FAST))), min(R - 1, math.ceil(at(SLOW)))
        keep = [1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(R // 2)]
        return [t * k + t / f * (1 - k) for t, k in zip(th, keep)], 0.1 * math.log(f) + 1.0
    return th, 1.0


def _rows(gen, S, n, N, D):
    """K | V rows [S][n][2ND] in fp32: keys drift by topic (a new centroid every 200 or so
    tokens) around per-channel offsets, some of them large; values are near normal."""
    dev = "cuda"
    k = torch.randn(S, n, N, D, generator=gen, device=dev)
    off = torch.randn(1, 1, N, D, generator=gen, device=dev)
    off = off * torch.where(torch.rand(1, 1, N, D, generator=gen, device=dev) < 0.05, 6.0, 0.7)
    topics = torch.randn(S, n // 200 + 1, N, D, generator=gen, device=dev) * 0.8
    k = k.mul_(0.7).add_(topics.repeat_interleave(200, dim=1)[:, :n]).add_(off)
    v = torch.randn(S, n, N, D, generator=gen, device=dev)
    return torch.cat([k.reshape(S, n, N * D), v.reshape(S, n, N * D)], dim=2)


def _lengths(c, seed):
    """Tokens of each packed prompt: the first is full, the others anything from none on, two
    of them together as long as the first (so that the rows of a batch do not go by the seed)."""
    r = random.Random(seed * 7919 + 13)
    lens, T = [c["T"]], c["T"]
    while len(lens) < c["S"]:
        m = T // 2 if len(lens) == c["S"] - 1 else r.choice([0, 1]) if r.random() < 0.12 else r.randint(0, T)
        lens += [m, T - m][: c["S"] - len(lens)]
    return lens


def _inputs(c, seed):
    """The user's tensors, from the seed alone.  q, k, v are views of one projection's rows
    q | k | v where the case is fused."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    H, N, D = c["H"], c["N"], c["D"]
    x = {}
    if c["op"] == "rotate":
        rows, dt = c["rows"], torch.float32 if c["f32"] else torch.bfloat16
        wide = (H + 2 * N) * D if c["fused"] else (H + N) * D
        p = torch.randn(rows, wide, generator=gen, device="cuda").mul_(1.5).to(dt)
        q, k = p[:, : H * D].view(rows, H, D), p[:, H * D: (H + N) * D].view(rows, N, D)
        x["q"], x["k"] = (q, k) if c["fused"] else (q.contiguous(), k.contiguous())
        # prompts behind one another, each from its own position on
        r = random.Random(seed * 31 + 5)
        first = r.randint(0, 131072 - 1)
        at = torch.arange(rows, device="cuda")
        x["pos"] = ((first + at * (4093 if rows <= 64 else 1)) % 131072).to(torch.int32)
        if c["norm"]:
            x["q_weight"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
            x["k_weight"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        return x
    if c["op"] == "prompt":
        lens = _lengths(c, seed)
        start = [0]
        for m in lens:
            start.append(start[-1] + m)
        rows = start[-1] + c["behind"]
        q = torch.randn(rows, H, D, generator=gen, device="cuda").mul_(1.2).to(torch.bfloat16)
        kv = _rows(gen, 1, rows, N, D)[0].to(torch.bfloat16)
        if c["fused"]:
            p = torch.cat([q.view(rows, H * D), kv], dim=1)
            q = p[:, : H * D].view(rows, H, D)
            kv = p[:, H * D:]
        x["q"], x["k"], x["v"] = q, kv[:, : N * D].unflatten(1, (N, D)), kv[:, N * D:].unflatten(1, (N, D))
        x["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        return x
    S, T, n = c["S"], c["T"], c["n"]
    r = random.Random(seed * 7919 + 13)
    lens = [T - n] + [r.randint((T - n) // 4, T - n) for _ in range(S - 1)]
    new = [n] + [r.randint(max(1, n // 4), n) for _ in range(S - 1)]
    x["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    x["past"] = _rows(gen, S, T - n, N, D).to(torch.bfloat16)
    x["kv"] = _rows(gen, S, n, N, D).to(torch.bfloat16)
    x["q"] = torch.randn(S, n, H, D, generator=gen, device="cuda").mul_(1.2).to(torch.bfloat16)
    return x


def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    st = {"c": c, "x": x}
    if c["op"] == "rotate":
        if own:
            from reference_residual_kv_gb300 import rkv
            scaling = {"plain": None, "linear": ("linear", FACTOR), "bands": ("bands", FACTOR, ORIGINAL, LOW, HIGH),
                       "yarn": ("yarn", FACTOR, ORIGINAL, FAST, SLOW)}[c["scaling"]]
            st["rope"] = rkv.make_rope(c["D"], c["R"], layout=c["layout"], base=c["base"], scaling=scaling)
            st["heads"] = rkv.PromptHeads(c["H"], c["N"], c["D"])
        else:
            theta, st["gain"] = _theta(c)
            st["theta"] = torch.tensor(theta, dtype=torch.float64, device="cuda")
        st["q"] = torch.zeros(c["rows"], c["H"], c["D"], dtype=x["q"].dtype, device="cuda")
        st["k"] = torch.zeros(c["rows"], c["N"], c["D"], dtype=x["q"].dtype, device="cuda")
        return st
    st["out"] = torch.zeros(x["q"].shape, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "prompt":
        if own:
            from reference_residual_kv_gb300 import rkv
            st["heads"] = rkv.PromptHeads(c["H"], c["N"], c["D"])
        return st
    past = x.pop("past")
    if own:
        from reference_residual_kv_gb300 import rkv
        st["cache"] = rkv.DenseCache(rkv.make_dense_params(c["S"], c["T"], c["N"], c["D"], bits=c["bits"]))
        st["cache"].write(past, torch.zeros_like(x["len"]), x["len"])
    else:
        st["cache"] = _held_in_blocks(c, past)
    return st


# ------------------------------------------------------------------ plain forms
def _rotated(c, x, weight, pos, theta, gain):
    R = c["R"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    # whole turns drop out in 64 bits
    turns = pos.double()[:, None] * (theta / (2 * math.pi))
    angle = ((turns - torch.floor(turns)) * (2 * math.pi))[:, None]
    co, si = (torch.cos(angle) * gain).float(), (torch.sin(angle) * gain).float()
    if c["layout"] == "pairs":
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * co - b * si, a * si + b * co], dim=-1).flatten(-2)
    else:
        a, b = y[..., : R // 2], y[..., R // 2: R]
        turned = torch.cat([a * co - b * si, a * si + b * co], dim=-1)
    return torch.cat([turned, y[..., R:]], dim=-1).to(x.dtype)


def _softmax_sum(score, value):
    """softmax(score) value over the last axis of score (overwritten); rows with nothing give zeros."""
    m = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ value) / torch.where(total > 0, total, 1.0)


def _prompt(c, q, k, v, start, out):
    S, T, H, N, D = c["S"], c["T"], c["H"], c["N"], c["D"]
    g = H // N
    t = torch.arange(T, device="cuda")
    at = start[:-1].long()[:, None] + t
    there = at < start[1:].long()[:, None]
    at = torch.where(there, at, 0)
    # every prompt in a box of T rows: [S][N][T g][D], [S][N][T][D]
    rows = torch.where(there[..., None, None], q[at].float(), 0.0).view(S, T, N, g, D).permute(0, 2, 1, 3, 4).reshape(S, N, T * g, D)
    keys = torch.where(there[..., None, None], k[at].float(), 0.0).permute(0, 2, 1, 3)
    vals = torch.where(there[..., None, None], v[at].float(), 0.0).permute(0, 2, 1, 3)
    score = ((rows / math.sqrt(D)) @ keys.transpose(2, 3)).view(S, N, T, g, T)
    score.masked_fill_((t[None, :] > t[:, None])[None, None, :, None], -math.inf)
    o = _softmax_sum(score.view(S, N, T * g, T), vals).view(S, N, T, g, D).permute(0, 2, 1, 3, 4).reshape(S, T, H, D)
    out[at[there]] = o[there].to(torch.bfloat16)
    return out


def _to_bf16(x):
    """Rounds 64 bits to bf16 once: a 32-bit value that lands on a border by its own
    rounding is put back on the side that it came from."""
    f = x.float()
    at_border = (f.contiguous().view(torch.int32) & 0xFFFF) == 0x8000
    e = x - f.double()
    f = torch.where(at_border & (e > 0), torch.nextafter(f, torch.full_like(f, math.inf)), f)
    f = torch.where(at_border & (e < 0), torch.nextafter(f, torch.full_like(f, -math.inf)), f)
    return f.to(torch.bfloat16)


def _quant(x, dim, qmax):
    """x in 64 bits; extremes over `dim`: (codes, min, step)."""
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    step = _to_bf16((hi - lo) / qmax)
    d = step.double()
    code = torch.where(d > 0, torch.round((x - lo) / torch.where(d > 0, d, 1.0)), 0.0).clamp_(0, qmax)
    return code.to(torch.uint8), lo.to(torch.bfloat16), step


def _held_in_blocks(c, past):
    S, N, D, m = c["S"], c["N"], c["D"], past.shape[1]
    nb, qmax = m // G, 2 ** c["bits"] - 1
    raw = past.view(S, m, 2, N, D)
    x = raw[:, : nb * G].reshape(S, nb, G, 2, N, D)
    qk, k_min, k_step = _quant(x[:, :, :, 0].double(), 2, qmax)
    qv, v_min, v_step = _quant(x[:, :, :, 1].double().unflatten(4, (D // G, G)), 5, qmax)
    return {"raw": raw, "k": (qk, k_min, k_step), "v": (qv, v_min, v_step)}


def _values(held, shape):
    code, lo, step = held
    return (code.float() * step.float() + lo.float()).to(torch.bfloat16).float().reshape(shape)


def _chunk(c, cache, q, kv, length, n_new, out):
    S, n, H, N, D = c["S"], c["n"], c["H"], c["N"], c["D"]
    g, raw = H // N, cache["raw"]
    m = raw.shape[1]
    full = m // G * G
    t = torch.arange(m, device="cuda")
    done = (t < length.long()[:, None] // G * G)[..., None, None]
    k, v = raw[:, :, 0].float(), raw[:, :, 1].float()
    k[:, :full] = torch.where(done[:, :full], _values(cache["k"], (S, full, N, D)), k[:, :full])
    v[:, :full] = torch.where(done[:, :full], _values(cache["v"], (S, full, N, D)), v[:, :full])
    new = kv.view(S, n, 2, N, D).float()
    k = torch.cat([k, new[:, :, 0]], dim=1).permute(0, 2, 1, 3)
    v = torch.cat([v, new[:, :, 1]], dim=1).permute(0, 2, 1, 3)
    j = torch.arange(n, device="cuda")
    rows = q.float().view(S, n, N, g, D).permute(0, 2, 1, 3, 4).reshape(S, N, n * g, D)
    score = ((rows / math.sqrt(D)) @ k.transpose(2, 3)).view(S, N, n, g, m + n)
    hidden = torch.cat([(t >= length.long()[:, None])[:, None].expand(S, n, m), (j[None, :] > j[:, None]).expand(S, n, n)], dim=2)
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    o = _softmax_sum(score.view(S, N, n * g, m + n), v).view(S, N, n, g, D).permute(0, 2, 1, 3, 4).reshape(S, n, H, D)
    live = j < n_new.long()[:, None]
    out[live] = o[live].to(torch.bfloat16)
    return out


def run(state):
    c, x = state["c"], state["x"]
    if c["op"] == "rotate":
        if own:
            state["heads"].rotate(state["rope"], x["q"], x["k"], x["pos"], state["q"], state["k"], x.get("q_weight"), x.get("k_weight"), eps=EPS)
            return {"q": state["q"], "k": state["k"]}
        return {"q": _rotated(c, x["q"], x.get("q_weight"), x["pos"], state["theta"], state["gain"]),
                "k": _rotated(c, x["k"], x.get("k_weight"), x["pos"], state["theta"], state["gain"])}
    if c["op"] == "prompt":
        if own:
            state["heads"].attend(x["q"], x["k"], x["v"], x["start"], state["out"])
            return {"out": state["out"]}
        return {"out": _prompt(c, x["q"], x["k"], x["v"], x["start"], state["out"])}
    if own:
        state["cache"].chunk_attend(c["H"], x["q"], x["kv"], x["len"], state["out"], n_new=x["n_new"])
        return {"out": state["out"]}
    return {"out": _chunk(c, state["cache"], x["q"], x["kv"], x["len"], x["n_new"], state["out"])}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    H, N, D = c["H"], c["N"], c["D"]
    if c["op"] == "rotate":
        values = c["rows"] * (H + N) * D
        return {"bytes": values * (8 if c["f32"] else 4) + 4.0 * c["rows"], "flops": values * (7.0 if c["norm"] else 3.0)}
    S, T = c["S"], c["T"]
    if c["op"] == "prompt":
        # the first prompt is full, two others are as long as it together
        mean = T * (1 + (S - 1) * 0.5) / S
        square = T * T * (1 + (S - 1) // 2 * 0.707 + (S - 1) % 2 * 0.25) / S
        return {"bytes": S * mean * (2 * H + 2 * N) * D * 2, "flops": 4.0 * S * H * D * (square + mean) / 2}
    n = c["n"]
    block = N * (8 * D * c["bits"] + 8 * D)            # codes, extremes and steps of 32 tokens
    past = (T - n) * (1 + (S - 1) * 0.625) / S
    new = n * (1 + (S - 1) * 0.625) / S
    square = n * n * (1 + (S - 1) * 0.4375) / S
    return {"bytes": S * (past / G * block + new * (2 * H + 2 * N) * D * 2),
            "flops": 4.0 * H * D * ((T - n) * n * (1 + (S - 1) * 0.39) + S * (square + new) / 2)}


# ------------------------------------------------------------------ the definition in 64 bits
def _bf16_of(x):
    """Nearest value with eight significant bits, ties to even (normal range)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0) / 256.0, e)


def _block_values(x, dim, qmax):
    """What groups of values (64 bits, extremes over `dim`) read as: the code counts the half
    steps that a value has passed; on a half step it goes to the even code."""
    lo = x.min(dim, keepdim=True).values
    step = _bf16_of((x.max(dim, keepdim=True).values - lo) / qmax)
    code = torch.zeros_like(x)
    for j in range(qmax):
        border = (2 * j + 1) * step
        code += ((2.0 * (x - lo) > border) if j % 2 == 0 else (2.0 * (x - lo) >= border)).double()
    return _bf16_of(lo + torch.where(step > 0, code, 0.0) * step)


def _causal(q, keys, vals, before):
    """One KV head: q [n][g][D], keys and vals [before + n][D]; row i sees before + i + 1 tokens."""
    n, g, D = q.shape
    out = torch.empty_like(q)
    for a in range(0, n, 2048):
        b = min(n, a + 2048)
        z = torch.einsum("igd,jd->gij", q[a:b], keys[: before + b]) / math.sqrt(D)
        late = torch.arange(before + b, device="cuda") > torch.arange(before + a, before + b, device="cuda")[:, None]
        out[a:b] = torch.einsum("gij,jd->igd", torch.softmax(z.masked_fill_(late, -math.inf), dim=-1), vals[: before + b])
    return out


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    H, N, D = c["H"], c["N"], c["D"]
    g = H // N
    if c["op"] == "rotate":
        theta, gain = _theta(c)
        R = c["R"]
        angle = torch.remainder(x["pos"].double()[:, None] * torch.tensor(theta, dtype=torch.float64, device="cuda"), 2 * math.pi)
        turn = torch.polar(torch.full_like(angle, gain), angle)[:, None]
        got = {}
        for name in ("q", "k"):
            y = x[name].double()
            if c["norm"]:
                y = y / torch.sqrt(torch.linalg.vecdot(y, y)[..., None] / D + EPS) * x[name + "_weight"].double()
            if c["layout"] == "pairs":
                z = torch.view_as_real(torch.view_as_complex(y[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn).flatten(-2)
            else:
                w = torch.complex(y[..., : R // 2].contiguous(), y[..., R // 2: R].contiguous()) * turn
                z = torch.cat([w.real, w.imag], dim=-1)
            got[name] = torch.cat([z, y[..., R:]], dim=-1)
        return got
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    if c["op"] == "prompt":
        start = x["start"].tolist()
        for a, b in zip(start[:-1], start[1:]):
            for h in range(N):
                if b > a:
                    out[a:b, h * g: (h + 1) * g] = _causal(x["q"][a:b, h * g: (h + 1) * g].double(), x["k"][a:b, h].double(), x["v"][a:b, h].double(), 0)
        return {"out": out}
    qmax = 2 ** c["bits"] - 1
    for s, (m, n) in enumerate(zip(x["len"].tolist(), x["n_new"].tolist())):
        past = x["past"][s, :m].view(m, 2, N, D)
        new = x["kv"][s, :n].view(n, 2, N, D)
        full = m // G * G
        for h in range(N):
            k, v = past[:, 0, h].double(), past[:, 1, h].double()
            if full:
                k[:full] = _block_values(k[:full].view(full // G, G, D), 1, qmax).view(full, D)
                v[:full] = _block_values(v[:full].view(full, D // G, G), 2, qmax).view(full, D)
            k, v = torch.cat([k, new[:, 0, h].double()]), torch.cat([v, new[:, 1, h].double()])
            out[s, :n, h * g: (h + 1) * g] = _causal(x["q"][s, :n, h * g: (h + 1) * g].double(), k, v, m)
    return {"out": out}
