"""Cases of the dense quantised cache: the cache that a full-attention layer keeps whole,
quantised block by block as it is written, read back, and attended over by single tokens
(all blocks, or those that a cheap score selects) and by trees of drafted tokens.

A block is 32 tokens of one KV head.  Keys are quantised per channel over the block,
values per token over groups of 32 channels:
    delta = bf16((max - min) / (2^b - 1)),  code = min(2^b - 1, rint((x - min) / delta)),
    value = bf16(min + code delta)
(each bf16() one rounding to nearest even).  The tokens of the last, unfinished block stay
as they are, in bf16.

Plain forms compute in 32 bits, borders (codes, steps, scores that are ranked) in 64.
"""
import math
import random

import torch

own = False

G = 32          # tokens of a block, channels of a value group
KV_BASE = dict(S=1, N=8, D=128, H=32, bits=4)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's write for 32 sequences at different places (some finish a block),
        # read back over the last 32 tokens: the smallest call, latency counts
        dict(name="write-append", op="write", S=32, N=8, D=128, bits=4, T=2048, n=1, append=True, f32=False, back=32),
        # eight prompts of uneven lengths at 2 bits (image and text batch), read back whole
        dict(name="write-ragged-int2", op="write", S=8, N=8, D=128, bits=2, T=4096, n=4001, append=False, f32=False, back=4001),
        # short fp32 rows, small heads, an odd length that ends inside a block
        dict(name="write-f32-odd", op="write", S=3, N=4, D=64, bits=4, T=1024, n=717, append=False, f32=True, back=717),
        # one long prompt
        dict(name="write-long", op="write", S=1, N=8, D=128, bits=4, T=131072, n=131072, append=False, f32=False, back=131072),
        # a decode step's sparse read from a long cache: 30 % of the tokens and the last 512
        dict(name="read-sparse", op="read", S=1, N=8, D=128, bits=4, T=131072, frac=0.3, last=512),
        # single-token attention over the blocks that the score selects: short cache, latency
        dict(name="blocks-short", op="attend", S=1, N=8, D=128, H=32, bits=4, T=8192, sel=32, per_head=True, bf16=False),
        # the same over a long cache, an eighth of its blocks, one list for all heads (it
        # goes on to the sparse read of the layers behind)
        dict(name="blocks-long", op="attend", S=1, N=8, D=128, H=32, bits=4, T=131072, sel=512, per_head=False, bf16=False),
        # sixteen sequences of uneven lengths, seven query heads to a KV head
        dict(name="blocks-batch", op="attend", S=16, N=4, D=128, H=28, bits=4, T=32768, sel=128, per_head=True, bf16=True),
        # single-token attention over whole caches (a full-attention layer's decode step)
        dict(name="dense-decode", op="attend", S=8, N=8, D=128, H=32, bits=4, T=32768, sel=0, per_head=False, bf16=False),
        # a small tree of drafted tokens over a short cache
        dict(name="tree-small", op="tree", S=1, N=8, D=128, H=32, bits=4, T=4096, n=8, bf16=False),
        # sixteen sequences of uneven lengths, trees of up to 24 drafted tokens, odd groups
        dict(name="tree-batch", op="tree", S=16, N=4, D=128, H=28, bits=4, T=8192, n=24, bf16=True),
        # a full tree of 64 drafted tokens over a long cache: the largest work
        dict(name="tree-long", op="tree", S=1, N=8, D=128, H=32, bits=4, T=131072, n=64, bf16=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "attend", "attend", "tree", "tree"])
    D = rng.choice([64, 128, 128, 256]) if op != "tree" else rng.choice([64, 128, 128, 128])
    N = rng.choice([2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8]) if D <= 128 else rng.choice([1, 2, 3, 4])
    bits = rng.choice([2, 4, 4])
    S = _log(rng, 1, 24)
    cap = max(512, 131072 * 1024 // (S * N * D) // 2)          # half the largest listed cache
    T = _log(rng, 257, min(cap, 131072))
    if op == "write":
        if rng.random() < 0.4:
            return dict(op=op, S=S, N=N, D=D, bits=bits, T=T, n=1, append=True, f32=rng.random() < 0.3, back=rng.randint(1, 40))
        n = rng.randint(max(1, T // 3), T)
        return dict(op=op, S=S, N=N, D=D, bits=bits, T=T, n=n, append=False, f32=rng.random() < 0.3, back=n)
    if op == "read":
        return dict(op=op, S=S, N=N, D=D, bits=bits, T=T, frac=round(rng.uniform(0.02, 0.5), 3), last=rng.choice([0, 31, 64, 200]))
    if op == "attend":
        sel = rng.choice([0, _log(rng, 2, max(2, T // G))])
        return dict(op=op, S=S, N=N, D=D, H=N * g, bits=bits, T=T, sel=sel, per_head=rng.random() < 0.6, bf16=rng.random() < 0.5)
    return dict(op=op, S=S, N=N, D=D, H=N * g, bits=bits, T=T, n=_log(rng, 1, 64), bf16=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _lengths(c, seed, least=0):
    """Tokens of each sequence: the first is full, the others uneven (seeded on the host)."""
    r = random.Random(seed * 7919 + 13)
    return [c["T"]] + [r.randint(max(least, c["T"] // 4), c["T"]) for _ in range(c["S"] - 1)]


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


def _tree(c, seed):
    """Parents of the drafted tokens: -1 hangs on the cached text, -2 is padding."""
    r = random.Random(seed * 104729 + 7)
    rows = []
    for s in range(c["S"]):
        m = c["n"] if s == 0 else r.randint(max(1, c["n"] // 2), c["n"])
        rows.append([-2 if j >= m else -1 if j == 0 or r.random() < 0.08 else r.randint(max(0, j - 6), j - 1) for j in range(c["n"])])
    return rows


def _inputs(c, seed):
    """The user's tensors, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    S, N, D, T = c["S"], c["N"], c["D"], c["T"]
    x = {}
    if c["op"] == "write":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        if c["append"]:
            ends = _lengths(c, seed, least=40)
            pos = [e - 1 for e in ends]
            x["past"] = _rows(gen, S, T, N, D).to(torch.bfloat16)
            x["kv"] = _rows(gen, S, 1, N, D).to(dt)
            x["n_new"] = torch.ones(S, dtype=torch.int32, device="cuda")
            x["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        else:
            r = random.Random(seed * 31 + 5)
            ends = [c["n"]] + [r.randint(c["n"] // 3, c["n"]) for _ in range(S - 1)]
            x["kv"] = _rows(gen, S, c["n"], N, D).to(dt)
            x["n_new"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            x["pos"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        x["len"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        # the last `back` tokens of each sequence; -1 where it has fewer
        at = x["len"][:, None] - c["back"] + torch.arange(c["back"], device="cuda", dtype=torch.int32)
        x["sel"] = torch.where(at >= 0, at, -1).to(torch.int32).contiguous()
        return x
    lens = _lengths(c, seed)
    x["past"] = _rows(gen, S, T, N, D).to(torch.bfloat16)
    x["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["op"] == "read":
        n = int(c["frac"] * T) + c["last"]
        at = torch.rand(S, n, generator=gen, device="cuda") * x["len"][:, None]
        at = torch.minimum(at.to(torch.int32), x["len"][:, None] - 1)
        if c["last"]:
            at[:, n - c["last"]:] = x["len"][:, None] - c["last"] + torch.arange(c["last"], device="cuda", dtype=torch.int32)
        at = at.sort(dim=1).values
        x["sel"] = torch.where(at >= 0, at, -1).to(torch.int32).contiguous()
        return x
    n = c["n"] if c["op"] == "tree" else 1
    x["q"] = (torch.randn(S, n, c["H"], D, generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    if c["op"] == "attend":
        x["q"] = x["q"][:, 0].contiguous()
    else:
        x["draft"] = _rows(gen, S, n, N, D).to(torch.bfloat16)
        x["parent"] = torch.tensor(_tree(c, seed), dtype=torch.int32, device="cuda")
    return x


def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    S, N, D, T = c["S"], c["N"], c["D"], c["T"]
    st = {"c": c, "x": x}
    if c["op"] == "write" and c["append"]:
        first, count = x["past"], x["pos"]
    elif c["op"] == "write":
        first, count = None, None
    else:
        first, count = x.pop("past"), x["len"]
    zero = torch.zeros(S, dtype=torch.int32, device="cuda")
    out_dt = torch.bfloat16 if c.get("bf16") else torch.float32
    if own:
        from reference_residual_kv_gb300 import rkv
        st["cache"] = rkv.DenseCache(rkv.make_dense_params(S, T, N, D, bits=c["bits"]))
        if first is not None:
            st["cache"].write(first, zero, count)
        if "sel" in x:
            st["k"] = torch.empty(S, x["sel"].shape[1], N * D, dtype=torch.bfloat16, device="cuda")
            st["v"] = torch.empty_like(st["k"])
        else:
            st["out"] = torch.empty(x["q"].shape, dtype=out_dt, device="cuda")
            if c.get("sel"):
                st["blocks"] = torch.empty(S, N if c["per_head"] else 1, c["sel"], dtype=torch.int32, device="cuda")
    else:
        st["cache"] = _empty(c)
        if first is not None:
            _write(c, st["cache"], first, zero, count)
    x.pop("past", None)
    return st


# ------------------------------------------------------------------ plain forms
def _empty(c):
    S, N, D, nb = c["S"], c["N"], c["D"], c["T"] // G
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    return {"raw": z(S, c["T"], 2, N, D, dtype=torch.bfloat16),
            "codes": z(S, nb, G, 2, N, D, dtype=torch.uint8),
            "k_min": z(S, nb, 1, N, D, dtype=torch.bfloat16), "k_step": z(S, nb, 1, N, D, dtype=torch.bfloat16),
            "v_min": z(S, nb, G, N, D // G, dtype=torch.bfloat16), "v_step": z(S, nb, G, N, D // G, dtype=torch.bfloat16)}


def _to_bf16(x):
    """Rounds 64 bits to bf16 once: a 32-bit value that lands on a border by its own
    rounding is put back on the side that it came from."""
    f = x.float()
    at_border = (f.contiguous().view(torch.int32) & 0xFFFF) == 0x8000
    e = x - f.double()
    up, down = torch.full_like(f, math.inf), torch.full_like(f, -math.inf)
    f = torch.where(at_border & (e > 0), torch.nextafter(f, up), f)
    f = torch.where(at_border & (e < 0), torch.nextafter(f, down), f)
    return f.to(torch.bfloat16)


def _quant(x, dim, qmax):
    """x in 64 bits; extremes over `dim`: (codes, min, step)."""
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    step = _to_bf16((hi - lo) / qmax)
    d = step.double()
    q = torch.where(d > 0, torch.round((x - lo) / torch.where(d > 0, d, 1.0)), 0.0).clamp_(0, qmax)
    return q.to(torch.uint8), lo.to(torch.bfloat16), step


def _write(c, cache, kv, pos, n_new):
    S, n, N, D, T = c["S"], kv.shape[1], c["N"], c["D"], c["T"]
    qmax = 2 ** c["bits"] - 1
    rows = kv.to(torch.bfloat16).view(S, n, 2, N, D)
    j = torch.arange(n, device="cuda")
    live = j[None] < n_new[:, None]
    s_at, j_at = live.nonzero(as_tuple=True)
    cache["raw"][s_at, pos.long()[s_at] + j_at] = rows[s_at, j_at]
    # the blocks that these rows finish
    b = pos.long()[:, None] // G + torch.arange(n // G + 1, device="cuda")
    done = (b + 1) * G <= (pos + n_new).long()[:, None]
    s_at, i_at = done.nonzero(as_tuple=True)
    b_at = b[s_at, i_at]
    x = cache["raw"][: , : T // G * G].view(S, T // G, G, 2, N, D)[s_at, b_at].double()
    qk, k_min, k_step = _quant(x[:, :, 0], 1, qmax)
    qv, v_min, v_step = _quant(x[:, :, 1].unflatten(3, (D // G, G)), 4, qmax)
    cache["codes"][s_at, b_at] = torch.stack([qk, qv.flatten(3)], dim=2)
    cache["k_min"][s_at, b_at], cache["k_step"][s_at, b_at] = k_min, k_step
    cache["v_min"][s_at, b_at], cache["v_step"][s_at, b_at] = v_min.squeeze(4), v_step.squeeze(4)


def _values(codes, lo, step):
    """What codes stand for, in 32 bits (rounded to bf16 as the cache defines)."""
    return (codes.float() * step.float() + lo.float()).to(torch.bfloat16).float()


def _read(c, cache, length, sel):
    S, N, D = c["S"], c["N"], c["D"]
    t = sel.long().clamp(min=0)
    b = (t // G).clamp(max=max(0, c["T"] // G - 1))
    s = torch.arange(S, device="cuda")[:, None].expand_as(t)
    o = t % G
    q = cache["codes"][s, b, o]
    k = _values(q[:, :, 0], cache["k_min"][s, b, 0], cache["k_step"][s, b, 0])
    v = _values(q[:, :, 1].unflatten(3, (D // G, G)), cache["v_min"][s, b, o][..., None], cache["v_step"][s, b, o][..., None]).flatten(3)
    raw = cache["raw"][s, t].float()
    done = (t // G < length.long()[:, None] // G)[..., None, None]
    live = (sel >= 0)[..., None, None]
    k = torch.where(live, torch.where(done, k, raw[:, :, 0]), 0.0)
    v = torch.where(live, torch.where(done, v, raw[:, :, 1]), 0.0)
    return k.flatten(2).to(torch.bfloat16), v.flatten(2).to(torch.bfloat16)


def _all_values(c, cache, length):
    """K and V of every token in 32 bits, [S][T][N][D]; what lies behind a length is zero."""
    S, T, N, D = c["S"], c["T"], c["N"], c["D"]
    full = T // G * G
    k = torch.zeros(S, T, N, D, device="cuda")
    v = torch.zeros(S, T, N, D, device="cuda")
    k[:, :full] = _values(cache["codes"][:, :, :, 0], cache["k_min"], cache["k_step"]).flatten(1, 2)
    v[:, :full] = _values(cache["codes"][:, :, :, 1].unflatten(4, (D // G, G)), cache["v_min"][..., None], cache["v_step"][..., None]).flatten(4).flatten(1, 2)
    t = torch.arange(T, device="cuda")[None]
    done = (t < length.long()[:, None] // G * G)[..., None, None]
    there = (t < length.long()[:, None])[..., None, None]
    k = torch.where(done, k, torch.where(there, cache["raw"][:, :, 0].float(), 0.0))
    v = torch.where(done, v, torch.where(there, cache["raw"][:, :, 1].float(), 0.0))
    return k, v


def _select(c, cache, q, length):
    """The blocks with the largest bound on q . k, the first and the last one always:
    [S][N or 1][sel] ascending, -1 behind."""
    S, N, D, H, nb = c["S"], c["N"], c["D"], c["H"], c["T"] // G
    q = q.view(S, 1, N, H // N, D).double()
    lo = cache["k_min"].double()[:, :, 0, :, None]
    hi = _values(torch.full_like(cache["k_min"], 2 ** c["bits"] - 1), cache["k_min"], cache["k_step"]).double()[:, :, 0, :, None]
    score = (torch.maximum(q, torch.zeros_like(q)) * hi + torch.minimum(q, torch.zeros_like(q)) * lo).sum(-1).amax(-1)
    score = score.permute(0, 2, 1)
    if not c["per_head"]:
        score = score.amax(1, keepdim=True)
    b = torch.arange(nb, device="cuda")
    have = (length.long() // G)[:, None, None]
    score = torch.where((b == 0) | (b == have - 1), math.inf, score)
    score = torch.where(b < have, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices[:, :, : c["sel"]]
    picked = torch.where(order < have, order, nb).sort(dim=2).values
    picked = torch.where(picked < nb, picked, -1)
    pad = torch.full((S, picked.shape[1], c["sel"] - picked.shape[2]), -1, device="cuda")
    return torch.cat([picked, pad], dim=2).to(torch.int32)


def _softmax_sum(score, value):
    """softmax(score) value over the last axis of score; rows with nothing give zeros."""
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return (p @ value) / torch.where(total > 0, total, 1.0)


def _attend(c, cache, q, length, blocks):
    S, N, D, H, T = c["S"], c["N"], c["D"], c["H"], c["T"]
    k, v = _all_values(c, cache, length)
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    score = q.view(S, N, H // N, D).float() @ k.transpose(2, 3) / math.sqrt(D)
    t = torch.arange(T, device="cuda")
    seen = (t < length.long()[:, None])[:, None].expand(S, N, T)
    if blocks is not None:
        hit = torch.zeros(S, blocks.shape[1], T // G + 2, dtype=torch.bool, device="cuda")
        hit.scatter_(2, torch.where(blocks >= 0, blocks, T // G + 1).long(), True)
        hit = torch.where(torch.arange(T // G + 2, device="cuda") == (length.long() // G)[:, None, None], True, hit)
        seen = seen & hit[:, :, : T // G + 1].repeat_interleave(G, dim=2)[:, :, :T]
    score = torch.where(seen[:, :, None], score, -math.inf)
    return _softmax_sum(score, v).reshape(S, H, D)


def _sees(parent):
    """[S][n][n]: which drafted tokens each one sees: itself and its line of parents."""
    n = parent.shape[1]
    up = torch.nn.functional.one_hot(parent.long().clamp(min=-1) + 1, n + 1)[..., 1:].double()
    line = torch.eye(n, dtype=torch.float64, device="cuda") + up
    for _ in range(max(1, (n - 1).bit_length())):      # twice as many steps up each time
        line = ((line @ line) > 0).double()
    return (line > 0) & (parent > -2)[..., None]


def _attend_tree(c, cache, q, parent, draft, length):
    S, N, D, H, T, n = c["S"], c["N"], c["D"], c["H"], c["T"], c["n"]
    g = H // N
    k, v = _all_values(c, cache, length)
    d = draft.view(S, n, 2, N, D).float()
    k = torch.cat([k, d[:, :, 0]], dim=1).permute(0, 2, 1, 3)
    v = torch.cat([v, d[:, :, 1]], dim=1).permute(0, 2, 1, 3)
    rows = q.view(S, n, N, g, D).float().permute(0, 2, 1, 3, 4).reshape(S, N, n * g, D)
    score = (rows @ k.transpose(2, 3) / math.sqrt(D)).view(S, N, n, g, T + n)
    old = (torch.arange(T, device="cuda") < length.long()[:, None])[:, None] & (parent > -2)[..., None]
    seen = torch.cat([old, _sees(parent)], dim=2)[:, None, :, None]
    score = torch.where(seen, score, -math.inf).view(S, N, n * g, T + n)
    out = _softmax_sum(score, v).view(S, N, n, g, D)
    return out.permute(0, 2, 1, 3, 4).reshape(S, n, H, D)


def run(state):
    c, x, cache = state["c"], state["x"], state["cache"]
    if own:
        if c["op"] == "write":
            cache.write(x["kv"], x["pos"], x["n_new"])
        if "sel" in x:
            cache.read(x["len"], x["sel"], state["k"], state["v"])
            return {"k": state["k"], "v": state["v"]}
        if c["op"] == "tree":
            cache.tree_attend(c["H"], x["q"], x["parent"], x["draft"], x["len"], state["out"])
            return {"out": state["out"]}
        if not c["sel"]:
            cache.attend(c["H"], x["q"], x["len"], state["out"])
            return {"out": state["out"]}
        cache.select(c["H"], x["q"], x["len"], state["blocks"], keep_first=1, keep_last=1)
        cache.attend(c["H"], x["q"], x["len"], state["out"], blocks=state["blocks"])
        return {"out": state["out"], "blocks": state["blocks"]}
    if c["op"] == "write":
        _write(c, cache, x["kv"], x["pos"], x["n_new"])
    if "sel" in x:
        k, v = _read(c, cache, x["len"], x["sel"])
        return {"k": k, "v": v}
    out_dt = torch.bfloat16 if c["bf16"] else torch.float32
    if c["op"] == "tree":
        return {"out": _attend_tree(c, cache, x["q"], x["parent"], x["draft"], x["len"]).to(out_dt)}
    if not c["sel"]:
        return {"out": _attend(c, cache, x["q"], x["len"], None).to(out_dt)}
    blocks = _select(c, cache, x["q"], x["len"])
    return {"out": _attend(c, cache, x["q"], x["len"], blocks).to(out_dt), "blocks": blocks}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    S, N, D, T = c["S"], c["N"], c["D"], c["T"]
    head = 4 * N * D                                   # K and V of a token in bf16
    block = N * (8 * D * c["bits"] + 8 * D)            # codes, extremes and steps of 32 tokens
    mean = (T + (S - 1) * 0.625 * T) / S               # tokens of a sequence: one full, others 1/4 .. 1
    if c["op"] == "write":
        item = 2 if c["f32"] else 1
        if c["append"]:
            back = min(c["back"], mean)
            # the row, a block's worth of rows for one sequence in 32, and what is read back
            b = S * (head * item + head + (G * head + block) / G + back * head + back / G * block)
            return {"bytes": b, "flops": 0.0}
        rows = c["n"] * (1 + (S - 1) * 2 / 3)
        return {"bytes": rows * (head * item + head + 2 * block / G) + (S * c["back"] - rows) * head, "flops": 0.0}
    if c["op"] == "read":
        n = int(c["frac"] * T) + c["last"]
        return {"bytes": S * n * (head + block / G), "flops": 0.0}
    out = 2 if c["bf16"] else 4
    if c["op"] == "tree":
        rows = S * c["n"]
        io = rows * (c["H"] * D * (2 + out) + head)
        return {"bytes": S * mean / G * block + io, "flops": 4.0 * rows * c["H"] * D * mean}
    io = S * c["H"] * D * (2 + out)
    if not c["sel"]:
        return {"bytes": S * mean / G * block + io, "flops": 4.0 * S * c["H"] * D * mean}
    nb = mean / G
    n_sel = min(c["sel"], nb)
    key = 4 * N * D                                    # a block's extremes and steps of the keys
    once = S * ((nb - n_sel) * key + n_sel * block)
    return {"bytes": once + io + S * (N if c["per_head"] else 1) * c["sel"] * 4,
            "flops": S * (4.0 * c["H"] * D * nb + 4.0 * c["H"] * D * n_sel * G)}


# ------------------------------------------------------------------ the definition in 64 bits
def _bf16_of(x):
    """Nearest value with eight significant bits, ties to even (normal range)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0) / 256.0, e)


def _held(x, dim, qmax):
    """What a group of values (64 bits, extremes over `dim`) reads as: the code counts the
    half steps that a value has passed; on a half step it goes to the even code."""
    lo = x.min(dim, keepdim=True).values
    step = _bf16_of((x.max(dim, keepdim=True).values - lo) / qmax)
    twice = 2.0 * (x - lo)
    code = torch.zeros_like(x)
    for j in range(qmax):
        border = (2 * j + 1) * step
        code += ((twice > border) if j % 2 == 0 else (twice >= border)).double()
    return _bf16_of(lo + torch.where(step > 0, code, 0.0) * step)


def _history(c, rows, length):
    """[S][T][2][N][D] in 64 bits: what a cache that holds `rows` up to `length` reads as."""
    S, T, N, D = c["S"], c["T"], c["N"], c["D"]
    x = rows.double().view(S, -1, 2, N, D)
    full = x.shape[1] // G * G
    qmax = 2 ** c["bits"] - 1
    for s in range(S):
        m = min(int(length[s]) // G * G, full)
        if m:
            b = x[s, :m].view(m // G, G, 2, N, D)
            x[s, :m, 0] = _held(b[:, :, 0], 1, qmax).reshape(m, N, D)
            x[s, :m, 1] = _held(x[s, :m, 1].unflatten(2, (D // G, G)), 3, qmax).reshape(m, N, D)
    return x


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    S, N, D, T = c["S"], c["N"], c["D"], c["T"]
    length = x["len"].tolist()
    if c["op"] == "write":
        rows = x["kv"].to(torch.bfloat16)
        if c["append"]:
            past = x["past"].clone()
            for s in range(S):
                past[s, length[s] - 1] = rows[s, 0]
            rows = past
    else:
        rows = x["past"]
    h = _history(c, rows, length)
    if "sel" in x:
        sel = x["sel"].long()
        got = torch.stack([h[s, sel[s].clamp(min=0)] for s in range(S)])
        got[sel < 0] = 0.0
        return {"k": got[:, :, 0].reshape(S, -1, N * D), "v": got[:, :, 1].reshape(S, -1, N * D)}
    g = c["H"] // N
    n = c["n"] if c["op"] == "tree" else 1
    q = x["q"].double().view(S, n, N, g, D)
    out = torch.zeros(S, n, N, g, D, dtype=torch.float64, device="cuda")
    for s in range(S):
        m = length[s]
        keys, vals = h[s, :m, 0], h[s, :m, 1]
        extra = 0
        allow = torch.ones(n, N, m, dtype=torch.bool, device="cuda")
        if c["op"] == "tree":
            d = x["draft"][s].double().view(n, 2, N, D)
            keys, vals, extra = torch.cat([keys, d[:, 0]]), torch.cat([vals, d[:, 1]]), n
            parent = x["parent"][s].tolist()
            line = torch.zeros(n, n, dtype=torch.bool)
            for j, p in enumerate(parent):
                if p >= 0:
                    line[j] = line[p]
                line[j, j] = p > -2
            allow[torch.tensor([p == -2 for p in parent], device="cuda")] = False
            allow = torch.cat([allow, line.cuda()[:, None].expand(n, N, n)], dim=2)
        elif c["sel"]:
            nb = m // G
            raw = rows[s, : nb * G, : N * D].double().view(nb, G, N, D)
            lo = raw.min(1).values
            hi = _bf16_of(lo + (2 ** c["bits"] - 1) * _bf16_of((raw.max(1).values - lo) / (2 ** c["bits"] - 1)))
            u = q[s, 0]
            bound = torch.einsum("ngd,bnd->nbg", u.clamp(min=0), hi) + torch.einsum("ngd,bnd->nbg", u.clamp(max=0), lo)
            bound = bound.amax(2) if c["per_head"] else bound.amax(2).amax(0, keepdim=True).expand(N, nb)
            for h_ in range(N):
                score = bound[h_].clone()
                if nb:
                    score[0] = score[nb - 1] = math.inf
                keep = torch.zeros(nb + 1, dtype=torch.bool, device="cuda")
                keep[score.sort(descending=True, stable=True).indices[: c["sel"]]] = True
                keep[nb] = True
                allow[0, h_] = keep.repeat_interleave(G)[:m]
        for h_ in range(N):
            z = q[s, :, h_] @ keys[:, h_].T / math.sqrt(D)
            z = torch.where(allow[:, h_][:, None].expand_as(z), z, -math.inf)
            if m + extra:
                w = torch.softmax(z, dim=-1).nan_to_num_(0.0)
                out[s, :, h_] = w @ vals[:, h_]
    out = out.reshape(S, n, c["H"], D)
    return {"out": out if c["op"] == "tree" else out[:, 0]}
