"""fp64 restatement of the prompt's operators, from the definitions in include/rkv.h; shares no
code with the library.  Attention runs in torch float64 on whatever device its inputs are on."""
import math

import numpy as np
import torch


def theta(R, base, scaling=None):
    """Frequencies of the R/2 pairs and the gain."""
    i = np.arange(R // 2)
    th = np.power(float(base), -2.0 * i / R) if R else np.zeros(0)
    if scaling is None:
        return th, 1.0
    kind, f = scaling[0], float(scaling[1])
    if kind == "linear":
        return th / f, 1.0
    original, low, high = scaling[2:]
    if kind == "bands":
        wave = 2 * math.pi / th
        out = []
        for t, w in zip(th, wave):
            if w > original / low:
                out.append(t / f)
            elif w < original / high:
                out.append(t)
            else:
                s = (original / w - low) / (high - low)
                out.append((1 - s) * t / f + s * t)
        return np.array(out), 1.0
    turns = lambda n: R * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    a, b = max(0, math.floor(turns(low))), min(R - 1, math.ceil(turns(high)))
    w = 1 - np.clip((i - a) / max(b - a, 1e-3), 0, 1)
    return (1 - w) * th / f + w * th, (0.1 * math.log(f) + 1 if f > 1 else 1.0)


def rotate(x, pos, th, gain, layout, weight=None, eps=1e-6):
    """x float64 [rows][heads][D] -> (rotated, magnitude of what each output is made of)."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    R = 2 * len(th)
    ang = np.outer(np.asarray(pos, np.float64), th)[:, None]
    c, s = gain * np.cos(ang), gain * np.sin(ang)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if layout == "pairs" else (slice(0, R // 2), slice(R // 2, R))
    out, mag = y.copy(), np.abs(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    mag[..., a] = mag[..., b] = gain * np.hypot(y[..., a], y[..., b])
    return out, mag


def causal(q, k, v, before=0):
    """q [n][H][D], k and v [before + n][N][D] in float64 -> (out, sum of weight |v|), both [n][H][D]."""
    n, H, D = q.shape
    g = H // k.shape[1]
    late = torch.arange(before + n, device=q.device)[None] > torch.arange(before, before + n, device=q.device)[:, None]
    out, mag = torch.empty_like(q), torch.empty_like(q)
    for h in range(H):
        s = (q[:, h] @ k[:, h // g].T / math.sqrt(D)).masked_fill(late, -math.inf)
        w = torch.softmax(s, dim=-1)
        out[:, h], mag[:, h] = w @ v[:, h // g], w @ v[:, h // g].abs()
    return out, mag
