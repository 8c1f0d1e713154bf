"""The operators around the experts' products in 64 bits, from their definitions (test infrastructure only)."""

import numpy as np
import torch


def bits64(t):
    """A tensor's values as float64 on the CPU."""
    return t.detach().cpu().double()


def grid8(x):
    """float64 rows -> (their MX-FP8 values, scale bytes) from the definition; x holds no NaN or infinity."""
    b = x.reshape(*x.shape[:-1], -1, 32).numpy()
    top = np.abs(b).max(-1)
    mant, exp = np.frexp(top)                     # top = mant 2^exp, 448 = 0.875 2^9
    e = np.where(top > 0, exp - 9 + (mant > 0.875), -127).clip(-127, 127)
    y = b * np.exp2(-e.astype(np.float64))[..., None]
    quantum = np.exp2(np.maximum(np.frexp(np.abs(y))[1] - 1, -6).astype(np.float64) - 3)
    v = np.rint(y / quantum) * quantum * np.exp2(e.astype(np.float64))[..., None]
    return torch.from_numpy(v.reshape(x.shape)), torch.from_numpy((e + 127).astype(np.uint8))


def code8_values():
    """The 256 E4M3 codes' values in float64 (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    f, p = (c >> 3) & 15, c & 7
    v = np.where(f == 0, p / 8 * 2.0 ** -6, (1 + p / 8) * np.exp2(f.astype(np.float64) - 7))
    v[(c & 127) == 127] = np.nan
    return torch.from_numpy(np.where(c >= 128, -v, v))


def decode8(codes, scales):
    """uint8 codes [..., n] and scale bytes [..., >= n / 32] -> float64 values."""
    v = code8_values()[codes.cpu().long()].reshape(*codes.shape[:-1], -1, 32)
    s = scales.cpu()[..., :codes.shape[-1] // 32].double()
    unit = torch.where(s == 255, torch.nan, torch.exp2(s - 127))
    return (v * unit[..., None]).reshape(codes.shape)


def norm(x, weight, residual=None, eps=1e-6):
    """(y, s) in float64."""
    s = x if residual is None else x + residual
    return s * ((s * s).mean(-1, keepdim=True) + eps) ** -0.5 * weight, s


def norm_backward(dy, s, weight, dstream=None, eps=1e-6):
    """(dx, dweight) in float64."""
    r = ((s * s).mean(-1, keepdim=True) + eps) ** -0.5
    n, g = s * r, dy * weight
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return (dx if dstream is None else dx + dstream), (dy * n).flatten(0, -2).sum(0)


def scores(row, score):
    """float64 scores of one token's logits (a list of floats)."""
    row = np.asarray(row, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-row))
    top = row.max()
    if np.isneginf(top):
        return np.zeros_like(row)
    p = np.exp(row - top)
    return p / p.sum()


def select(logits, k, score="softmax", balance=None, groups=1, top_groups=1, group_best=2, renormalise=True, scale=1.0):
    """(idx, w) of float64 logits [T, E], one token and one comparison at a time."""
    T, E = logits.shape
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    b = np.zeros(E) if balance is None else balance.numpy()
    per = E // groups
    for t in range(T):
        row = logits[t].numpy()
        s = scores(row, score)
        rank = s + b
        rank[np.isneginf(row)] = -np.inf
        if top_groups < groups:
            best = []
            for g in range(groups):
                inside = sorted((r for r in rank[g * per:(g + 1) * per] if r > -np.inf), reverse=True)[:group_best]
                best.append(sum(inside) if inside else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    rank[g * per:(g + 1) * per] = -np.inf
        order = rank if balance is not None else np.where(np.isneginf(rank), -np.inf, row)
        picks = sorted(range(E), key=lambda e: (-order[e], e))[:k]
        chosen = np.array([0.0 if np.isneginf(rank[e]) else s[e] for e in picks])
        total = chosen.sum() if renormalise else 1.0
        idx[t], w[t] = picks, scale * (chosen / total if total > 0 else 0)
    return torch.from_numpy(idx), torch.from_numpy(w)


def select_weights(logits, idx, out, score, renormalise, scale):
    """The chosen weights as a differentiable function of float64 logits; out: picks that take no part."""
    s = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    p = s.gather(1, idx.long()).masked_fill(out, 0.0)
    return scale * (p / p.sum(1, keepdim=True).clamp(min=1e-300) if renormalise else p)


def swiglu(gate_up):
    a, b = gate_up.chunk(2, -1)
    return a * torch.sigmoid(a) * b


def swiglu_backward(dh, gate_up):
    """(dgate_up, h) in float64."""
    a, b = gate_up.chunk(2, -1)
    sg = torch.sigmoid(a)
    return torch.cat([dh * b * sg * (1 + a * (1 - sg)), dh * a * sg], -1), a * sg * b
