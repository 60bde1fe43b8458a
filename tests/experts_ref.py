"""Plain 64-bit implementations of the router's and the experts' operators on the CPU, for the tests."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # unit roundoffs
BLOCK = 128


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


def power(e):
    """2^e exactly."""
    return torch.from_numpy(np.ldexp(1.0, e.numpy().astype(np.int64)))


def quantised(x, rows=1, cols=BLOCK):
    """What x stands for in blocks of rows x cols: e4m3 with the smallest power of two 2^e, e >= -126, that brings a block to
    at most 448; NaN for a block with an infinity or a NaN."""
    x = f64(x)
    M, K = x.shape
    v = torch.zeros((-(-M // rows) * rows, -(-K // cols) * cols), dtype=torch.float64)
    v[:M, :K] = x
    v = v.view(v.shape[0] // rows, rows, v.shape[1] // cols, cols)
    top = v.abs().amax((1, 3), keepdim=True)
    bad = ~torch.isfinite(top)
    m, e = torch.frexp(torch.where(bad, torch.ones_like(top), top))  # top = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 448 / 512, e - 9, e - 8).clamp(min=-126)
    e = torch.where(top == 0, torch.full_like(e, -126), e)
    u = v * power(-e)
    _, lead = torch.frexp(u)
    step = power((lead - 1).clamp(min=-6) - 3)
    out = torch.round(u / step) * step * power(e)
    out = torch.where(bad.expand_as(out), torch.full_like(out, float("nan")), out)
    return out.reshape(out.shape[0] * rows, -1)[:M, :K].contiguous()


def product(x, w):
    """(x w^T, |x| |w|^T, sum over eights of inputs of the largest product)."""
    top = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64)
    for k in range(0, x.shape[1], 8):
        top += (x[:, None, k:k + 8] * w[None, :, k:k + 8]).abs().amax(2)
    return x @ w.t(), x.abs() @ w.abs().t(), top


def plan(experts, E):
    """(offsets, tokens, slots) of choices [T][k]."""
    ids = experts.cpu().numpy()
    T, k = ids.shape
    flat = ids.reshape(-1)
    slots = np.full(T * k, -1, np.int32)
    tokens = np.full(T * k, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    n = 0
    for e in range(E):
        for i in np.flatnonzero(flat == e):
            slots[i] = n
            tokens[n] = i // k
            n += 1
        offsets[e + 1] = n
    return torch.from_numpy(offsets), torch.from_numpy(tokens), torch.from_numpy(slots.reshape(T, k))


def scores(logits, score):
    l = f64(logits).numpy()
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
            return np.where(np.isneginf(l), 0.0, s)
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def route(logits, k, score, bias, groups, keep, renormalise, scale):
    """(weights, experts); a plain loop over the tokens."""
    l = f64(logits).numpy()
    T, E = l.shape
    s = scores(logits, score)
    c = s + (0.0 if bias is None else f64(bias).numpy())
    if bias is None and groups == 1:
        c = l  # scores order as the logits do
    experts, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    size = E // groups
    for t in range(T):
        on = ~np.isneginf(l[t])
        key = np.where(np.isnan(c[t]), -1e300, c[t])
        allowed = on.copy()
        if groups > 1:
            total = np.full(groups, -np.inf)
            for g in range(groups):
                best = sorted((key[e] for e in range(g * size, (g + 1) * size) if on[e]), reverse=True)[:2]
                if best:
                    total[g] = sum(best)
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:keep]
            allowed &= np.isin(np.arange(E) // size, kept)
        order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-key[e], e))[:k]
        experts[t, :len(order)] = order
        w = s[t, order]
        with np.errstate(all="ignore"):
            weights[t, :len(order)] = scale * (w / (w.sum() + 1e-20) if renormalise else w)
    return torch.from_numpy(weights), torch.from_numpy(experts)


def route_weights(l, experts, score, renormalise, scale):
    """weights [T][k] as a function of 64-bit logits for given choices (torch, for autograd and differences)."""
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    e = experts.long()
    w = torch.where(e >= 0, s.gather(1, e.clamp(min=0)), torch.zeros((), dtype=s.dtype))
    return scale * (w / (w.sum(1, keepdim=True) + 1e-20) if renormalise else w)
