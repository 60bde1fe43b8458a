"""Plain 64-bit implementations of the layer operators on the CPU (numpy), for the tests.

Beside each result they give a magnitude: the same formula with every term taken
absolutely.  An FP32 evaluation with c roundings on any path from an input to an
output differs by at most about c 2^-24 times it, whatever cancels.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # unit roundoffs


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def w4_weights(q, scales, zeros, group):
    """(w, |terms|): dequantised weights, and scale (32 + q + z), the sum of the magnitudes the kernel adds."""
    qb = q.cpu().numpy()
    N, half = qb.shape
    K = 2 * half
    v = np.empty((N, K))
    v[:, 0::2], v[:, 1::2] = qb & 15, qb >> 4
    rep = np.minimum(np.arange(K) // group, scales.shape[1] - 1)
    s = f64(scales)[:, rep]
    z = np.full((N, K), 8.0) if zeros is None else zeros.cpu().numpy().astype(np.float64)[:, rep]
    return s * (v - z), np.abs(s) * (32 + v + z)


def block_norm(parts, residual, pre, post, gate, a, b, eps):
    """parts [P][S][N]; returns dict of (value, magnitude) for y, h, z and rstd [2][S]."""
    parts, residual, pre, post, gate = (f64(t) for t in (parts, residual, pre, post, gate))
    y, ym = parts.sum(0), np.abs(parts).sum(0)
    with np.errstate(all="ignore"):
        ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if post is not None else np.ones((y.shape[0], 1))
        u = y * ry * (post if post is not None else 1.0)
        um = ym * ry * (np.abs(post) if post is not None else 1.0)
        g = gate if gate is not None else 1.0
        h = a * g * u
        hm = np.abs(a * g) * um
        if residual is not None:
            h = h + b * residual
            hm = hm + np.abs(b * residual)
        rh = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        out = {"y": (y, ym), "h": (h, hm)}
        if pre is not None:
            out["z"] = (h * rh * pre, hm * rh * np.abs(pre))
        else:
            rh = np.zeros_like(rh)
    out["rstd"] = np.stack([ry[:, 0], rh[:, 0]])
    return out


def block_norm_backward(dz, dh, h, y, rstd, pre, post, gate, a, b):
    """dict of (value, magnitude) for residual, y, pre_weight, post_weight, gate."""
    kind = None if gate is None else "channel" if gate.dim() == 1 else "token" if gate.shape[1] == 1 and y.shape[1] != 1 else "full"
    dz, dh, h, y, rstd, pre, post, gate = (f64(t) for t in (dz, dh, h, y, rstd, pre, post, gate))
    S, N = (dz if dz is not None else y).shape
    A = np.abs
    d = dh if dh is not None else np.zeros((S, N))
    m = A(d)
    out = {}

    def through(d, m, t, w, r):
        hat, wd, wm = t * r, w * d, A(w) * m
        dot, dotm = (wd * hat).mean(1, keepdims=True), (wm * A(hat)).mean(1, keepdims=True)
        return r * (wd - hat * dot), r * (wm + A(hat) * dotm), (d * hat).sum(0), (m * A(hat)).sum(0)

    if pre is not None:
        v, vm, w, wm = through(dz, A(dz), h, pre, rstd[1][:, None])
        d, m = d + v, m + vm
        out["pre_weight"] = (w, wm)
    out["residual"] = (b * d, A(b) * m)
    d, m = a * d, A(a) * m
    ry = rstd[0][:, None] if post is not None else 1.0
    if gate is not None:
        u = y * ry * (post if post is not None else 1.0)
        dg, dgm = d * u, m * A(u)
        if kind == "channel":
            dg, dgm = dg.sum(0), dgm.sum(0)
        elif kind == "token":
            dg, dgm = dg.sum(1, keepdims=True), dgm.sum(1, keepdims=True)
        out["gate"] = (dg, dgm)
        d, m = d * gate, m * A(gate)
    if post is not None:
        d, m, w, wm = through(d, m, y, post, ry)
        out["post_weight"] = (w, wm)
    out["y"] = (d, m)
    return out


def ckpt_pack(x):
    """(q int8 [M][Kp], exps int8 [M][Kp/32]) of a float tensor, from integers and exponent bits only."""
    v = x.detach().cpu().to(torch.float64).numpy()
    M, K = v.shape
    blocks = -(-K // 32)
    p = np.zeros((M, blocks * 32))
    p[:, :K] = v
    p = p.reshape(M, blocks, 32)
    bad = ~np.isfinite(p).all(-1)
    p[bad] = 0
    top = np.abs(p).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 6, -126)  # frexp: top = f 2^k, 0.5 <= f < 1
    e = np.maximum(e, -126)
    q = np.clip(np.rint(np.ldexp(p, -e[..., None])), -127, 127)
    e[bad] = 127
    return q.astype(np.int8).reshape(M, -1), e.astype(np.int8)


def ckpt_value(q, e, K):
    M = q.shape[0]
    v = np.ldexp(q.reshape(M, -1, 32).astype(np.float64), e.astype(np.int64)[..., None])
    v[e == 127] = np.nan
    return v.reshape(M, -1)[:, :K]


def assert_close(got, want, mag, roundings, what=""):
    """|got - want| <= unit roundoff of the output type + `roundings` FP32 roundings of the magnitude."""
    g = got.detach().cpu().to(torch.float64).numpy()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in other places"
    tiny = torch.finfo(got.dtype).tiny
    bound = UNIT[got.dtype] * np.abs(want) + (1 + UNIT[got.dtype]) * roundings * U32 * mag + tiny
    bad = ~nan & (np.abs(g - want) > bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / bound, 0)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} beyond the bound; at {i} got {g[i]!r}, want {want[i]!r}, "
                             f"bound {bound[i]:.3g}")
