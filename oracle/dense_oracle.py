"""Plain fp64 forms of the dense operators: 8-bit row quantisation, the integer product, the
gated block with its gradient, and error bounds for the library's arithmetic.

The bounds are worst cases of the documented arithmetic, evaluated on the data: products of
n terms accumulate in fp32 in any order (n * 2^-24 * sum |term|), and each stored intermediate
or result is off by half a step of its type (``half``: 2^-24 for fp32, 2^-8 for bf16).
"""
from __future__ import annotations

import numpy as np

F32_HALF = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
KEPT = {"f32": 0.0, "bf16": 2.0 ** -15}          # pre-activations: fp32 cut after 15 fraction bits
# exp, the reciprocal and the products of the sigmoid: a few steps each, and the argument's own
# rounding times its size (|z| <= 88 before the result is 0 or 1)
SIGMOID_REL = 2.0 ** -17


def quantize_rows(x):
    """(codes, scales): scale = fp32(max|row| / 127), codes = row / scale, half to even, on the
    exact quotient (two fp32 numbers' quotient is at least 2^-33 from a half-way point it does
    not equal, so fp64 decides it)."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(axis=1)
    bad = ~np.isfinite(top)
    with np.errstate(over="ignore"):
        s = (np.where(bad, 0.0, top) / 127.0).astype(np.float32)
    s[s < np.float32(2.0 ** -126)] = 0
    s64 = s.astype(np.float64)
    safe = np.where(s64 > 0, s64, 1.0)[:, None]
    q = np.where((s64 > 0)[:, None] & ~bad[:, None], np.rint(np.where(bad[:, None], 0.0, x) / safe), 0.0)
    s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
    return q.astype(np.int8), s


def i8_matmul(xq, xs, wq, ws):
    """fp64 value of x_scale * w_scale * integer sum."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T          # exact: below 2^53
    return acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]


def i8_bound(ref, y_type):
    """The sum's conversion and two multiplications in fp32, then one rounding to y_type."""
    return np.abs(ref) * (3.01 * F32_HALF + (HALF["bf16"] if y_type == "bf16" else 0.0)) + 1e-45


def interleave(g, u):
    """Gate and up rows [I][H] as the blob's [2I][H]."""
    I, H = g.shape
    return np.stack([g.reshape(I // 16, 16, H), u.reshape(I // 16, 16, H)], 1).reshape(2 * I, H)


def deinterleave(gu):
    """Rows of [2I][H] to (gate [I][H], up [I][H])."""
    H = gu.shape[1]
    v = gu.reshape(-1, 2, 16, H)
    return v[:, 0].reshape(-1, H), v[:, 1].reshape(-1, H)


def sigmoid(z):
    """1 / (1 + e^-z), through e^-|z|: nothing cancels or overflows at either end."""
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def block(x, wg, wu, wd):
    """y, and the pieces the backward pass uses."""
    g, u = x @ wg.T, x @ wu.T
    a = g * sigmoid(g)
    h = a * u
    return h @ wd.T, (g, u, a, h)


def block_backward(dy, x, wg, wu, wd):
    """dx, dWg, dWu, dWd in fp64."""
    _, (g, u, a, h) = block(x, wg, wu, wd)
    s = sigmoid(g)
    dh = dy @ wd
    dg, du = dh * u * (s + g * s * (1 - s)), dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h


def _gamma(n):
    return n * F32_HALF * 1.01


def block_bounds(dy, x, wg, wu, wd, dtype, exact=False):
    """Elementwise bounds of the library's y, dx, dWg, dWu, dWd (dy None: y's only).  exact: every
    pre-activation is one product that its type holds whole (no error, and kept as it is)."""
    half = HALF[dtype]
    H, I, T = x.shape[1], wg.shape[0], x.shape[0]
    y, (g, u, a, h) = block(x, wg, wu, wd)
    ax, awd = np.abs(x), np.abs(wd)
    eg, eu = _gamma(H) * (ax @ np.abs(wg).T), _gamma(H) * (ax @ np.abs(wu).T)
    if exact:
        eg, eu = np.zeros_like(eg), np.zeros_like(eu)
    ag, au, aa, ah = np.abs(g), np.abs(u), np.abs(a), np.abs(h)
    # silu' lies in (-0.1, 1.1)
    eh = (aa * (1 + SIGMOID_REL) + 1.1 * eg) * (au + eu) - aa * au
    eh = eh + (ah + eh) * (half + 2 * F32_HALF)
    by = eh @ awd.T + _gamma(I) * ((ah + eh) @ awd.T)
    out = {"y": by + (np.abs(y) + by) * half}
    if dy is None:
        return out
    ady = np.abs(dy)
    s = sigmoid(g)
    sp = s + g * s * (1 - s)
    dh = dy @ wd
    adh, ed = np.abs(dh), _gamma(H) * (ady @ awd)
    kept = 0.0 if exact else KEPT[dtype]
    egs, eus = eg + (ag + eg) * kept, eu + (au + eu) * kept             # as saved
    asp = np.abs(sp)
    # silu'' lies in (-0.1, 0.5]; silu' is a sum of terms of size s and s |g|
    esp = 0.5 * egs + SIGMOID_REL * (s + (ag + egs) * s)
    edg = (adh + ed) * (au + eus) * (asp + esp) - adh * au * asp
    edu = (adh + ed) * (aa * (1 + SIGMOID_REL) + 1.1 * egs) - adh * aa
    dg, du = dh * u * sp, dh * a
    edg = edg + (np.abs(dg) + edg) * (half + 4 * F32_HALF)
    edu = edu + (np.abs(du) + edu) * (half + 4 * F32_HALF)
    mg, mu = np.abs(dg) + edg, np.abs(du) + edu
    dx, dwg, dwu, dwd = block_backward(dy, x, wg, wu, wd)

    def fin(e, v):
        return e + (np.abs(v) + e) * half

    out["dx"] = fin(edg @ np.abs(wg) + edu @ np.abs(wu) + _gamma(2 * I) * (mg @ np.abs(wg) + mu @ np.abs(wu)), dx)
    out["dwg"] = fin(edg.T @ ax + _gamma(T) * (mg.T @ ax), dwg)
    out["dwu"] = fin(edu.T @ ax + _gamma(T) * (mu.T @ ax), dwu)
    out["dwd"] = fin(ady.T @ eh + _gamma(T) * (ady.T @ (ah + eh)), dwd)
    return out


def i8_block(x, wgq, wgs, wuq, wus, wdq, wds):
    """The 8-bit block in fp64 (scales fp32, codes whole)."""
    xq, xs = quantize_rows(x)
    g, u = i8_matmul(xq, xs, wgq, wgs), i8_matmul(xq, xs, wuq, wus)
    h = g * sigmoid(g) * u
    hq, hs = quantize_rows(h)
    return i8_matmul(hq, hs, wdq, wds), (h, hs)
