"""Plain fp64 forms of the operators on 4-bit weights: quantisation of rows, the weights that codes
stand for, products and experts, and error bounds for the library's arithmetic.

The bounds are worst cases of the documented arithmetic, evaluated on the data: sums of n products in
fp32 in any order are off by n * 2^-24 * sum |term|.  A kernel may sum x * code and take z * sum x off
again, so a term counts as |x| * s * (code + z).
"""
from __future__ import annotations

import numpy as np

from .dense_oracle import F32_HALF, HALF, SIGMOID_REL, sigmoid


def e4m3_values():
    """The numbers of the e4m3 bytes 0..0x7E."""
    b = np.arange(0x7F)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = e4m3_values()


def e4m3_byte(v, up):
    """Bytes of nonnegative numbers: nearest (ties to the even byte) or the least not below."""
    v = np.asarray(v, np.float64)
    hi = np.minimum(np.searchsorted(E4M3, v), 0x7E)
    if up:
        return hi
    lo = np.maximum(hi - 1, 0)
    below, above = v - E4M3[lo], E4M3[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantize(x, group, zero):
    """(codes [N][K], words [N][groups], exps [N]) of rows of fp32 numbers."""
    x = np.asarray(x, np.float64)
    N, K = x.shape
    n = -(-K // group)
    codes, words, exps = np.full((N, K), 8, np.uint8), np.zeros((N, n), np.uint16), np.zeros(N, np.uint8)
    words[:] = 8 << 8
    for r in range(N):
        v = x[r]
        if not (np.abs(v) < 2.0 ** 120).all():
            exps[r] = 255
            continue
        parts = [v[g * group:(g + 1) * group] for g in range(n)]
        lo = np.array([min(p.min(), 0.0) for p in parts])
        hi = np.array([max(p.max(), 0.0) for p in parts])
        t = (hi - lo) / 15.0 if zero else np.maximum(hi, -lo) / 7.0
        if t.max() == 0:
            continue
        m, e = np.frexp(t.max() / 448.0)
        e = int(e) - (m == 0.5)
        if e < -100:
            continue
        S = 2.0 ** e
        exps[r] = e + 127
        s = e4m3_byte(t / S, zero)
        for g, p in enumerate(parts):
            d = S * E4M3[s[g]]
            if d == 0:
                continue
            z = int(min(np.rint(-lo[g] / d), 15)) if zero else 8
            words[r, g] = s[g] | z << 8
            codes[r, g * group:(g + 1) * group] = np.clip(np.rint(p / d) + z, 0, 15)
    return codes, words, exps


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)


def lay_words(words):
    """Words [N][groups] as the library holds them: by runs of 16 rows, in each group by group."""
    return np.concatenate([words[r:r + 16].T.ravel() for r in range(0, len(words), 16)])


def unlay_words(flat, N, groups):
    return np.concatenate([flat[r * groups:min(r + 16, N) * groups].reshape(groups, -1).T for r in range(0, N, 16)])


def scales(words, exps, group, K):
    """(s * S spread over K, z spread over K)."""
    s = np.where(words & 0x80, -1.0, 1.0) * np.concatenate([E4M3, [np.nan]])[words & 0x7F]
    S = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    at = np.arange(K) // group
    return s[:, at] * S[:, None], (words >> 8).astype(np.float64)[:, at]


def weights(codes, words, exps, group):
    s, z = scales(words, exps, group, codes.shape[1])
    return s * (codes - z)


def sizes(codes, words, exps, group):
    """What a weight may count as in a sum: s * (code + z)."""
    s, z = scales(words, exps, group, codes.shape[1])
    return np.abs(s) * (codes + z)


def gamma(n):
    return n * F32_HALF * 1.01


def matmul_bound(x, codes, words, exps, group, y_type, parts=1):
    """Elementwise bound of x . weights^T: the sums (64: z * sum x and the scales of a run), one rounding."""
    x = np.asarray(x, np.float64)
    e = gamma(x.shape[1] * parts + 64) * (np.abs(x) @ sizes(codes, words, exps, group).T)
    ref = x @ weights(codes, words, exps, group).T
    return ref, e + (np.abs(ref) + e) * HALF[y_type] + 2.0 ** -133


def expert_bound(x, gate, up, down, group):
    """(o, bound) of tokens x through an expert whose three parts are (codes, words, exps)."""
    x = np.asarray(x, np.float64)
    H, I = x.shape[1], gate[0].shape[0]
    wg, wu, wd = (weights(*p, group) for p in (gate, up, down))
    bg, bu, bd = (sizes(*p, group) for p in (gate, up, down))
    g, u = x @ wg.T, x @ wu.T
    eg, eu = gamma(H + 64) * (np.abs(x) @ bg.T), gamma(H + 64) * (np.abs(x) @ bu.T)
    a = g * sigmoid(g)
    h = a * u
    # silu' lies in (-0.1, 1.1)
    eh = (np.abs(a) * (1 + SIGMOID_REL) + 1.1 * eg) * (np.abs(u) + eu) - np.abs(h)
    eh = eh + (np.abs(h) + eh) * (HALF["bf16"] + 2 * F32_HALF)
    o = h @ wd.T
    e = eh @ np.abs(wd).T + gamma(I + 64) * ((np.abs(h) + eh) @ bd.T)
    return o, e + (np.abs(o) + e) * HALF["bf16"] + 2.0 ** -133
