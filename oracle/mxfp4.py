"""OCP MXFP4: quantization, the expert-grouped product, and the gradients of
the combine and of the routing.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

MXFP4 has the E2M1 elements of the pages (gist.science technical summary §1)
with one power-of-two scale (E8M0) per 32 elements along a row.  All in
float64.
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_decode, e2m1_encode
from .nvfp4 import pack_codes, unpack_codes

E_MIN, E_MAX = -125, 125


def encode(x):
    """x [M][K] bf16 values as float64 -> packed codes uint8 [M][K/2], scales
    uint8 [M][K/32] (value 2^(byte - 127), 255 = NaN).  Per block of 32: the
    smallest power of two 2^E, E from -125 to 125, with max |x| <= 7 * 2^E;
    code = E2M1(x / 2^E), ties to even, saturating.  A block with a NaN or an
    infinity: byte 255, codes 7."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    E = np.full(amax.shape, E_MIN)
    while True:                                          # the definition, literally
        low = (amax > 7.0 * np.ldexp(1.0, E)) & (E < E_MAX)
        if not low.any():
            break
        E = E + low
    codes = e2m1_encode(b * np.ldexp(1.0, -E)[..., None])    # exact in float32
    codes = np.where(bad[..., None], 7, codes).astype(np.uint8)
    scales = np.where(bad, 255, E + 127).astype(np.uint8)
    return pack_codes(codes.reshape(M, K)), scales


def value(codes, scales):
    """float64 values [M][K] of packed codes [M][K/2] with scales [M][K/32]."""
    s = np.asarray(scales, dtype=np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    v = e2m1_decode(unpack_codes(np.asarray(codes)))
    return (v.reshape(s.shape + (32,)) * f[..., None]).reshape(v.shape)


def grouped_gemm(a, a_rows, w, offsets):
    """a [M_src][K], w [E][N][K] values -> y [M_total][N] float64 (not
    rounded) and the same sums over absolute values."""
    offs = np.asarray(offsets, dtype=np.int64)
    P = int(offs[-1])
    y = np.zeros((P, w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(len(offs) - 1):
        lo, hi = offs[e], offs[e + 1]
        rows = np.arange(lo, hi) if a_rows is None else np.asarray(a_rows, dtype=np.int64)[lo:hi]
        y[lo:hi] = a[rows] @ w[e].T
        mag[lo:hi] = np.abs(a[rows]) @ np.abs(w[e]).T
    return y, mag


def swiglu(y):
    """silu(gate) * up of y = [gate | up], float64, not rounded."""
    g, u = np.split(y, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def combine_backward(d_out, y, inv_perm, topk_w):
    """Gradients of out[t] = sum_j topk_w[t][j] y[inv_perm[t][j]] -> dy, d_topk_w
    (float64, not rounded)."""
    inv = np.asarray(inv_perm, dtype=np.int64)
    dy = np.zeros_like(np.asarray(y, dtype=np.float64))
    dw = np.zeros(inv.shape)
    for t in range(inv.shape[0]):
        for j in range(inv.shape[1]):
            dy[inv[t, j]] = np.float64(topk_w[t, j]) * d_out[t]
            dw[t, j] = float(np.dot(d_out[t], y[inv[t, j]]))
    return dy, dw


def permute_backward(topk_ids, topk_w, d_topk_w, E):
    """Gradient of the routing weights (softmax over the chosen experts) with
    respect to all logits [T][E] and to the bias [E], float64."""
    w, d = np.asarray(topk_w, dtype=np.float64), np.asarray(d_topk_w, dtype=np.float64)
    g = w * (d - (w * d).sum(axis=1, keepdims=True))
    out = np.zeros((w.shape[0], E))
    np.add.at(out, (np.arange(w.shape[0])[:, None], np.asarray(topk_ids, dtype=np.int64)), g)
    return out, out.sum(axis=0)
