"""The training step around the W4A16 product: 8-bit activation checkpoints,
the gradients of the product and of the SwiGLU with its routing weights.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

The pages describe the trainer's forward only (asymmetric W4A16 QAT,
gist.science technical summary §2.2 A).  Everything here is the plain
derivative of that forward, with the straight-through gradient for the
weights, in float64.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_MAX, e4m3_decode, e4m3_encode_nonneg
from .nvfp4 import dequantize_unscaled


def mxfp8_encode(x):
    """x [M][K] bf16 values as float64 -> codes uint8 [M][K], scales uint8
    [M][K/32] (E8M0, value 2^(byte - 127)).  Per block of 32: the smallest
    power of two 2^E, E >= -117, with the largest finite |x| <= 448 * 2^E;
    code = E4M3(x / 2^E), round to nearest even, but 240 where 256 * 2^120 =
    2^128 would be next (bf16 does not hold it); NaN and infinities: 0x7F with
    x's sign bit."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    fin = np.isfinite(b)
    a = np.where(fin, np.abs(b), 0.0)
    amax = a.max(axis=2)
    E = np.full(amax.shape, -117)
    while True:                                          # the definition, literally
        low = amax > E4M3_MAX * np.ldexp(1.0, E)
        if not low.any():
            break
        E = E + low
    v = a * np.ldexp(1.0, -E)[..., None]                 # exact in float32
    v = np.where((E == 120)[..., None], np.minimum(v, 240.0), v)
    codes = np.where(fin, e4m3_encode_nonneg(v), 0x7F).astype(np.uint8)
    codes |= np.signbit(b).astype(np.uint8) << 7
    return codes.reshape(M, K), (E + 127).astype(np.uint8)


def mxfp8_value(codes, scales):
    """float64 values of codes [M][K] with scales [M][K/32]."""
    M, K = codes.shape
    s = np.ldexp(1.0, np.asarray(scales, dtype=np.int64) - 127)
    return (e4m3_decode(codes).reshape(M, K // 32, 32) * s[..., None]).reshape(M, K)


def _pick(rows, lo, hi):
    return np.arange(lo, hi) if rows is None else np.asarray(rows, dtype=np.int64)[lo:hi]


def grouped_dgrad(dy, dy_rows, w_codes, w_scales, g_w, offsets):
    """dx[p] = g_w[e] * dy[t_p] @ w~e, [M_total][K] float64 (not rounded), and
    the same sum over absolute values (the scale of its rounding errors)."""
    offs = np.asarray(offsets, dtype=np.int64)
    dy = np.asarray(dy, dtype=np.float64)
    out = np.zeros((int(offs[-1]), w_codes.shape[2]))
    mag = np.zeros_like(out)
    for e in range(len(offs) - 1):
        lo, hi = offs[e], offs[e + 1]
        if lo == hi:
            continue
        w = dequantize_unscaled(w_codes[e], w_scales[e]) * np.float64(g_w[e])
        d = dy[_pick(dy_rows, lo, hi)]
        out[lo:hi] = d @ w
        mag[lo:hi] = np.abs(d) @ np.abs(w)
    return out, mag


def grouped_wgrad(dy, dy_rows, x, x_rows, offsets):
    """dw[e] = dy_e^T x_e over the expert's rows, [E][N][K] float64, and the
    same sum over absolute values."""
    offs = np.asarray(offsets, dtype=np.int64)
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    E = len(offs) - 1
    out = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(out)
    for e in range(E):
        d, v = dy[_pick(dy_rows, offs[e], offs[e + 1])], x[_pick(x_rows, offs[e], offs[e + 1])]
        out[e] = d.T @ v
        mag[e] = np.abs(d).T @ np.abs(v)
    return out, mag


def swiglu_backward(y, dh, inv_perm, topk_w):
    """y [P][2I] = [gate | up], dh [P][I], inv_perm [T][tk] or None (slot t is
    row t), topk_w [T][tk] or None (ones) -> dy [P][2I], hw [P][I], d_topk_w
    [T][tk], float64, not rounded.  h = silu(gate) up, row p of slot (t, j)
    enters the output with weight topk_w[t][j], dh is the gradient of
    topk_w[t][j] * h divided by the weight."""
    y, dh = np.asarray(y, dtype=np.float64), np.asarray(dh, dtype=np.float64)
    P, I = dh.shape
    inv = np.arange(P)[:, None] if inv_perm is None else np.asarray(inv_perm, dtype=np.int64)
    w = np.ones(P)
    if topk_w is not None:
        w[inv.reshape(-1)] = np.asarray(topk_w, dtype=np.float64).reshape(-1)
    g, u = y[:, :I], y[:, I:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        t = 1.0 / (1.0 + np.exp(g))                      # 1 - s
    h = g * s * u
    d = w[:, None] * dh
    dy = np.concatenate([d * u * s * (1.0 + g * t), d * g * s], axis=1)
    return dy, w[:, None] * h, (dh * h).sum(axis=1)[inv]


def route_backward(topk_w, d_topk_w):
    """Gradient of the chosen logits of a softmax over the tk chosen experts."""
    w, d = np.asarray(topk_w, dtype=np.float64), np.asarray(d_topk_w, dtype=np.float64)
    return w * (d - (w * d).sum(axis=1, keepdims=True))
