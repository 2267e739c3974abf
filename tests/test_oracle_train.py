"""Pins of oracle/train.py: the checkpoint format against torch's E4M3 cast and
its own definition, the gradients against finite differences of the forward."""
import numpy as np
import pytest
import torch

from oracle import formats as OF
from oracle import moe as OM
from oracle import nvfp4 as OQ
from oracle import train as OT


def test_mxfp8_matches_torch_cast_and_keeps_half_a_step():
    rng = np.random.default_rng(0)
    x = OF.round_to_bf16(rng.standard_normal((40, 96)) * np.exp(2 * rng.standard_normal((40, 96))))
    codes, scales = OT.mxfp8_encode(x)
    s = np.ldexp(1.0, scales.astype(int) - 127)
    v = torch.from_numpy((x.reshape(40, 3, 32) / s[..., None]).astype(np.float32))
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(40, 96)
    assert np.array_equal(codes, want)
    y = OT.mxfp8_value(codes, scales)
    # half a step relative (2^-4 of the value), or half the smallest step
    lim = np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s, 32, axis=1) * 2.0 ** -10)
    assert np.all(np.abs(y - x) <= lim)
    # a restored checkpoint's values are bf16, and their own checkpoint
    assert np.array_equal(y, OF.round_to_bf16(y))
    c2, s2 = OT.mxfp8_encode(y)
    assert np.array_equal(OT.mxfp8_value(c2, s2), y)


def test_mxfp8_scale_rule():
    def scale_of(a):
        x = np.zeros((1, 32))
        x[0, 5] = a
        return int(OT.mxfp8_encode(x)[1][0, 0]) - 127
    assert scale_of(448.0) == 0 and scale_of(450.0) == 1 and scale_of(224.0) == -1
    assert scale_of(1.75) == -8 and scale_of(-1.7578125) == -7
    assert scale_of(0.0) == -117 and scale_of(2.0 ** -133) == -117
    assert scale_of(3.3895313892515355e38) == 120
    big = np.full((1, 32), -3.3895313892515355e38)       # 255 * 2^120: 240, not 256
    assert np.all(OT.mxfp8_value(*OT.mxfp8_encode(big)) == -240.0 * 2.0 ** 120)
    x = np.zeros((1, 64))
    x[0, 3], x[0, 4], x[0, 40] = np.inf, 448.0, np.nan
    codes, scales = OT.mxfp8_encode(x)
    assert codes[0, 3] == 0x7F and codes[0, 4] == 0x7E and codes[0, 40] == 0x7F
    assert list(scales[0]) == [127, 10]


def _forward(y, inv, w):
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    h = g / (1 + np.exp(-g)) * u
    return h


def test_swiglu_backward_against_differences():
    rng = np.random.default_rng(1)
    T, tk, I = 5, 3, 4
    P = T * tk
    inv = rng.permutation(P).reshape(T, tk)
    w = rng.random((T, tk))
    y = rng.standard_normal((P, 2 * I)) * 3
    a = rng.standard_normal((P, I))                       # dL/d(w h)

    def loss(y, w):
        wr = np.empty(P)
        wr[inv.reshape(-1)] = w.reshape(-1)
        return float((a * wr[:, None] * _forward(y, inv, w)).sum())

    dy, hw, dw = OT.swiglu_backward(y, a, inv, w)
    eps = 1e-6
    for p in range(P):
        for c in range(2 * I):
            d = np.zeros_like(y)
            d[p, c] = eps
            num = (loss(y + d, w) - loss(y - d, w)) / (2 * eps)
            assert abs(num - dy[p, c]) < 1e-6
    for t in range(T):
        for j in range(tk):
            d = np.zeros_like(w)
            d[t, j] = eps
            num = (loss(y, w + d) - loss(y, w - d)) / (2 * eps)
            assert abs(num - dw[t, j]) < 1e-6
    wr = np.empty(P)
    wr[inv.reshape(-1)] = w.reshape(-1)
    assert np.allclose(hw, wr[:, None] * _forward(y, inv, w), rtol=1e-14)


def test_block_gradients_against_differences():
    """The chain of the four operators is the derivative of the whole block
    (products without their bf16 roundings) for x, both weights and the
    routing weights through the softmax."""
    rng = np.random.default_rng(2)
    T, H, E, tk, I = 6, 16, 3, 2, 16
    x = rng.standard_normal((T, H))
    w1c, w1s, w1g, _ = OQ.qdq_weights(OF.round_to_bf16(rng.standard_normal((E, 2 * I, H)) * 0.3))
    w2c, w2s, w2g, _ = OQ.qdq_weights(OF.round_to_bf16(rng.standard_normal((E, H, I)) * 0.3))
    W1 = np.stack([OQ.dequantize_unscaled(w1c[e], w1s[e]) * np.float64(w1g[e]) for e in range(E)])
    W2 = np.stack([OQ.dequantize_unscaled(w2c[e], w2s[e]) * np.float64(w2g[e]) for e in range(E)])
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids, _ = OM.route(logits, tk)
    offs, perm, inv = OM.permute(ids, E)
    a = rng.standard_normal((T, H))
    expert = np.searchsorted(offs, np.arange(T * tk), side="right") - 1

    def weights(lg):
        z = np.exp(np.take_along_axis(lg, ids.astype(np.int64), 1))
        return z / z.sum(1, keepdims=True)

    def loss(x, W1, W2, lg):
        w = weights(lg)
        total = 0.0
        for t in range(T):
            for j in range(tk):
                e = expert[inv[t, j]]
                y = W1[e] @ x[t]
                h = y[:I] / (1 + np.exp(-y[:I])) * y[I:]
                total += w[t, j] * float(a[t] @ (W2[e] @ h))
        return total

    lg = logits.astype(np.float64)
    w = weights(lg)
    y1 = np.stack([W1[expert[p]] @ x[perm[p]] for p in range(T * tk)])
    dh, _ = OT.grouped_dgrad(a, perm, w2c, w2s, w2g, offs)
    dy1, hw, dtw = OT.swiglu_backward(y1, dh, inv, w)
    dw2, _ = OT.grouped_wgrad(a, perm, hw, None, offs)
    dw1, _ = OT.grouped_wgrad(dy1, None, x, perm, offs)
    dxp, _ = OT.grouped_dgrad(dy1, None, w1c, w1s, w1g, offs)
    dx = dxp[inv].sum(axis=1)
    dl = OT.route_backward(w, dtw)
    eps = 1e-6
    for arr, grad, name in [(x, dx, "x"), (W1, dw1, "W1"), (W2, dw2, "W2")]:
        for _ in range(60):
            i = tuple(rng.integers(0, n) for n in arr.shape)
            keep = arr[i]
            arr[i] = keep + eps
            up = loss(x, W1, W2, lg)
            arr[i] = keep - eps
            down = loss(x, W1, W2, lg)
            arr[i] = keep
            assert abs((up - down) / (2 * eps) - grad[i]) < 1e-5, name
    for t in range(T):
        for j in range(tk):
            d = np.zeros_like(lg)
            d[t, ids[t, j]] = eps
            num = (loss(x, W1, W2, lg + d) - loss(x, W1, W2, lg - d)) / (2 * eps)
            assert abs(num - dl[t, j]) < 1e-5


def test_grouped_gradients_by_hand():
    offs = np.array([0, 2, 2, 3])
    dy = np.array([[1.0, 2.0], [3.0, 4.0]])
    x = np.array([[5.0], [7.0], [11.0]])
    dw, mag = OT.grouped_wgrad(-dy, np.array([1, 0, 1]), x, None, offs)
    assert np.array_equal(dw, -mag)
    assert dw[0].tolist() == [[-(3 * 5 + 1 * 7)], [-(4 * 5 + 2 * 7)]]
    assert not dw[1].any()
    assert dw[2].tolist() == [[-33.0], [-44.0]]


@pytest.mark.parametrize("w,d", [([[0.25, 0.75]], [[1.0, 3.0]])])
def test_route_backward_by_hand(w, d):
    # sum w d = 2.5: [0.25 (1 - 2.5), 0.75 (3 - 2.5)]
    assert np.allclose(OT.route_backward(w, d), [[-0.375, 0.375]])
