"""Pins of oracle/mxfp4.py: the format against exact rationals and the closed
form of its scale rule, the gradients against finite differences of the
forward."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import formats as OF
from oracle import moe as OM
from oracle import mxfp4 as OX
from oracle import nvfp4 as OQ
from tests.exact import E2M1_MAGS, e2m1_code_by_thresholds


def test_encode_matches_exact_rationals():
    rng = np.random.default_rng(0)
    x = OF.round_to_bf16(rng.standard_normal((20, 64)) * np.exp(2 * rng.standard_normal((20, 64))))
    x[3, :32] = np.arange(32) * 0.25                     # ties, and 7.75
    codes, scales = OX.encode(x)
    c = OQ.unpack_codes(codes)
    for i in range(20):
        for b in range(2):
            v = [Fraction(float(t)) for t in x[i, 32 * b:32 * b + 32]]
            top = max(abs(t) for t in v)
            E = -125
            while top > 7 * Fraction(2) ** E:
                E += 1
            assert scales[i, b] == E + 127
            for j, t in enumerate(v):
                assert c[i, 32 * b + j] == e2m1_code_by_thresholds(t / Fraction(2) ** E, t < 0)


def test_scale_rule():
    def scale_of(a):
        x = np.zeros((1, 32))
        x[0, 9] = a
        return int(OX.encode(x)[1][0, 0]) - 127
    assert scale_of(7.0) == 0 and scale_of(7.03125) == 1 and scale_of(3.5) == -1
    assert scale_of(-6.0) == 0 and scale_of(6.5) == 0 and scale_of(1.75) == -2
    assert scale_of(0.0) == -125 and scale_of(2.0 ** -133) == -125
    assert scale_of(3.3895313892515355e38) == 125
    x = np.full((1, 32), -3.3895313892515355e38)
    assert np.all(OX.value(*OX.encode(x)) == -6 * 2.0 ** 125)
    x[0, 3] = np.inf
    x = np.concatenate([x, np.full((1, 32), 2.0)], axis=1)
    v = OX.value(*OX.encode(x))
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 2).all()


def test_error_is_half_a_step_and_values_are_kept():
    rng = np.random.default_rng(1)
    x = OF.round_to_bf16(rng.standard_normal((50, 96)))
    c, s = OX.encode(x)
    y = OX.value(c, s)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    a = np.abs(x) / scale
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0)) * scale
    assert np.all(np.abs(y - x) <= half)
    assert np.array_equal(y, OF.round_to_bf16(y))
    c2, s2 = OX.encode(y)                                # values are their own quantization
    assert np.array_equal(OX.value(c2, s2), y)
    assert sorted({abs(float(t)) for t in OX.value(np.arange(16, dtype=np.uint8)[None] * 17,
                                                   np.full((1, 1), 127, np.uint8)).ravel()}) \
        == [float(m) for m in E2M1_MAGS]


def test_grouped_gemm_is_each_experts_product():
    rng = np.random.default_rng(2)
    a, w = rng.standard_normal((5, 64)), rng.standard_normal((3, 4, 64))
    rows, offs = [4, 0, 0, 2], [0, 1, 1, 4]
    y, mag = OX.grouped_gemm(a, rows, w, offs)
    for p, (t, e) in enumerate(zip(rows, (0, 2, 2, 2))):
        for n in range(4):
            assert y[p, n] == pytest.approx(sum(a[t, k] * w[e, n, k] for k in range(64)), rel=1e-12)
    assert np.all(mag >= np.abs(y))


def test_gradients_against_differences():
    """d of sum(c * combine(y, softmax of the chosen logits)) in every input."""
    rng = np.random.default_rng(3)
    T, E, tk, N = 4, 6, 3, 5
    P = T * tk
    logits, bias, y = rng.standard_normal((T, E)), rng.standard_normal(E), rng.standard_normal((P, N))
    c = rng.standard_normal((T, N))
    ids, _ = OM.route(logits.astype(np.float32), tk, bias.astype(np.float32))
    inv = rng.permutation(P).reshape(T, tk)

    def weights(lg, b):
        z = np.exp(np.take_along_axis(lg + b, ids.astype(int), axis=1))
        return z / z.sum(axis=1, keepdims=True)

    def loss(lg, b, yy):
        w = weights(lg, b)
        return sum(float(c[t] @ (w[t, j] * yy[inv[t, j]])) for t in range(T) for j in range(tk))

    w = weights(logits, bias)
    dy, dw = OX.combine_backward(c, y, inv, w)
    dl, db = OX.permute_backward(ids, w, dw, E)
    h = 1e-6
    for arr, grad in ((logits, dl), (bias, db), (y, dy)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss(logits, bias, y)
            arr[i] = keep - h
            down = loss(logits, bias, y)
            arr[i] = keep
            # truncation h^2, cancellation 1e-16 / h
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-8
