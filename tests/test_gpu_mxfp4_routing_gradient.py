"""The training step's gradient of the routing weights where the state keeps the
down projection's output (keep_y2): that of the output which the forward
returned, against the float64 oracle and against differences.

d_topk_w[t][j] = <d_out[t], y2[row of (t, j)]>: H products in float32, each added
with one rounding of at most U = 2^-24 of what is held, which is at most the sum
of magnitudes: H U of it."""
import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from oracle import mxfp4 as OX
from tests.gpu_util import host_vals
from tests.test_gpu_mxfp4 import check
from tests.test_gpu_mxfp4_block import BLOCKS, U, block, cu, dev_vals, same, say

pytestmark = pytest.mark.gpu


def prepared(fmt, w):
    w = dev_vals(w)
    return pipeline.prepare_mxfp4_weights(w, want_transposed=True) if fmt == "mxfp4" else pipeline.prepare_weights(w)


@pytest.mark.parametrize("T,H,E,tk,I,with_bias", BLOCKS)
@pytest.mark.parametrize("fmt,ckpt", [("mxfp4", "bf16"), ("mxfp4", "mxfp8"), ("w4a16", "mxfp8")])
def test_gradient_of_the_output_that_was_returned(dev, T, H, E, tk, I, with_bias, fmt, ckpt):
    say(f"routing gradient T={T} H={H} E={E} tk={tk} I={I} {fmt} {ckpt}")
    rng = np.random.default_rng(T + H + E + 2)
    x, w1, w2, logits, d_out = block(rng, T, H, E, I)
    bias = cu(rng.standard_normal(E).astype(np.float32)) if with_bias else None
    args = (dev_vals(x), cu(logits), tk, prepared(fmt, w1), prepared(fmt, w2), bias, ckpt)
    dd = dev_vals(d_out)
    plain, ps = pipeline.moe_train_forward(*args)
    out, st = pipeline.moe_train_forward(*args, keep_y2=True)
    assert ps.y2 is None and same(out, plain)
    assert same(out, F.moe_unpermute_combine(st.y2, st.inv_perm, st.topk_w))
    a = pipeline.moe_train_backward(ps, dd, want_d_logits=True)
    g = pipeline.moe_train_backward(st, dd, want_d_logits=True)
    torch.cuda.synchronize()
    # nothing else changes
    assert set(a) == set(g) and all(same(a[k], g[k]) for k in ("dx", "dw_first", "dw_down"))

    inv, tw = st.inv_perm.cpu().numpy(), st.topk_w.cpu().numpy()
    y2 = host_vals(st.y2)
    _, want = OX.combine_backward(d_out, y2, inv, tw)
    _, mag = OX.combine_backward(np.abs(d_out), np.abs(y2), inv, tw)
    check(g["d_topk_w"].cpu().numpy().astype(np.float64), want, H * U * mag + 2.0 ** -149, "d_topk_w")
    dl, db = F.moe_permute_backward(st.topk_ids, st.topk_w, g["d_topk_w"], E, want_bias=True)
    assert same(g["d_logits"], dl) and (not with_bias or same(g["d_bias"], db))


@pytest.mark.parametrize("T,H,E,tk,I,with_bias", [BLOCKS[1], BLOCKS[4]])
def test_logits_gradient_against_differences(dev, T, H, E, tk, I, with_bias):
    """Of sum(out d_out) over the logits, in float64, out as the combine forms it
    from the rows that the forward combined.  A step of s = 2^-10 is off by
    s^2 / 6 of the third derivative, at most 6 of the spread 2 max|d| of a softmax's
    values: 2^-19 max|d|; by rounding, 2^-52 / s of |L| <= max|d|: 2^-42.  The
    calls' own: H U mag for d_topk_w, which enters twice, and for weights whose
    float32 exponent is off by a few steps of |l| < 8, (tk + 3 + 32) U of 2 max|d|."""
    say(f"routing differences T={T} H={H} E={E}")
    rng = np.random.default_rng(T + E)
    x, w1, w2, logits, d_out = block(rng, T, H, E, I)
    bias = rng.standard_normal(E).astype(np.float32)
    _, st = pipeline.moe_train_forward(dev_vals(x), cu(logits), tk, prepared("mxfp4", w1), prepared("mxfp4", w2),
                                       cu(bias), keep_y2=True)
    g = pipeline.moe_train_backward(st, dev_vals(d_out), want_d_logits=True)
    ids, y = st.topk_ids.cpu().numpy().astype(np.int64), host_vals(st.y2)[st.inv_perm.cpu().numpy()]
    dots = np.einsum("tn,tjn->tj", d_out, y)
    mag = np.einsum("tn,tjn->tj", np.abs(d_out), np.abs(y)).max(1, keepdims=True)

    def per_token(l):
        z = np.take_along_axis(l, ids, 1)
        e = np.exp(z - z.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True) * dots).sum(1)

    base, s, num = logits.astype(np.float64) + bias, 2.0 ** -10, np.zeros((T, E))
    for e in range(E):
        up, dn = base.copy(), base.copy()
        up[:, e] += s
        dn[:, e] -= s
        num[:, e] = (per_token(up) - per_token(dn)) / (2 * s)
    big = np.abs(dots).max(1, keepdims=True)
    lim = (2.0 ** -19 + 2.0 ** -42) * big + 2 * H * U * mag + (tk + 35) * U * 2 * big
    check(g["d_logits"].cpu().numpy().astype(np.float64), num, np.broadcast_to(lim, num.shape), "d_logits")
    check(g["d_bias"].cpu().numpy().astype(np.float64), num.sum(0), lim.sum() + 8 * U * np.abs(num).sum(0), "d_bias")


def test_strided_gradient_is_refused_and_adds_nothing(dev):
    rng = np.random.default_rng(6)
    x, w1, w2, logits, d_out = block(rng, 20, 128, 4, 128)
    _, st = pipeline.moe_train_forward(dev_vals(x), cu(logits), 2, prepared("w4a16", w1), prepared("w4a16", w2),
                                       keep_y2=True)
    wide = torch.zeros((20, 256), dtype=torch.bfloat16, device="cuda")[:, :128]
    acc = torch.ones((4, 256, 128), device="cuda")
    with pytest.raises(F.NvfpError):
        pipeline.moe_train_backward(st, wide, dw_first=acc)
    torch.cuda.synchronize()
    assert bool((acc == 1).all())


@pytest.mark.parametrize("T", [0, 30])
def test_graph_replays_and_no_tokens(dev, T):
    say(f"routing gradient graph T={T}")
    rng = np.random.default_rng(T + 3)
    x, w1, w2, logits, d_out = block(rng, 30, 128, 4, 128)
    s = [dev_vals(x)[:T], cu(logits)[:T], dev_vals(d_out)[:T]]
    q1, q2 = prepared("mxfp4", w1), prepared("mxfp4", w2)

    def step():
        out, st = pipeline.moe_train_forward(s[0], s[1], 2, q1, q2, keep_y2=True)
        g = pipeline.moe_train_backward(st, s[2], want_d_logits=True)
        return [out, *(g[k] for k in sorted(g))]
    want = step()
    torch.cuda.synchronize()
    if T == 0:
        assert want[0].shape == (0, 128) and not any(t.any() for t in want)
        return
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want)), i
        s[2].mul_(-0.5)
        want = [t.clone() for t in step()]
