"""The MXFP4 block as it is used (pipeline.moe_forward_mxfp4, the training pair
with MXFP4 weights, the routing's gradients): against the float64 oracle stage
by stage, as captured graphs, on several streams, and at the largest sizes.

Tolerances are those of the single calls (test_gpu_mxfp4.py,
test_gpu_route_grad.py): a stage is given what the one before it returned, so
no rounding is passed on."""
import sys

import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from oracle import formats as OF
from oracle import moe as OM
from oracle import mxfp4 as OX
from oracle import train as OT
from tests.gpu_util import heavy_bf16, host_vals, to_dev_bf16
from tests.test_gpu_mxfp4 import check, limits, operands, swiglu_limits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_vals(v):
    return to_dev_bf16(OF.f64_to_bf16_bits(v))


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def block(rng, T, H, E, I):
    return (heavy_bf16(rng, (T, H)), OF.round_to_bf16(rng.standard_normal((E, 2 * I, H)) * 0.05),
            OF.round_to_bf16(rng.standard_normal((E, H, I)) * 0.05),
            rng.standard_normal((T, E)).astype(np.float32),
            OF.round_to_bf16(rng.standard_normal((T, H)) * 1e-3))


def kept(v):
    """The values that the MXFP4 codes of v [.., M, K] stand for."""
    return OX.value(*OX.encode(v.reshape(-1, v.shape[-1]))).reshape(v.shape)


def of_dev(c, s):
    return OX.value(c.cpu().numpy(), s.cpu().numpy())


# few rows (one launch), large tiles, one expert, experts without rows
BLOCKS = [(5, 128, 4, 2, 128, False), (96, 256, 8, 2, 128, True), (700, 512, 4, 3, 256, True),
          (300, 128, 1, 1, 384, False), (40, 256, 60, 4, 128, True)]


@pytest.mark.parametrize("T,H,E,tk,I,with_bias", BLOCKS)
def test_forward(dev, T, H, E, tk, I, with_bias):
    say(f"mxfp4 block T={T} H={H} E={E} tk={tk} I={I}")
    rng = np.random.default_rng(T + H + E)
    x, w1, w2, logits, _ = block(rng, T, H, E, I)
    bias = rng.standard_normal(E).astype(np.float32) if with_bias else None
    q1, q2 = pipeline.prepare_mxfp4_weights(dev_vals(w1)), pipeline.prepare_mxfp4_weights(dev_vals(w2))
    assert q1.t_codes is None
    args = (dev_vals(x), cu(logits), tk, q1, q2, None if bias is None else cu(bias))
    out, st = pipeline.moe_forward_mxfp4(*args, keep=True)
    out2, none = pipeline.moe_forward_mxfp4(*args)
    torch.cuda.synchronize()
    assert same(out, out2) and none == {}
    ids, tw = OM.route(logits, tk, bias)
    offs, perm, inv = OM.permute(ids, E)
    assert np.array_equal(st["topk_ids"].cpu().numpy(), ids)
    y1, mag = OX.grouped_gemm(kept(x), perm, kept(w1), offs)
    check(host_vals(st["h"]), OX.swiglu(y1), swiglu_limits(y1, mag, H), "h")
    y2, mag = OX.grouped_gemm(kept(host_vals(st["h"])), None, kept(w2), offs)
    check(host_vals(st["y2"]), y2, limits(y2, mag, I), "y2")
    # tk products of float32 weights (off by a few steps of the softmax) and bf16
    # rows, tk sums, one rounding
    yd, w = host_vals(st["y2"]), st["topk_w"].cpu().numpy().astype(np.float64)
    want = (w[..., None] * yd[inv]).sum(1)
    lim = 2 * tk * U * (w[..., None] * np.abs(yd[inv])).sum(1) + 2.0 ** -8 * np.abs(want) + 2.0 ** -126
    check(host_vals(out), want, lim, "out")


@pytest.mark.parametrize("T,H,E,tk,I,with_bias", BLOCKS)
@pytest.mark.parametrize("ckpt", ["bf16", "mxfp8"])
def test_training_step(dev, T, H, E, tk, I, with_bias, ckpt):
    """The step's outputs are those of the calls it is made of, and these are
    the formulas' on what they were given."""
    say(f"mxfp4 train T={T} H={H} E={E} tk={tk} I={I} {ckpt}")
    rng = np.random.default_rng(T + H + E + 1)
    x, w1, w2, logits, d_out = block(rng, T, H, E, I)
    bias = rng.standard_normal(E).astype(np.float32) if with_bias else None
    wd1, wd2 = dev_vals(w1), dev_vals(w2)
    q1 = pipeline.prepare_mxfp4_weights(wd1, want_transposed=True)
    q2 = pipeline.prepare_mxfp4_weights(wd2, want_transposed=True)
    xd, dd = dev_vals(x), dev_vals(d_out)
    out, st = pipeline.moe_train_forward(xd, cu(logits), tk, q1, q2, None if bias is None else cu(bias), ckpt)
    g = pipeline.moe_train_backward(st, dd, want_d_logits=True)
    assert ("d_bias" in g) == with_bias and "d_logits" not in pipeline.moe_train_backward(st, dd)

    ids, tw, offs, perm, inv = F.moe_permute(cu(logits), tk, None if bias is None else cu(bias))
    P = perm.numel()
    y1 = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(xd), perm, *F.mxfp4_quantize(wd1), offs, M_total=P)
    h = F.mxfp8_checkpoint(y1, glu=True)["h"]
    y2 = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(h), None, *F.mxfp4_quantize(wd2), offs, M_total=P)
    assert same(out, F.moe_unpermute_combine(y2, inv, tw))
    t2 = F.mxfp4_quantize(wd2, transpose=True)
    dh = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(dd), perm, *t2, offs, M_total=P)
    dy1, hw, d_tw = F.moe_swiglu_backward(st.y1, dh, inv, tw, y_scales=st.y1_scales)
    dxp = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(dy1), None, *F.mxfp4_quantize(wd1, transpose=True), offs,
                               M_total=P)
    dl, db = F.moe_permute_backward(ids, tw, d_tw, E, want_bias=True)
    assert same(g["dx"], F.moe_unpermute_combine(dxp, inv, torch.ones_like(tw)))
    assert same(g["d_topk_w"], d_tw) and same(g["d_logits"], dl) and (not with_bias or same(g["d_bias"], db))
    assert same(g["dw_first"], F.grouped_wgrad(dy1, None, st.x, perm, offs, x_scales=st.x_scales, M_total=P))
    assert same(g["dw_down"], F.grouped_wgrad(dd, perm, hw, None, offs, M_total=P))

    # the products of the backward pass, on what they were given
    ho, hp = offs.cpu().numpy(), perm.cpu().numpy()
    tr = lambda w: np.stack([kept(np.ascontiguousarray(m.T)) for m in w])        # noqa: E731
    ref, mag = OX.grouped_gemm(kept(d_out), hp, tr(w2), ho)
    check(host_vals(dh), ref, limits(ref, mag, H), "dh")
    ref, mag = OX.grouped_gemm(kept(host_vals(dy1)), None, tr(w1), ho)
    check(host_vals(dxp), ref, limits(ref, mag, 2 * I), "dxp")

    # the other way round the down projection: the combine's own gradient, whose
    # rows carry the routing weight
    dy2, dw2 = F.moe_unpermute_combine_backward(dd, y2, inv, tw)
    rdy, rdw = OX.combine_backward(d_out, host_vals(y2), inv.cpu().numpy(), tw.cpu().numpy())
    check(host_vals(dy2), rdy, np.abs(rdy) * (2.0 ** -8 + 2 * U) + 2.0 ** -133, "dy2")
    mag = OX.combine_backward(np.abs(d_out), np.abs(host_vals(y2)), inv.cpu().numpy(), tw.cpu().numpy())[1]
    check(dw2.cpu().numpy().astype(np.float64), rdw, H * U * mag + 2.0 ** -149, "dw2")
    dh2 = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(dy2), None, *t2, offs, M_total=P)
    ref, mag = OX.grouped_gemm(kept(host_vals(dy2)), None, tr(w2), ho)
    check(host_vals(dh2), ref, limits(ref, mag, H), "dh2")


def test_routing_gradient_against_differences(dev):
    """d(sum out d_out)/d(logits, bias) through the combine and the routing
    weights, against central differences of the formula in float64.

    Of step s = 2^-10: the difference is off by s^2 / 6 of the third derivative,
    which a softmax bounds by 6 of the spread of its values, 2 max |d_topk_w|:
    12 max|dw| s^2 / 6 = 2^-19 max|dw|, and by its rounding, 2^-52 / s of
    |L|.  The calls' own: the sums' N U mag and (tk + 3) U, of at most max mag."""
    say("routing differences")
    rng = np.random.default_rng(77)
    T, E, tk, N = 24, 12, 4, 256
    logits, bias = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal(E).astype(np.float32)
    y, d_out = heavy_bf16(rng, (T * tk, N)), OF.round_to_bf16(rng.standard_normal((T, N)))
    ids, tw, offs, perm, inv = F.moe_permute(cu(logits), tk, cu(bias))
    _, dw = F.moe_unpermute_combine_backward(dev_vals(d_out), dev_vals(y), inv, tw)
    dl, db = F.moe_permute_backward(ids, tw, dw, E, want_bias=True)
    hi, hinv = ids.cpu().numpy().astype(np.int64), inv.cpu().numpy()
    dots = np.einsum("tn,tjn->tj", d_out, y[hinv])
    mag = np.einsum("tn,tjn->tj", np.abs(d_out), np.abs(y[hinv]))

    def per_token(l):
        z = np.take_along_axis(l, hi, 1)
        e = np.exp(z - z.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True) * dots).sum(1)

    base = logits.astype(np.float64) + bias
    s = 2.0 ** -10
    num = np.zeros((T, E))
    for e in range(E):
        up, dn = base.copy(), base.copy()
        up[:, e] += s
        dn[:, e] -= s
        num[:, e] = (per_token(up) - per_token(dn)) / (2 * s)
    big = np.abs(dots).max(1, keepdims=True)
    # (the calls' weights: a float32 exponent off by 2^-23 of |l| < 8, a few steps)
    lim = 2.0 ** -19 * big + 2.0 ** -42 * big + 2 * (N * U * mag.max(1, keepdims=True)) + \
        (tk + 3 + 32) * U * 2 * big
    check(dl.cpu().numpy().astype(np.float64), num, np.broadcast_to(lim, num.shape), "d_logits")
    check(db.cpu().numpy().astype(np.float64), num.sum(0), lim.sum() + 8 * U * np.abs(num).sum(0), "d_bias")


def steps(s, tk):
    out, _ = pipeline.moe_forward_mxfp4(s[0], s[3], tk, s[1], s[2], s[5])
    o, st = pipeline.moe_train_forward(s[0], s[3], tk, s[1], s[2], s[5])
    g = pipeline.moe_train_backward(st, s[4], want_d_logits=True)
    y = torch.empty_like(s[0])
    F.mxfp4_restore(*F.mxfp4_quantize(s[0]), out=y)
    dy, dw = F.moe_unpermute_combine_backward(s[4], None, st.inv_perm, st.topk_w)
    return [out, o, y, dy, *(g[k] for k in sorted(g))]


def on_device(rng, T, H, E, I):
    x, w1, w2, logits, d_out = block(rng, T, H, E, I)
    prep = lambda w: pipeline.prepare_mxfp4_weights(dev_vals(w), want_transposed=True)   # noqa: E731
    return [dev_vals(x), prep(w1), prep(w2), cu(logits), dev_vals(d_out),
            cu(rng.standard_normal(E).astype(np.float32))]


@pytest.mark.parametrize("T,H,E,tk,I", [(6, 128, 4, 2, 128), (500, 512, 4, 2, 256)])
def test_graph_replays_match_eager(dev, T, H, E, tk, I):
    """Two graphs captured from the same calls, replayed one after the other and
    with eager calls between, also for new inputs in place."""
    say(f"mxfp4 graph T={T}")
    rng = np.random.default_rng(T)
    s = on_device(rng, T, H, E, I)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(s, tk)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = steps(s, tk)
        graphs.append((g, got))
    for i in range(4):
        if i == 2:                                       # other data, other routing
            n = on_device(rng, T, H, E, I)
            for k in (0, 3, 4, 5):
                s[k].copy_(n[k])
        want = [t.clone() for t in steps(s, tk)]
        for g, got in graphs:
            for t in got:
                t.zero_()
        for g, got in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, got in graphs:
            assert all(same(a, b) for a, b in zip(got, want)), f"replay {i}"


def test_two_streams_at_once(dev):
    say("mxfp4 streams")
    rng = np.random.default_rng(23)
    sets = [on_device(rng, 400, 256, 4, 128) for _ in range(2)]
    want = [steps(s, 2) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, q in zip(sets, streams):
            with torch.cuda.stream(q):
                got.append(steps(s, 2))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(same(u, v) for u, v in zip(a, b))


def test_no_tokens(dev):
    rng = np.random.default_rng(1)
    s = on_device(rng, 3, 128, 2, 128)
    x, lg = s[0][:0], s[3][:0]
    out, _ = pipeline.moe_forward_mxfp4(x, lg, 1, s[1], s[2], s[5])
    o, st = pipeline.moe_train_forward(x, lg, 1, s[1], s[2], s[5])
    g = pipeline.moe_train_backward(st, x, want_d_logits=True)
    torch.cuda.synchronize()
    assert out.shape == o.shape == g["dx"].shape == (0, 128) and g["d_logits"].shape == (0, 2)
    assert not g["dw_first"].any() and not g["dw_down"].any() and not g["d_bias"].any()


def test_w4a16_step_gives_the_same_logit_gradient(dev):
    """want_d_logits with the W4A16 products; what the step returned before
    stays as it is."""
    rng = np.random.default_rng(4)
    x, w1, w2, logits, d_out = block(rng, 50, 128, 8, 128)
    q1, q2 = pipeline.prepare_weights(dev_vals(w1)), pipeline.prepare_weights(dev_vals(w2))
    _, st = pipeline.moe_train_forward(dev_vals(x), cu(logits), 2, q1, q2)
    a = pipeline.moe_train_backward(st, dev_vals(d_out))
    b = pipeline.moe_train_backward(st, dev_vals(d_out), want_d_logits=True)
    torch.cuda.synchronize()
    assert set(b) - set(a) == {"d_logits"} and all(same(a[k], b[k]) for k in a)
    w, dw = st.topk_w.cpu().numpy().astype(np.float64), a["d_topk_w"].cpu().numpy().astype(np.float64)
    got = np.take_along_axis(b["d_logits"].cpu().numpy(), st.topk_ids.cpu().numpy().astype(np.int64), 1)
    ref = OT.route_backward(w, dw)
    assert np.all(np.abs(got - ref) <= 5 * U * w * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True)))


# ---------------------------------------------------------------- the calls' edges
@pytest.mark.parametrize("counts,N,K", [([5, 0, 9], 64, 640), ([200, 300, 12], 512, 896)])
def test_unaligned_scales_rows_and_views(dev, counts, N, K):
    """Scales and row lists that begin 4 bytes into their memory, codes 16
    bytes, an output that is a view: the bits of the aligned call."""
    say(f"mxfp4 views {counts}")
    rng = np.random.default_rng(N)
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    P, E = int(offs[-1]), len(counts)
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, P, E, N, K))
    rows = cu(rng.integers(0, P, P).astype(np.int32))
    od = cu(offs)

    def at(t, skip):
        m = torch.empty(t.numel() + skip, dtype=t.dtype, device="cuda")
        v = m[skip:].view(t.shape)
        v.copy_(t)
        return v

    want = F.grouped_mxfp4_gemm(ac, asc, rows, wc, wsc, od)
    out = torch.full((P + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    F.grouped_mxfp4_gemm(at(ac, 16), at(asc, 4), at(rows, 1), at(wc, 16), at(wsc, 4), at(od, 1),
                         out=out[1:-1])
    torch.cuda.synchronize()
    assert same(out[1:-1], want) and bool((out[0] == 9).all()) and bool((out[-1] == 9).all())


@pytest.mark.parametrize("N", [64, 1024])
def test_offsets_and_rows_out_of_range(dev, N):
    """Offsets beyond the output count as its end, rows beyond the source as its
    last; offsets that decrease write no more than the output's rows and the
    workspace."""
    say(f"mxfp4 out of range N={N}")
    rng = np.random.default_rng(N)
    M, K = 300, 256
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, M, 3, N, K))
    rows = rng.integers(0, M, M).astype(np.int32)
    far = rows.copy()
    far[[0, 7]], far[[3, 299]] = -5, M + 1000
    rows[[0, 7]], rows[[3, 299]] = 0, M - 1
    a = F.grouped_mxfp4_gemm(ac, asc, cu(far), wc, wsc, cu(np.array([-9, 100, 200, 1 << 30], np.int32)))
    b = F.grouped_mxfp4_gemm(ac, asc, cu(rows), wc, wsc, cu(np.array([0, 100, 200, M], np.int32)))
    torch.cuda.synchronize()
    assert same(a, b)
    # 64 experts whose offsets swing between the ends: 32 M rows instead of M
    E = 64
    w, ws = wc[:1].expand(E, -1, -1).contiguous(), wsc[:1].expand(E, -1, -1).contiguous()
    offs = np.array([0, M] * (E // 2) + [0], np.int32)
    out = torch.full((M + 1, N), 9.0, dtype=torch.bfloat16, device="cuda")
    nb = F.lib().grouped_mxfp4_gemm_workspace_size(E, M, N, K)
    mem = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    F._call("grouped_mxfp4_gemm", out.device, ac.data_ptr(), asc.data_ptr(), None, M, w.data_ptr(),
            ws.data_ptr(), cu(offs).data_ptr(), E, M, N, K, out.data_ptr(), mem.data_ptr(), nb)
    one = F.grouped_mxfp4_gemm(ac, asc, None, wc[:1], wsc[:1], cu(np.array([0, M], np.int32)))
    torch.cuda.synchronize()
    assert bool((mem[nb:] == 0xA5).all()) and bool((out[M] == 9).all())
    assert bool(((out[:M] == one) | (out[:M] == 9)).all())


def test_many_experts(dev):
    """1024 experts, most without a row, through both kernels."""
    say("mxfp4 1024 experts")
    rng = np.random.default_rng(9)
    E, N, K = 1024, 96, 128
    for P in (3, 900):
        counts = np.bincount(np.where(rng.random(P) < 0.3, 1023, rng.integers(0, E, P)), minlength=E)
        offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ac, asc, wc, wsc = operands(rng, P, E, N, K)
        y = F.grouped_mxfp4_gemm(cu(ac), cu(asc), None, cu(wc), cu(wsc), cu(offs))
        torch.cuda.synchronize()
        w = OX.value(wc.reshape(E * N, -1), wsc.reshape(E * N, -1)).reshape(E, N, K)
        ref, mag = OX.grouped_gemm(OX.value(ac, asc), None, w, offs)
        check(host_vals(y), ref, limits(ref, mag, K), f"y of {P}")


def test_products_past_2_31_elements(dev):
    """An output of more than 2^31 elements and codes of more than 2^31 bytes:
    rows of either end are those of the same rows alone."""
    say("mxfp4 large product")
    rng = np.random.default_rng(10)
    N, K, M = 32768, 128, 66000
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, M, 1, N, K))
    y = F.grouped_mxfp4_gemm(ac, asc, None, wc, wsc, cu(np.array([0, M], np.int32)))
    for lo in (0, 32768, 65500, M - 128):
        part = F.grouped_mxfp4_gemm(ac[lo:lo + 128].contiguous(), asc[lo:lo + 128].contiguous(), None, wc, wsc,
                                    cu(np.array([0, 128], np.int32)))
        assert same(y[lo:lo + 128], part), lo
    del y
    K, M = 65536, 70000
    c = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.randint(100, 140, (M, K // 32), dtype=torch.uint8, device="cuda")
    wc = torch.randint(0, 256, (2, 64, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(100, 140, (2, 64, K // 32), dtype=torch.uint8, device="cuda")
    y = F.grouped_mxfp4_gemm(c, s, None, wc, ws, cu(np.array([0, 65537, M], np.int32)))
    rows = [0, 65535, 65536, 65537, M - 1]
    for i, r in enumerate(rows):
        e = int(r >= 65537)
        ref, mag = OX.grouped_gemm(of_dev(c[r:r + 1], s[r:r + 1]), None, of_dev(wc[e], ws[e])[None], [0, 1])
        check(host_vals(y[r:r + 1]), ref, limits(ref, mag, K), f"row {r}")


def test_quantize_past_2_31_elements(dev):
    say("mxfp4 large quantize")
    M, K = 131104, 16416
    x = torch.randn((M, K), dtype=torch.bfloat16, device="cuda")
    c, s = F.mxfp4_quantize(x)
    y = F.mxfp4_restore(c, s)
    for lo in (0, 65536, 130816, M - 32):
        part = F.mxfp4_quantize(x[lo:lo + 32])
        assert same(c[lo:lo + 32], part[0]) and same(s[lo:lo + 32], part[1])
        assert same(y[lo:lo + 32], F.mxfp4_restore(*part)), lo
    del c, s, y
    c, s = F.mxfp4_quantize(x, transpose=True)
    for lo in (0, 8192, K - 32):
        part = F.mxfp4_quantize(x[:, lo:lo + 32].t().contiguous())
        assert same(c[lo:lo + 32], part[0]) and same(s[lo:lo + 32], part[1]), lo


def test_combine_backward_past_2_31_elements(dev):
    say("combine backward large")
    T, tk, N = 40000, 2, 32768
    d = torch.randn((T, N), dtype=torch.bfloat16, device="cuda")
    y = torch.randn((T * tk, N), dtype=torch.bfloat16, device="cuda")
    inv = torch.randperm(T * tk, device="cuda").to(torch.int32).view(T, tk)
    w = torch.rand((T, tk), device="cuda")
    dy, dw = F.moe_unpermute_combine_backward(d, y, inv, w)
    pick = torch.tensor([0, 20000, 33000, T - 1], device="cuda")
    k = inv[pick].long()
    want = (w[pick][..., None] * d[pick].float()[:, None]).to(torch.bfloat16)
    assert torch.equal(dy[k.view(-1)], want.view(-1, N))
    p = d[pick].double()[:, None] * y[k.view(-1)].view(4, tk, N).double()
    assert bool(((dw[pick] - p.sum(-1)).abs() <= N * U * p.abs().sum(-1)).all())
