"""GPU parity of the training-step calls (8-bit activation checkpoints, input
and weight gradients of the W4A16 product, SwiGLU backward) against the float64
oracle, one by one and as the chain pipeline.moe_train_forward/_backward runs.

Tolerances, from the arithmetic.  A product of two bf16 values is exact in
float32 and the kernels add n of them in float32, so a sum is off by at most
n * 2^-24 times the sum of magnitudes (any order); an output rounded to bf16
adds half a step, 2^-8 of its value.  One more 2^-24 for g_w."""
import sys

import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from oracle import formats as OF
from oracle import gemm as OG
from oracle import moe as OM
from oracle import nvfp4 as OQ
from oracle import train as OT
from tests.gpu_util import gemm_wcodes, gemm_wscales, heavy_bf16, host_bits, host_vals, to_dev_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_vals(v):
    return to_dev_bf16(OF.f64_to_bf16_bits(v))


def check(got, ref, lim, what):
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= lim)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / lim, 0)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.size} off; worst at {i}: got "
                             f"{got[i]!r} want {ref[i]!r} allowed {lim[i]!r}")


def offsets_of(counts):
    offs = np.zeros(len(counts) + 1, dtype=np.int32)
    offs[1:] = np.cumsum(counts)
    return offs


# ---------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (64, 512), (129, 96), (37, 4096), (5, 32768)])
def test_checkpoint_and_restore(dev, M, K):
    say(f"checkpoint M={M} K={K}")
    rng = np.random.default_rng(M + K)
    x = heavy_bf16(rng, (M, K))
    x[0, :32] = 0.0
    x[-1, -3:] = [448.0, -450.0, 2.0 ** -130]
    xd = dev_vals(x)
    c = F.mxfp8_checkpoint(xd)
    y = F.mxfp8_restore(c["codes"], c["scales"])
    torch.cuda.synchronize()
    codes, scales = OT.mxfp8_encode(x)
    assert c["h"] is None
    assert np.array_equal(c["scales"].cpu().numpy(), scales)
    assert np.array_equal(c["codes"].cpu().numpy(), codes)
    assert np.array_equal(host_vals(y), OT.mxfp8_value(codes, scales))


def test_checkpoint_every_bf16(dev):
    """Every bf16 bit pattern, each as the largest of a block and as a small
    one beside 448, 449 and the largest value; NaN and infinities among them."""
    say("checkpoint every bf16")
    bits = np.arange(65536, dtype=np.uint16)
    x = np.zeros((4 * 65536, 32), dtype=np.uint16)
    x[:, 7] = np.tile(bits, 4)
    x[:, 20] = np.repeat(np.array([0x0000, 0x43E0, 0x43E1, 0x7F7F], dtype=np.uint16), 65536)
    xd = to_dev_bf16(x)
    c = F.mxfp8_checkpoint(xd)
    y = F.mxfp8_restore(c["codes"], c["scales"])
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        vals = OF.bf16_bits_to_f64(x)
    codes, scales = OT.mxfp8_encode(vals)
    got = c["codes"].cpu().numpy()
    nan = (codes & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], codes[~nan])
    assert np.array_equal(c["scales"].cpu().numpy(), scales)
    back = host_vals(y)
    assert np.all(np.isnan(back[nan]))
    assert np.array_equal(back[~nan], OT.mxfp8_value(codes, scales)[~nan])


def test_checkpoint_strided_rows(dev):
    say("checkpoint strided")
    rng = np.random.default_rng(3)
    wide = dev_vals(heavy_bf16(rng, (21, 320)))
    x = wide[:, 64:288]
    c = F.mxfp8_checkpoint(x)
    d = F.mxfp8_checkpoint(x.contiguous())
    assert torch.equal(c["codes"], d["codes"]) and torch.equal(c["scales"], d["scales"])
    out = torch.full((21, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    F.mxfp8_restore(c["codes"], c["scales"], out=out[:, 64:288])
    torch.cuda.synchronize()
    assert torch.equal(out[:, 64:288], F.mxfp8_restore(c["codes"], c["scales"]))
    assert bool((out[:, :64] == 7).all()) and bool((out[:, 288:] == 7).all())
    with pytest.raises(F.NvfpError):
        F.mxfp8_checkpoint(wide[:, 4:292])               # 8-byte aligned rows only
    with pytest.raises(F.NvfpError):
        F.mxfp8_checkpoint(wide.t())


@pytest.mark.parametrize("M,I", [(1, 32), (7, 96), (130, 768), (3, 4096)])
def test_checkpoint_with_swiglu(dev, M, I):
    say(f"checkpoint glu M={M} I={I}")
    rng = np.random.default_rng(M * I)
    y = heavy_bf16(rng, (M, 2 * I))
    yd = dev_vals(y)
    c = F.mxfp8_checkpoint(yd, glu=True)
    only = F.mxfp8_checkpoint(yd, glu=True, want_codes=False)
    h = F.nvfp4_quantize_act(yd, glu=True)["x_used"]
    torch.cuda.synchronize()
    codes, scales = OT.mxfp8_encode(y)
    assert np.array_equal(c["codes"].cpu().numpy(), codes)
    assert np.array_equal(c["scales"].cpu().numpy(), scales)
    assert torch.equal(c["h"].view(torch.int16), h.view(torch.int16))
    assert only["codes"] is None and torch.equal(only["h"].view(torch.int16), h.view(torch.int16))


def test_checkpoint_no_rows(dev):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    c = F.mxfp8_checkpoint(x, glu=True)
    assert c["codes"].shape == (0, 64) and c["h"].shape == (0, 32)
    assert F.mxfp8_restore(c["codes"], c["scales"]).shape == (0, 64)


# ------------------------------------------------------------- input gradient
def dgrad_case(rng, counts, N, K, gather, M_src=None, pad=0):
    E, offs = len(counts), offsets_of(counts)
    P = int(offs[-1])
    M_src = M_src or (max(1, P // 2) if gather else P + pad)
    dy = heavy_bf16(rng, (M_src, N)) * 2.0 ** -10
    w = OF.round_to_bf16(rng.standard_normal((E, N, K)) * 0.02)
    wc, ws, gw, _ = OQ.qdq_weights(w)
    rows = rng.integers(0, M_src, P + pad).astype(np.int32) if gather else None
    return dy, rows, wc, ws, gw, offs


def run_dgrad(dy, rows, wc, ws, gw, offs, **kw):
    return F.grouped_w4a16_dgrad(dev_vals(dy), None if rows is None else cu(rows),
                                 cu(gemm_wcodes(OQ.pack_codes(wc))), cu(gemm_wscales(ws)), cu(gw),
                                 cu(offs), **kw)


def check_dgrad(dx, ref, mag, N, what):
    check(dx, ref, np.abs(ref) * 2.0 ** -8 + (N + 2) * U * mag + TINY, what)


DGRAD = [
    ([1], 16, 64, False),
    ([1], 512, 512, False),
    ([64], 512, 512, False),
    ([5], 1040, 192, True),
    ([0, 130, 1, 257], 144, 256, True),                 # empty and single-row experts
    ([300, 1, 511, 0, 255], 528, 768, True),            # several row tiles
    ([3, 0, 17, 33, 1, 0, 16, 40], 272, 384, True),     # a few rows each
    ([20, 9, 0, 19], 80, 640, False),
    ([300], 4096, 320, False),
    ([1] * 33 + [0] * 7 + [2] * 9, 48, 128, True),
    ([700, 33], 64, 1088, False),
    ([17, 64, 65], 32, 64, True),
    ([9, 2], 4112, 256, True),                          # a long contraction for few rows
]


@pytest.mark.parametrize("counts,N,K,gather", DGRAD)
def test_dgrad(dev, counts, N, K, gather):
    say(f"dgrad counts={counts} N={N} K={K} gather={gather}")
    rng = np.random.default_rng(sum(counts) + N + K)
    dy, rows, wc, ws, gw, offs = dgrad_case(rng, counts, N, K, gather)
    dx = run_dgrad(dy, rows, wc, ws, gw, offs, M_total=int(offs[-1]))
    torch.cuda.synchronize()
    ref, mag = OT.grouped_dgrad(dy, rows, wc, ws, gw, offs)
    check_dgrad(host_vals(dx), ref, mag, N, "dx")


@pytest.mark.parametrize("counts,K", [
    ([128, 129, 0, 256, 257, 384, 385, 64, 65], 320),     # every kind of last tile
    ([256, 512, 256], 1088),                              # no tails
    ([191, 192, 193, 448, 449, 130], 256),                # whole tiles of three and four parts
    ([100, 0, 64, 128, 1, 127], 576),                     # nothing but tails
    ([2, 640, 3] + [40] * 70, 64),                        # tails past the first 64 experts
])
def test_dgrad_row_tile_edges(dev, counts, K):
    say(f"dgrad edges {counts} K={K}")
    rng = np.random.default_rng(sum(counts) + K)
    dy, rows, wc, ws, gw, offs = dgrad_case(rng, counts, 80, K, True)
    dx = run_dgrad(dy, rows, wc, ws, gw, offs, M_total=int(offs[-1]))
    torch.cuda.synchronize()
    ref, mag = OT.grouped_dgrad(dy, rows, wc, ws, gw, offs)
    check_dgrad(host_vals(dx), ref, mag, 80, "dx")


def test_dgrad_is_the_forward_transposed(dev):
    """<dy, W x> = <W^T dy, x> with the forward's own product."""
    say("dgrad adjoint")
    rng = np.random.default_rng(5)
    counts, N, K = [40, 0, 77], 256, 384
    dy, _, wc, ws, gw, offs = dgrad_case(rng, counts, N, K, False)
    x = heavy_bf16(rng, (117, K))
    pc, ps = cu(gemm_wcodes(OQ.pack_codes(wc))), cu(gemm_wscales(ws))
    y = host_vals(F.grouped_w4a16_gemm(dev_vals(x), None, pc, ps, cu(gw), cu(offs)))
    dx = host_vals(F.grouped_w4a16_dgrad(dev_vals(dy), None, pc, ps, cu(gw), cu(offs)))
    a, b = dy * y, dx * x
    # both sides rounded to bf16 element by element
    lim = 2.0 ** -8 * (np.abs(a).sum() + np.abs(b).sum())
    assert abs(a.sum() - b.sum()) <= lim


def test_dgrad_leaves_other_rows_alone(dev):
    say("dgrad padding rows")
    rng = np.random.default_rng(6)
    for counts in ([30, 70], [3, 2], [0, 0]):
        dy, rows, wc, ws, gw, offs = dgrad_case(rng, counts, 128, 256, True, M_src=50, pad=29)
        P = int(offs[-1])
        out = torch.full((P + 29, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        run_dgrad(dy, rows, wc, ws, gw, offs, out=out)
        torch.cuda.synchronize()
        ref, mag = OT.grouped_dgrad(dy, rows[:P], wc, ws, gw, offs)
        check_dgrad(host_vals(out)[:P], ref, mag, 128, "dx")
        assert bool((out[P:] == 3).all())


@pytest.mark.parametrize("counts", [[70, 61], [3, 5]])
def test_dgrad_keeps_nan_and_inf_to_their_rows(dev, counts):
    say(f"dgrad nan {counts}")
    rng = np.random.default_rng(7)
    dy, _, wc, ws, gw, offs = dgrad_case(rng, counts, 80, 192, False, pad=4)
    P = int(offs[-1])
    clean = host_vals(run_dgrad(dy, None, wc, ws, gw, offs, M_total=P))
    dy[1, 5], dy[counts[0], 79], dy[P:] = np.nan, np.inf, np.nan
    got = host_vals(run_dgrad(dy, None, wc, ws, gw, offs, M_total=P))
    keep = np.ones(P, bool)
    keep[[1, counts[0]]] = False
    assert np.array_equal(got[keep], clean[keep])
    assert not np.isfinite(got[~keep]).any()


def test_dgrad_zero_weights_and_no_rows(dev):
    say("dgrad zero weights")
    z = torch.zeros((2, 32, 128), dtype=torch.bfloat16, device="cuda")
    wq = F.nvfp4_qdq_weights(z, want_qdq=False)
    dy = torch.ones((6, 32), dtype=torch.bfloat16, device="cuda")
    offs = cu(np.array([0, 4, 6], np.int32))
    dx = F.grouped_w4a16_dgrad(dy, None, wq.packed_codes, wq.packed_scales, wq.g, offs)
    assert bool((dx == 0).all())
    dx = F.grouped_w4a16_dgrad(dy, None, wq.packed_codes, wq.packed_scales, wq.g,
                               torch.zeros_like(offs), M_total=0)
    torch.cuda.synchronize()
    assert dx.shape == (0, 128)


def test_dgrad_many_experts(dev):
    """1024 experts, most without rows, the first rows of the permutation in
    none of them; few rows per expert and, on 40 experts, many."""
    for E, top, N, K in [(1024, 6, 32, 64), (40, 200, 48, 320)]:
        say(f"dgrad E={E}")
        rng = np.random.default_rng(E)
        counts = np.where(rng.random(E) < 0.5, 0, rng.integers(0, top, E))
        offs = offsets_of(counts) + 7
        P = int(offs[-1])
        dy = heavy_bf16(rng, (P, N)) * 2.0 ** -10
        w = OF.round_to_bf16(rng.standard_normal((E, N, K)) * 0.02)
        wc, ws, gw, _ = OQ.qdq_weights(w)
        out = torch.full((P, K), 5.0, dtype=torch.bfloat16, device="cuda")
        run_dgrad(dy, None, wc, ws, gw, offs, out=out)
        torch.cuda.synchronize()
        ref, mag = OT.grouped_dgrad(dy, None, wc, ws, gw, offs)
        got = host_vals(out)
        assert np.all(got[:7] == 5.0)
        check_dgrad(got[7:], ref[7:], mag[7:], N, "dx")


# ------------------------------------------------------------ weight gradient
WGRAD = [
    ([1], 8, 8),
    ([64], 512, 512),
    ([0, 130, 1, 257], 144, 256),
    ([63, 64, 65, 0, 1, 2], 72, 200),
    ([300, 1, 511, 0, 255], 264, 520),
    ([5000], 64, 96),                                    # long sums, few outputs
    ([1] * 20 + [0] * 5 + [3] * 8, 40, 104),
    ([2049, 0], 328, 64),
]


def wgrad_case(rng, counts, N, K, gather, fp8):
    offs = offsets_of(counts)
    P = int(offs[-1])
    M_dy = max(1, P // 3) if "d" in gather else P
    M_x = max(1, P // 2) if "x" in gather else P
    dy = heavy_bf16(rng, (M_dy, N)) * 2.0 ** -10
    x = heavy_bf16(rng, (M_x, K))
    dyr = rng.integers(0, M_dy, P).astype(np.int32) if "d" in gather else None
    xr = rng.integers(0, M_x, P).astype(np.int32) if "x" in gather else None
    if not fp8:
        return offs, dy, dyr, x, xr, dev_vals(x), None
    codes, scales = OT.mxfp8_encode(x)
    return offs, dy, dyr, OT.mxfp8_value(codes, scales), xr, cu(codes), cu(scales)


def opt(a):
    return None if a is None else cu(a)


@pytest.mark.parametrize("gather", ["", "x", "d", "dx"])
@pytest.mark.parametrize("counts,N,K", WGRAD)
@pytest.mark.parametrize("fp8", [False, True])
def test_wgrad(dev, counts, N, K, gather, fp8):
    if fp8:
        K = (K + 31) // 32 * 32
    say(f"wgrad counts={counts} N={N} K={K} gather={gather!r} fp8={fp8}")
    rng = np.random.default_rng(sum(counts) + N + K + len(gather))
    offs, dy, dyr, x, xr, xd, xs = wgrad_case(rng, counts, N, K, gather, fp8)
    P = int(offs[-1])
    dyd, o = dev_vals(dy), cu(offs)
    args = (dyd, opt(dyr), xd, opt(xr), o)
    dw = F.grouped_wgrad(*args, x_scales=xs, M_total=P)
    db = F.grouped_wgrad(*args, x_scales=xs, M_total=P, dtype=torch.bfloat16)
    old = rng.standard_normal(dw.shape).astype(np.float32)
    acc = cu(old)
    F.grouped_wgrad(*args, x_scales=xs, M_total=P, out=acc, accumulate=True)
    torch.cuda.synchronize()
    ref, mag = OT.grouped_wgrad(dy, dyr, x, xr, offs)
    n = max(counts)
    lim = n * U * mag + TINY
    check(dw.cpu().numpy().astype(np.float64), ref, lim, "dw")
    check(host_vals(db), ref, np.abs(ref) * 2.0 ** -8 + lim, "dw bf16")
    check(acc.cpu().numpy().astype(np.float64), ref + old, lim + U * (np.abs(ref + old) + lim),
          "dw added")
    for e, c in enumerate(counts):
        if c == 0:
            assert not dw[e].any() and not db[e].any()
            assert np.array_equal(acc[e].cpu().numpy(), old[e])
    again = F.grouped_wgrad(*args, x_scales=xs, M_total=P)
    assert torch.equal(again.view(torch.int32), dw.view(torch.int32))


@pytest.mark.parametrize("fp8", [False, True])
def test_wgrad_keeps_other_rows_out(dev, fp8):
    """NaN and infinities in one expert's rows, in rows behind the last expert
    and in rows no list names reach nothing else."""
    say(f"wgrad nan fp8={fp8}")
    rng = np.random.default_rng(8)
    counts, N, K = [37, 70, 0, 5], 136, 160
    offs = offsets_of(counts)
    P = int(offs[-1])
    dy, x = heavy_bf16(rng, (P + 9, N)), heavy_bf16(rng, (P + 9, K))

    def run():
        xd, xs = dev_vals(x), None
        if fp8:
            c = F.mxfp8_checkpoint(xd)
            xd, xs = c["codes"], c["scales"]
        return F.grouped_wgrad(dev_vals(dy), None, xd, None, cu(offs), x_scales=xs,
                               M_total=P + 9).cpu().numpy()
    clean = run()
    dy[40, 3], x[41, 4], dy[P:], x[P:] = np.nan, np.inf, np.inf, np.nan
    got = run()
    for e in (0, 2, 3):
        assert np.array_equal(got[e], clean[e])
    bad = ~np.isfinite(got[1])
    assert bad[3].all() and bad[:, 4].all()
    bad[3], bad[:, 4] = False, False
    assert not bad.any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("E,N,K,top", [(40, 520, 800, 140), (1024, 16, 32, 5), (7, 1800, 2080, 90)])
def test_wgrad_more_tiles_than_workgroups(dev, E, N, K, top, fp8):
    """Several tiles per workgroup, of different lengths and without rows in
    any order; rows before the first expert belong to none."""
    say(f"wgrad E={E} N={N} K={K} fp8={fp8}")
    rng = np.random.default_rng(E + N)
    counts = np.where(rng.random(E) < 0.3, 0, rng.integers(0, top, E))
    offs = offsets_of(counts) + 3
    P = int(offs[-1])
    dy, x = heavy_bf16(rng, (P, N)) * 2.0 ** -10, heavy_bf16(rng, (P, K))
    xd, xs = dev_vals(x), None
    if fp8:
        codes, scales = OT.mxfp8_encode(x)
        x, xd, xs = OT.mxfp8_value(codes, scales), cu(codes), cu(scales)
    dyd, o = dev_vals(dy), cu(offs)
    dw = F.grouped_wgrad(dyd, None, xd, None, o, x_scales=xs)
    db = F.grouped_wgrad(dyd, None, xd, None, o, x_scales=xs, dtype=torch.bfloat16)
    acc = F.grouped_wgrad(dyd, None, xd, None, o, x_scales=xs, out=torch.ones_like(dw),
                          accumulate=True)
    torch.cuda.synchronize()
    ref, mag = OT.grouped_wgrad(dy, None, x, None, offs)
    lim = max(counts) * U * mag + TINY
    check(dw.cpu().numpy().astype(np.float64), ref, lim, "dw")
    check(host_vals(db), ref, np.abs(ref) * 2.0 ** -8 + lim, "dw bf16")
    check(acc.cpu().numpy().astype(np.float64), ref + 1, lim + U * (np.abs(ref + 1) + lim), "added")


def test_gradients_of_operands_near_4_gib(dev):
    """Gathered rows behind the 2 and 4 GiB marks of dy (and of x): the same
    bits as from small tensors."""
    say("near 4 GiB")
    rng = np.random.default_rng(9)
    M, N, n = 524000, 4096, 300                          # 4292608000 bytes
    small = dev_vals(heavy_bf16(rng, (n, N)))
    big = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    rows = torch.from_numpy(np.sort(rng.choice(M, n, replace=False))).cuda()
    rows[-1], rows[0] = M - 1, 0
    big[rows] = small
    order = torch.from_numpy(rng.permutation(n)).cuda()
    offs = cu(np.array([0, 20, 300], np.int32))
    far, near = rows[order].int(), order.int()
    w = F.nvfp4_qdq_weights(dev_vals(OF.round_to_bf16(rng.standard_normal((2, N, 128)) * 0.02)),
                            want_qdq=False)
    W = (w.packed_codes, w.packed_scales, w.g)
    for M_total in (300, 20):                            # both kernels
        o = offs.clamp(max=M_total)
        a = F.grouped_w4a16_dgrad(big, far, *W, o, M_total=M_total)
        b = F.grouped_w4a16_dgrad(small, near, *W, o, M_total=M_total)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    other = dev_vals(heavy_bf16(rng, (n, 64)))
    for dy, dyr, dys, dysr, x, xr, xs, xsr in [(big, far, small, near, other, None, other, None),
                                               (other, None, other, None, big, far, small, near)]:
        a = F.grouped_wgrad(dy, dyr, x, xr, offs)
        b = F.grouped_wgrad(dys, dysr, xs, xsr, offs)
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_wgrad_no_rows(dev):
    say("wgrad no rows")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    dw = F.grouped_wgrad(e, None, e, None, offs)
    torch.cuda.synchronize()
    assert dw.shape == (3, 64, 64) and not dw.any()


# ------------------------------------------------------------- SwiGLU backward
def swiglu_limits(y, dh, inv, w, ref):
    """Relative error of s = 1 / (1 + e^-g) in float32: the argument's rounding
    moves e^-g by |g| 2^-23 and its two products, the hardware exp2 and the
    reciprocal by an ulp each: r = (|g| + 8) 2^-23; each further step 2^-24.
    The two terms of dgate may cancel, so their magnitudes are what counts."""
    P, I = dh.shape
    g, u = y[:, :I], y[:, I:]
    r = (np.abs(g) + 16) * 2.0 ** -23
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    wr = np.ones((P, 1))
    if w is not None:
        wr[inv.reshape(-1), 0] = w.reshape(-1)
    d = np.abs(wr * dh)
    dy, hw, dw = ref
    h = np.abs(g * s * u)
    flush = TINY * (1 + d * (1 + np.abs(u)) * (1 + np.abs(g)))     # s below the normal range
    lim_g = 2.0 ** -8 * np.abs(dy[:, :I]) + d * np.abs(u) * s * (1 + np.abs(g) * t) * 2 * r + flush
    lim_u = 2.0 ** -8 * np.abs(dy[:, I:]) + d * np.abs(g) * s * r + flush
    lim_h = 2.0 ** -8 * np.abs(hw) + np.abs(hw) * r + TINY * (1 + np.abs(g * u))
    lim_w = (np.abs(dh) * h * (r + I * U)).sum(1) + TINY * (1 + np.abs(dh * g * u)).sum(1)
    return np.concatenate([lim_g, lim_u], 1), lim_h, lim_w[inv]


@pytest.mark.parametrize("T,tk,I,fp8", [
    (1, 1, 8, False), (1, 1, 32, True), (5, 3, 40, False), (33, 2, 768, True), (64, 8, 512, False),
    (3, 1, 8200, False), (2, 4, 4128, True), (300, 4, 1536, True), (1, 32, 64, True)])
def test_swiglu_backward(dev, T, tk, I, fp8):
    say(f"swiglu backward T={T} tk={tk} I={I} fp8={fp8}")
    rng = np.random.default_rng(T + tk + I)
    P = T * tk
    y = OF.round_to_bf16(rng.standard_normal((P, 2 * I)) * 4)
    if T > 1:
        y[0, :8] = [60.0, -60.0, 90.0, -90.0, 130.0, -130.0, 0.0, -0.0]
        y[0, I:I + 8] = [1.0, 2.0, -3.0, 4.0, 5.0, 6.0, 7.0, 8.0]
    dh = OF.round_to_bf16(rng.standard_normal((P, I)) * 2.0 ** -9)
    inv = rng.permutation(P).reshape(T, tk).astype(np.int32)
    w = rng.random((T, tk)).astype(np.float32)
    w[0, 0] = 0.0
    yd, ys = dev_vals(y), None
    if fp8:
        codes, scales = OT.mxfp8_encode(y)
        y, yd, ys = OT.mxfp8_value(codes, scales), cu(codes), cu(scales)
    dy, hw, dw = F.moe_swiglu_backward(yd, dev_vals(dh), cu(inv), cu(w), y_scales=ys)
    torch.cuda.synchronize()
    ref = OT.swiglu_backward(y, dh, inv, w)
    lims = swiglu_limits(y, dh, inv, w, ref)
    check(host_vals(dy), ref[0], lims[0], "dy")
    check(host_vals(hw), ref[1], lims[1], "hw")
    check(dw.cpu().numpy().astype(np.float64), ref[2], lims[2], "d_topk_w")
    # without the optional parts: the same dy
    dy2, none, _ = F.moe_swiglu_backward(yd, dev_vals(dh), cu(inv), cu(w), y_scales=ys, want_h=False)
    assert none is None and torch.equal(dy2.view(torch.int16), dy.view(torch.int16))


def test_swiglu_backward_dense(dev):
    say("swiglu backward dense")
    rng = np.random.default_rng(11)
    y, dh = heavy_bf16(rng, (45, 192)), heavy_bf16(rng, (45, 96))
    dy, hw, dw = F.moe_swiglu_backward(dev_vals(y), dev_vals(dh))
    torch.cuda.synchronize()
    assert dw is None
    ref = OT.swiglu_backward(y, dh, None, None)
    lims = swiglu_limits(y, dh, np.arange(45)[:, None], None, ref)
    check(host_vals(dy), ref[0], lims[0], "dy")
    check(host_vals(hw), ref[1], lims[1], "hw")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert F.moe_swiglu_backward(e, e[:, :32])[0].shape == (0, 64)


# ------------------------------------------------------------------ the chain
def block(rng, T, H, E, tk, I):
    x = OF.round_to_bf16(rng.standard_normal((T, H)))
    w1 = OF.round_to_bf16(rng.standard_normal((E, 2 * I, H)) * 0.05)
    w2 = OF.round_to_bf16(rng.standard_normal((E, H, I)) * 0.05)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    d_out = OF.round_to_bf16(rng.standard_normal((T, H)) * 2.0 ** -8)
    return x, w1, w2, logits, d_out


@pytest.mark.parametrize("ckpt", ["mxfp8", "bf16"])
@pytest.mark.parametrize("T,H,E,tk,I", [(70, 256, 4, 2, 128), (3, 128, 8, 2, 128),
                                        (600, 256, 3, 1, 384)])
def test_block_training_step(dev, T, H, E, tk, I, ckpt):
    """Forward and backward as a user runs them; every stage of the backward
    pass against the oracle on the stage's own GPU inputs, and the gradients of
    the whole step against the float64 block."""
    say(f"train step T={T} H={H} E={E} tk={tk} I={I} {ckpt}")
    rng = np.random.default_rng(T + H)
    x, w1, w2, logits, d_out = block(rng, T, H, E, tk, I)
    q1, q2 = pipeline.prepare_weights(dev_vals(w1)), pipeline.prepare_weights(dev_vals(w2))
    out, st = pipeline.moe_train_forward(dev_vals(x), cu(logits), tk, q1, q2, checkpoint=ckpt)
    dd = dev_vals(d_out)
    g = pipeline.moe_train_backward(st, dd)
    torch.cuda.synchronize()

    ids, tw = OM.route(logits, tk)
    offs, perm, inv = OM.permute(ids, E)
    c1, s1, g1, _ = OQ.qdq_weights(w1)
    c2, s2, g2, _ = OQ.qdq_weights(w2)
    y1 = OG.grouped_gemm_w4a16(x, perm, c1, s1, g1, offs)
    h = OM.swiglu(y1, I)
    o = OM.combine(OG.grouped_gemm_w4a16(h, None, c2, s2, g2, offs), inv, tw)
    # a bf16 rounding at each of four stages, in norm
    assert np.linalg.norm(host_vals(out) - o) <= 4 * 2.0 ** -8 * np.linalg.norm(o)

    kept = host_vals(F.mxfp8_restore(st.y1, st.y1_scales)) if ckpt == "mxfp8" else host_vals(st.y1)
    kx = host_vals(F.mxfp8_restore(st.x, st.x_scales)) if ckpt == "mxfp8" else host_vals(st.x)
    if ckpt == "mxfp8":
        assert np.array_equal(kx, OT.mxfp8_value(*OT.mxfp8_encode(x)))
    dh, _ = OT.grouped_dgrad(d_out, perm, c2, s2, g2, offs)
    dy1, hw, dtw = OT.swiglu_backward(kept, dh, inv, tw)
    ref = dict(dw_down=OT.grouped_wgrad(d_out, perm, hw, None, offs)[0],
               dw_first=OT.grouped_wgrad(dy1, None, kx, perm, offs)[0],
               dx=OT.grouped_dgrad(dy1, None, c1, s1, g1, offs)[0][inv].sum(1), d_topk_w=dtw)
    # at most four bf16 roundings on the way to any output (dh, dy1, dxp, dx),
    # each 2^-8 of its element at most: in norm, 4 * 2^-8, and twice that for
    # their passing through sums whose terms differ in size
    for k, r in ref.items():
        v = host_vals(g[k]) if g[k].dtype == torch.bfloat16 else g[k].cpu().numpy()
        err = np.linalg.norm(v - r) / np.linalg.norm(r)
        say(f"   {k}: {err:.2e}")
        assert err <= 8 * 2.0 ** -8, k

    # gradient accumulation: a second backward adds the same numbers
    a1, a2 = g["dw_first"].clone(), g["dw_down"].clone()
    pipeline.moe_train_backward(st, dd, dw_first=a1, dw_down=a2)
    torch.cuda.synchronize()
    assert torch.equal(a1, 2 * g["dw_first"]) and torch.equal(a2, 2 * g["dw_down"])


def test_training_step_without_tokens(dev):
    say("train step T=0")
    rng = np.random.default_rng(1)
    _, w1, w2, _, _ = block(rng, 1, 128, 2, 1, 128)
    q1, q2 = pipeline.prepare_weights(dev_vals(w1)), pipeline.prepare_weights(dev_vals(w2))
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    out, st = pipeline.moe_train_forward(x, torch.empty((0, 2), device="cuda"), 1, q1, q2)
    g = pipeline.moe_train_backward(st, x)
    torch.cuda.synchronize()
    assert out.shape == g["dx"].shape == (0, 128) and g["d_topk_w"].shape == (0, 1)
    assert not g["dw_first"].any() and not g["dw_down"].any()


def test_training_step_graph_replays_match_eager(dev):
    """Forward and backward captured as one graph; every replay, with eager
    calls between, gives the eager bits, also for new inputs in place."""
    say("train graph")
    rng = np.random.default_rng(21)
    T, H, E, tk, I = 150, 256, 4, 2, 128
    x, w1, w2, logits, d_out = block(rng, T, H, E, tk, I)
    q1, q2 = pipeline.prepare_weights(dev_vals(w1)), pipeline.prepare_weights(dev_vals(w2))
    xs, lg, dd = dev_vals(x), cu(logits), dev_vals(d_out)

    def step():
        out, st = pipeline.moe_train_forward(xs, lg, tk, q1, q2)
        g = pipeline.moe_train_backward(st, dd)
        return [out, g["dx"], g["dw_first"], g["dw_down"], g["d_topk_w"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        if i == 2:                                       # other data, other routing
            x2, _, _, l2, d2 = block(rng, T, H, E, tk, I)
            xs.copy_(dev_vals(x2)), lg.copy_(cu(l2)), dd.copy_(dev_vals(d2))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}"


def test_two_streams_at_once(dev):
    """The calls on two streams of their own at once, each with its own
    buffers: the bits of the calls alone."""
    say("two streams")
    rng = np.random.default_rng(22)
    sets = []
    for k in range(2):
        x, w1, w2, logits, d_out = block(rng, 300, 256, 4, 2, 128)
        sets.append((dev_vals(x), pipeline.prepare_weights(dev_vals(w1)),
                     pipeline.prepare_weights(dev_vals(w2)), cu(logits), dev_vals(d_out)))

    def step(s):
        out, st = pipeline.moe_train_forward(s[0], s[3], 2, s[1], s[2])
        g = pipeline.moe_train_backward(st, s[4])
        return [out, g["dx"], g["dw_first"], g["dw_down"], g["d_topk_w"]]

    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, q in zip(sets, streams):
            with torch.cuda.stream(q):
                got.append(step(s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_binding_refusals(dev):
    b = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    wq = F.nvfp4_qdq_weights(torch.ones((1, 64, 128), dtype=torch.bfloat16, device="cuda"))
    W = (wq.packed_codes, wq.packed_scales, wq.g)
    rows = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(F.NvfpError, match="bfloat16"):
        F.mxfp8_checkpoint(b.float())
    with pytest.raises(F.NvfpError, match="shape"):
        F.mxfp8_restore(b.view(torch.uint8)[:, :64].contiguous(), b.view(torch.uint8))
    with pytest.raises(F.NvfpError, match="shape"):
        F.grouped_w4a16_dgrad(b[:, :32].contiguous(), None, *W, offs)
    with pytest.raises(F.NvfpError, match="int32"):
        F.grouped_w4a16_dgrad(b, rows.long(), *W, offs)
    with pytest.raises(F.NvfpError, match="shape"):
        F.grouped_w4a16_dgrad(b, None, *W, rows)
    with pytest.raises(F.NvfpError, match="shorter"):
        F.grouped_w4a16_dgrad(b, rows, *W, offs, M_total=5)
    with pytest.raises(F.NvfpError, match="M_src"):
        F.grouped_w4a16_dgrad(b, None, *W, offs, M_total=5)
    with pytest.raises(F.NvfpError, match="negative"):
        F.grouped_w4a16_dgrad(b, rows, *W, offs, M_total=-1)
    with pytest.raises(F.NvfpError, match="contiguous"):
        F.grouped_w4a16_dgrad(torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")[:, ::2],
                              None, *W, offs)
    with pytest.raises(F.NvfpError, match="accumulate"):
        F.grouped_wgrad(b, None, b, None, offs, accumulate=True)
    with pytest.raises(F.NvfpError, match="float32"):
        F.grouped_wgrad(b, None, b, None, offs, accumulate=True,
                        out=torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(F.NvfpError, match="float16"):
        F.grouped_wgrad(b, None, b, None, offs, dtype=torch.float16)
    with pytest.raises(F.NvfpError, match="shape"):
        F.grouped_wgrad(b, None, b, None, offs,
                        out=torch.zeros((2, 64, 64), dtype=torch.float32, device="cuda"))
    with pytest.raises(F.NvfpError, match="one entry"):
        F.moe_swiglu_backward(b, b[:, :32].contiguous(), rows[:2].view(1, 2))
    with pytest.raises(F.NvfpError, match="shape"):
        F.moe_swiglu_backward(b, b)


def test_gradients_of_operands_of_the_last_size(dev):
    """The largest dy and x below 4 GiB whose rows do not divide it: the last
    row gathered, rows and columns past an edge still read as zeros."""
    rng = np.random.default_rng(31)
    n = 40
    offs = cu(np.array([0, 13, 13, 40], np.int32))

    def far_rows(M):
        rows = torch.from_numpy(np.sort(rng.choice(M, n, replace=False))).cuda()
        rows[-1], rows[0] = M - 1, 0
        order = torch.from_numpy(rng.permutation(n)).cuda()
        return rows, rows[order].int(), order.int()

    N, M = 48, 44739242                                  # 64 bytes below
    say(f"dgrad dy of {M * N * 2} bytes")
    rows, far, near = far_rows(M)
    small = dev_vals(heavy_bf16(rng, (n, N)))
    big = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[rows] = small
    w = F.nvfp4_qdq_weights(dev_vals(OF.round_to_bf16(rng.standard_normal((3, N, 192)) * 0.02)),
                            want_qdq=False)
    W = (w.packed_codes, w.packed_scales, w.g)
    for extra in (0, 60):                                # both kernels, by the rows allowed for
        f, m = (torch.cat([t, t[:1].expand(extra)]) for t in (far, near))
        a = F.grouped_w4a16_dgrad(big, f, *W, offs)
        b = F.grouped_w4a16_dgrad(small, m, *W, offs)
        assert torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16))
        assert bool(torch.isfinite(a[:n].float()).all())
    del big

    C, M = 24, 89478485                                  # 16 bytes below
    say(f"wgrad operand of {M * C * 2} bytes")
    rows, far, near = far_rows(M)
    small = dev_vals(heavy_bf16(rng, (n, C)))
    big = torch.full((M, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[rows] = small
    other = dev_vals(heavy_bf16(rng, (n, 64)))
    for args, ref in [((big, far, other, None), (small, near, other, None)),
                      ((other, None, big, far), (other, None, small, near))]:
        a, b = F.grouped_wgrad(*args, offs), F.grouped_wgrad(*ref, offs)
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
        assert bool(torch.isfinite(a).all())


@pytest.mark.parametrize("ckpt", ["mxfp8", "bf16"])
@pytest.mark.parametrize("T,H,E,tk,I", [(70, 256, 4, 2, 128), (3, 128, 8, 2, 128), (1, 128, 2, 1, 128),
                                        (600, 256, 3, 1, 384), (150, 384, 40, 8, 256)])
def test_block_backward_stage_by_stage(dev, T, H, E, tk, I, ckpt):
    """Each call of moe_train_backward against the oracle on that call's own
    GPU inputs, element by element; the step returns the bits of the calls made
    one by one.  No token takes expert 1."""
    say(f"stages T={T} H={H} E={E} tk={tk} I={I} {ckpt}")
    rng = np.random.default_rng(T + H + E)
    x, w1, w2, logits, d_out = block(rng, T, H, E, tk, I)
    logits[:, 1] = -100.0
    q1, q2 = pipeline.prepare_weights(dev_vals(w1)), pipeline.prepare_weights(dev_vals(w2))
    _, st = pipeline.moe_train_forward(dev_vals(x), cu(logits), tk, q1, q2, checkpoint=ckpt)
    dd = dev_vals(d_out)
    W1, W2 = [(q.packed_codes, q.packed_scales, q.g) for q in (q1, q2)]
    P, perm, o = T * tk, st.perm_token, st.offsets
    dh = F.grouped_w4a16_dgrad(dd, perm, *W2, o, M_total=P)
    dy1, hw, dtw = F.moe_swiglu_backward(st.y1, dh, st.inv_perm, st.topk_w, y_scales=st.y1_scales)
    dw2 = F.grouped_wgrad(dd, perm, hw, None, o, M_total=P)
    dw1 = F.grouped_wgrad(dy1, None, st.x, perm, o, x_scales=st.x_scales, M_total=P)
    dxp = F.grouped_w4a16_dgrad(dy1, None, *W1, o, M_total=P)
    g = pipeline.moe_train_backward(st, dd)
    torch.cuda.synchronize()

    offs, rows, inv = (t.cpu().numpy() for t in (o, perm, st.inv_perm))
    w = st.topk_w.cpu().numpy()
    assert offs[1] == offs[2] and offs[-1] == P
    c1, s1, g1, _ = OQ.qdq_weights(w1)
    c2, s2, g2, _ = OQ.qdq_weights(w2)
    mx = ckpt == "mxfp8"
    kx = host_vals(F.mxfp8_restore(st.x, st.x_scales) if mx else st.x)
    ky = host_vals(F.mxfp8_restore(st.y1, st.y1_scales) if mx else st.y1)
    dhv, dyv, hv, dxv = (host_vals(t) for t in (dh, dy1, hw, dxp))

    check_dgrad(dhv, *OT.grouped_dgrad(d_out, rows, c2, s2, g2, offs), H, "dh")
    ref = OT.swiglu_backward(ky, dhv, inv, w)
    lims = swiglu_limits(ky, dhv, inv, w, ref)
    for got, r, lim, what in zip((dyv, hv, dtw.cpu().numpy().astype(np.float64)), ref, lims,
                                 ("dy1", "hw", "d_topk_w")):
        check(got, r, lim, what)
    n = int(np.diff(offs).max())
    for got, (r, mag), what in ((dw2, OT.grouped_wgrad(d_out, rows, hv, None, offs), "dw_down"),
                                (dw1, OT.grouped_wgrad(dyv, None, kx, rows, offs), "dw_first")):
        check(got.cpu().numpy().astype(np.float64), r, n * U * mag + TINY, what)
        assert not got[1].any()
    check_dgrad(dxv, *OT.grouped_dgrad(dyv, None, c1, s1, g1, offs), 2 * I, "dxp")
    terms = dxv[inv]
    r = terms.sum(1)
    check(host_vals(g["dx"]), r, np.abs(r) * 2.0 ** -8 + (tk + 1) * U * np.abs(terms).sum(1) + TINY, "dx")
    for a, b in ((g["dw_down"], dw2), (g["dw_first"], dw1), (g["d_topk_w"], dtw)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def nvfp4_values(q):
    """float64 weights [E][N][K], g included, of QdqWeights on the device."""
    E, N, half = q.codes.shape
    c = torch.stack([q.codes & 15, q.codes >> 4], 3).view(E, N, 2 * half).long()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.cat([grid, -grid])[c]
    s = q.scales.view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, 2) * q.g.double()[:, None, None]


@pytest.mark.parametrize("counts", [[2, 1], [37, 63]])
@pytest.mark.parametrize("N,K", [(16, 1 << 20), (1 << 20, 64)])
def test_dgrad_widest(dev, N, K, counts):
    """N and K at their limit, on the few-row and the tiled kernel."""
    say(f"dgrad widest N={N} K={K} {counts}")
    gen = torch.Generator(device="cuda").manual_seed(N + counts[0])
    q = F.nvfp4_qdq_weights(torch.randn(2, N, K, device="cuda", generator=gen).bfloat16() * 0.02,
                            want_qdq=False)
    offs = offsets_of(counts)
    P = int(offs[-1])
    dy = torch.randn(P, N, device="cuda", generator=gen).bfloat16()
    dx = F.grouped_w4a16_dgrad(dy, None, q.packed_codes, q.packed_scales, q.g, cu(offs))
    w = nvfp4_values(q)
    for e in range(2):
        d, got = dy[offs[e]:offs[e + 1]].double(), dx[offs[e]:offs[e + 1]].double()
        ref, mag = d @ w[e], d.abs() @ w[e].abs()
        assert bool(((got - ref).abs() <= ref.abs() * 2.0 ** -8 + (N + 2) * U * mag + TINY).all())


@pytest.mark.parametrize("N,K", [(1 << 20, 8), (8, 1 << 20), (32768, 32760)])
def test_wgrad_widest(dev, N, K):
    """N and K at their limit, and a dw of 1 MiB less than 4 GiB."""
    say(f"wgrad widest N={N} K={K}")
    gen = torch.Generator(device="cuda").manual_seed(N)
    dy = torch.randn(5, N, device="cuda", generator=gen).bfloat16()
    x = torch.randn(5, K, device="cuda", generator=gen).bfloat16()
    offs = cu(np.array([0, 5], np.int32))
    dw = F.grouped_wgrad(dy, None, x, None, offs)
    db = F.grouped_wgrad(dy, None, x, None, offs, dtype=torch.bfloat16)
    acc = F.grouped_wgrad(dy, None, x, None, offs, out=torch.ones_like(dw), accumulate=True)
    for lo in range(0, N, 4096):                         # (float64 of all of it is 8 GiB)
        d = dy[:, lo:lo + 4096].double().t().contiguous()
        ref, lim = d @ x.double(), 5 * U * (d.abs() @ x.double().abs()) + TINY
        got, gb, ga = (t[0, lo:lo + 4096].double() for t in (dw, db, acc))
        assert bool(((got - ref).abs() <= lim).all())
        assert bool(((gb - ref).abs() <= ref.abs() * 2.0 ** -8 + lim).all())
        assert bool(((ga - ref - 1).abs() <= lim + U * ((ref + 1).abs() + lim)).all())


@pytest.mark.parametrize("glu", [False, True])
def test_checkpoint_of_more_than_2_31_chunks(dev, glu):
    """64-bit chunk numbers: a few rows among zeros get the codes they get by
    themselves."""
    K = 65536
    M = ((1 << 35 if glu else 1 << 34) // K) + 3
    torch.cuda.empty_cache()
    need = M * K * 2 * 5 // 2 + (1 << 34)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    say(f"checkpoint of {M} rows of {K}, glu={glu}")
    rows = torch.tensor([0, 1, M // 2, M - 4, M - 3, M - 2, M - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    small = torch.randn(7, K, device="cuda", generator=gen).bfloat16()
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[rows] = small
    a, b = F.mxfp8_checkpoint(x, glu=glu), F.mxfp8_checkpoint(small, glu=glu)

    def written(t):
        return int(t.view(torch.int64).ne(0).any(1).sum())
    assert torch.equal(a["codes"][rows], b["codes"]) and written(a["codes"]) == 7
    assert torch.equal(a["scales"][rows], b["scales"])
    if glu:
        assert torch.equal(a["h"][rows], b["h"]) and written(a["h"]) == 7
    else:
        F.mxfp8_restore(a["codes"], a["scales"], out=x.fill_(float("nan")))
        assert torch.equal(x[rows], F.mxfp8_restore(b["codes"], b["scales"])) and written(x) == 7
    del x, a, b
    torch.cuda.empty_cache()
