"""GPU parity of the MXFP4 calls (quantizer, values, expert-grouped product)
against the float64 oracle.

Tolerances, from the arithmetic.  Codes, scales and restored values are exact.
A product of two MXFP4 elements and their scales is exact in float32; a sum of
K of them adds at most K - 1 times, each addition off by at most one step of
float32, 2^-23 of what it holds (whichever way it rounds), which is at most the
sum of magnitudes: K * 2^-23 of it.  An output rounded to bf16 adds half a
step, 2^-8 of its value."""
import sys

import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from oracle import formats as OF
from oracle import mxfp4 as OX
from tests.gpu_util import heavy_bf16, host_bits, host_vals, to_dev_bf16

pytestmark = pytest.mark.gpu


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


# ---------------------------------------------------------------- quantizer
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (64, 512), (129, 96), (37, 4096), (5, 32768)])
def test_quantize_and_restore(dev, M, K):
    say(f"mxfp4 M={M} K={K}")
    rng = np.random.default_rng(M + K)
    x = heavy_bf16(rng, (M, K))
    x[0, :32] = 0.0
    x[-1, -3:] = [7.0, -7.25, 2.0 ** -130]
    c, s = F.mxfp4_quantize(dev_vals(x))
    y = F.mxfp4_restore(c, s)
    torch.cuda.synchronize()
    codes, scales = OX.encode(x)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(host_vals(y), OX.value(codes, scales))


def every_bf16():
    """Every bf16 bit pattern, each as the largest of a block and as a small
    one beside 7, 7.03 and the largest value; NaN and infinities among them."""
    bits = np.arange(65536, dtype=np.uint16)
    x = np.zeros((4 * 65536, 32), dtype=np.uint16)
    x[:, 7] = np.tile(bits, 4)
    x[:, 20] = np.repeat(np.array([0x0000, 0x40E0, 0x40E1, 0x7F7F], dtype=np.uint16), 65536)
    return x


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_every_bf16(dev, transpose):
    say(f"mxfp4 every bf16 transpose={transpose}")
    x = every_bf16()
    xd = to_dev_bf16(x)
    c, s = F.mxfp4_quantize(xd.t().contiguous(), transpose=True) if transpose else F.mxfp4_quantize(xd)
    y = F.mxfp4_restore(c, s)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        vals = OF.bf16_bits_to_f64(x)
    codes, scales = OX.encode(vals)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(c.cpu().numpy(), codes)
    back, want = host_vals(y), OX.value(codes, scales)
    assert np.array_equal(np.isnan(back), np.isnan(want))
    assert np.array_equal(back[~np.isnan(want)], want[~np.isnan(want)])


def test_restore_every_scale(dev):
    """Every E8M0 byte with every code, where bf16 holds the value."""
    say("mxfp4 restore every scale")
    codes = np.tile(np.arange(16, dtype=np.uint8) | (np.arange(16, dtype=np.uint8)[::-1] << 4), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    y = F.mxfp4_restore(cu(codes), cu(scales))
    torch.cuda.synchronize()
    want = OX.value(codes, scales)
    got = host_vals(y)
    assert np.isnan(got[255]).all()
    with np.errstate(over="ignore"):
        want = OF.round_to_bf16(want[:255])
    assert np.array_equal(got[:255], want)


def test_strided_rows(dev):
    say("mxfp4 strided")
    rng = np.random.default_rng(3)
    wide = dev_vals(heavy_bf16(rng, (64, 320)))
    x = wide[:, 64:288]
    for tr in (False, True):
        c, s = F.mxfp4_quantize(x, transpose=tr)
        d, t = F.mxfp4_quantize(x.contiguous(), transpose=tr)
        assert torch.equal(c, d) and torch.equal(s, t)
    c, s = F.mxfp4_quantize(x)
    out = torch.full((64, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    F.mxfp4_restore(c, s, out=out[:, 64:288])
    torch.cuda.synchronize()
    assert torch.equal(out[:, 64:288], F.mxfp4_restore(c, s))
    assert bool((out[:, :64] == 7).all()) and bool((out[:, 288:] == 7).all())
    with pytest.raises(F.NvfpError):
        F.mxfp4_quantize(wide[:, 4:292])                 # 8-byte aligned rows only
    with pytest.raises(F.NvfpError):
        F.mxfp4_quantize(wide.t())


@pytest.mark.parametrize("E,M,K", [(1, 32, 8), (3, 64, 72), (2, 288, 136), (5, 512, 64), (0, 32, 64)])
def test_quantize_transposed_is_the_transposes(dev, E, M, K):
    say(f"mxfp4 transposed E={E} M={M} K={K}")
    rng = np.random.default_rng(E + M + K)
    x = heavy_bf16(rng, (E, M, K))
    c, s = F.mxfp4_quantize(dev_vals(x), transpose=True)
    assert c.shape == (E, K, M // 2) and s.shape == (E, K, M // 32)
    torch.cuda.synchronize()
    for e in range(E):
        codes, scales = OX.encode(x[e].T)
        assert np.array_equal(s[e].cpu().numpy(), scales)
        assert np.array_equal(c[e].cpu().numpy(), codes)
    if E:
        c2, s2 = F.mxfp4_quantize(dev_vals(x[0]), transpose=True)
        assert torch.equal(c2, c[0]) and torch.equal(s2, s[0])


def test_quantize_stacked_and_empty(dev):
    rng = np.random.default_rng(5)
    x = heavy_bf16(rng, (3, 16, 64))
    c, s = F.mxfp4_quantize(dev_vals(x))
    assert c.shape == (3, 16, 32) and s.shape == (3, 16, 2)
    codes, scales = OX.encode(x.reshape(48, 64))
    assert np.array_equal(c.cpu().numpy().reshape(48, 32), codes)
    assert np.array_equal(s.cpu().numpy().reshape(48, 2), scales)
    assert np.array_equal(host_vals(F.mxfp4_restore(c, s)).reshape(48, 64), OX.value(codes, scales))
    c, s = F.mxfp4_quantize(dev_vals(np.zeros((0, 64))))
    assert c.shape == (0, 32) and F.mxfp4_restore(c, s).shape == (0, 64)


# ---------------------------------------------------------------- product
def operands(rng, M_src, E, N, K):
    ac, asc = OX.encode(heavy_bf16(rng, (M_src, K)))
    wc, wsc = OX.encode(OF.round_to_bf16(rng.standard_normal((E * N, K)) * 0.02))
    return ac, asc, wc.reshape(E, N, K // 2), wsc.reshape(E, N, K // 32)


def limits(y, mag, K):
    return K * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(y) + 2.0 ** -126


def swiglu_limits(y, mag, K):
    """silu(g) u for sums off by d = K 2^-23 mag: |silu'| <= 1.1; the hardware's
    exp2 and reciprocal and the products are good to 2^-21, and the exponent's
    argument is rounded to 2^-24 of itself, 1.45 |g| 2^-24 of the result; one
    rounding to bf16."""
    g, u = np.split(y, 2, axis=1)
    dg, du = np.split(K * 2.0 ** -23 * mag, 2, axis=1)
    h = OX.swiglu(y)
    rel = 2.0 ** -21 + 1.45 * np.abs(g) * 2.0 ** -24
    d = 1.1 * np.abs(u) * dg + (np.abs(g) + 1.1 * dg) * du + rel * np.abs(h)
    return d + 2.0 ** -8 * (np.abs(h) + d) + 2.0 ** -120 * (1 + np.abs(u))


COUNTS = [
    ([1], 16, 128), ([64], 512, 512), ([3, 0, 17], 48, 384), ([0, 0, 5], 272, 640),
    ([33, 1, 0, 100], 160, 1664), ([255], 80, 256), ([256, 257, 1], 256, 896),
    ([700, 0, 31, 300], 544, 512), ([1, 2, 0, 0, 1, 3, 16, 8], 1024, 1536),
    ([40] * 6, 96, 4096), ([129, 128, 127], 288, 1152), ([2000], 32, 128),
]


@pytest.mark.parametrize("counts,N,K", COUNTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_gemm(dev, counts, N, K, gather, glu):
    if glu and N % 32:
        N += 16
    say(f"mxfp4 gemm counts={counts} N={N} K={K} gather={gather} glu={glu}")
    rng = np.random.default_rng(sum(counts) + N + K)
    offs = offsets_of(counts)
    P, E = int(offs[-1]), len(counts)
    M_src = max(1, P // 2) if gather else P
    rows = rng.integers(0, M_src, P).astype(np.int32) if gather else None
    ac, asc, wc, wsc = operands(rng, M_src, E, N, K)
    # three rows more than the experts have: left as they were
    cols = N // 2 if glu else N
    out = torch.full((P + 3, cols), 3.0, dtype=torch.bfloat16, device="cuda")
    pad = None if rows is None else cu(np.concatenate([rows, [0, 0, 0]]).astype(np.int32))
    if not gather:
        ac, asc = np.concatenate([ac, ac[:1], ac[:1], ac[:1]]), np.concatenate([asc, asc[:1], asc[:1], asc[:1]])
    call = F.grouped_mxfp4_gemm_swiglu if glu else F.grouped_mxfp4_gemm
    got = call(cu(ac), cu(asc), pad, cu(wc), cu(wsc), cu(offs), M_total=P + 3, out=out)
    torch.cuda.synchronize()
    a = OX.value(ac, asc)
    w = OX.value(wc.reshape(E * N, -1), wsc.reshape(E * N, -1)).reshape(E, N, K)
    y, mag = OX.grouped_gemm(a, rows, w, offs)
    g = host_vals(got)
    assert np.all(g[P:] == 3.0)
    if glu:
        check(g[:P], OX.swiglu(y), swiglu_limits(y, mag, K), "h")
    else:
        check(g[:P], y, limits(y, mag, K), "y")
        assert np.mean(g[:P] == OF.round_to_bf16(y)) >= 0.95


def test_gemm_scales_far_apart(dev):
    """Scales from 2^-60 to 2^60 in either operand: their product's exponent
    and the sums stay in float32's range, no scale is lost or swapped."""
    say("mxfp4 gemm scales")
    rng = np.random.default_rng(11)
    M, N, K = 40, 64, 512
    ac = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
    wc = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    asc = (127 + rng.integers(-60, 61, (M, K // 32))).astype(np.uint8)
    wsc = (127 + rng.integers(-60, 61, (1, N, K // 32))).astype(np.uint8)
    y = F.grouped_mxfp4_gemm(cu(ac), cu(asc), None, cu(wc), cu(wsc), cu(np.array([0, M], np.int32)))
    torch.cuda.synchronize()
    ref, mag = OX.grouped_gemm(OX.value(ac, asc), None, OX.value(wc[0], wsc[0])[None], [0, M])
    check(host_vals(y), ref, limits(ref, mag, K), "y")


@pytest.mark.parametrize("M", [5, 300])
def test_gemm_nan_stays_in_its_row_and_column(dev, M):
    """A NaN block makes its row (activation) or column (weight) NaN and no
    other: neither in the same tile nor, for the row's end, in the next row."""
    say(f"mxfp4 gemm nan M={M}")
    rng = np.random.default_rng(M)
    N, K = 80, 640
    ac, asc, wc, wsc = operands(rng, M, 1, N, K)
    asc[2, -1], ac[2, -16:] = 255, 0x77
    asc[4, 0] = 255                                      # whatever the codes are
    wsc[0, 7, 3], wc[0, 7, 48:64] = 255, 0x77
    y = F.grouped_mxfp4_gemm(cu(ac), cu(asc), None, cu(wc), cu(wsc), cu(np.array([0, M], np.int32)))
    torch.cuda.synchronize()
    nan = np.isnan(host_vals(y))
    want = np.zeros((M, N), dtype=bool)
    want[2] = want[4] = want[:, 7] = True
    assert np.array_equal(nan, want)


def test_gemm_of_quantized_tensors_and_input_gradient(dev):
    """The calls as they are used: quantized activation and weights, and the
    input gradient through the transposed weights."""
    say("mxfp4 gemm and dgrad")
    rng = np.random.default_rng(8)
    counts, N, K = [70, 0, 130], 256, 384
    offs = offsets_of(counts)
    P, E = int(offs[-1]), 3
    x, w, dy = heavy_bf16(rng, (P, K)), OF.round_to_bf16(rng.standard_normal((E, N, K))), \
        OF.round_to_bf16(rng.standard_normal((P, N)) * 1e-3)
    od = cu(offs)
    y = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(dev_vals(x)), None, *F.mxfp4_quantize(dev_vals(w)), od)
    dx = F.grouped_mxfp4_gemm(*F.mxfp4_quantize(dev_vals(dy)), None,
                              *F.mxfp4_quantize(dev_vals(w), transpose=True), od)
    torch.cuda.synchronize()
    q = lambda v: OX.value(*OX.encode(v))                # noqa: E731
    ref, mag = OX.grouped_gemm(q(x), None, np.stack([q(m) for m in w]), offs)
    check(host_vals(y), ref, limits(ref, mag, K), "y")
    ref, mag = OX.grouped_gemm(q(dy), None, np.stack([q(m.T) for m in w]), offs)
    check(host_vals(dx), ref, limits(ref, mag, N), "dx")


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 768, 896, 1024, 1664, 4096, 4224, 4352, 4480])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("glu", [False, True])
def test_many_tiles_per_workgroup(dev, K, gather, glu):
    """More tiles than four rounds of the device's workgroups take (from K = 4096:
    taken as they get free), for every
    number of steps at a row's end, against the float64 product."""
    say(f"mxfp4 many tiles K={K} gather={gather} glu={glu}")
    g = torch.Generator("cuda").manual_seed(K)
    counts = [3000, 1, 70, 2500, 0, 130]
    N, E, P = 12288, len(counts), sum(counts)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    M_src = 4000 if gather else P
    a, w = F.mxfp4_quantize(rand(M_src, K)), F.mxfp4_quantize(rand(E, N, K))
    rows = torch.randint(0, M_src, (P,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    call = F.grouped_mxfp4_gemm_swiglu if glu else F.grouped_mxfp4_gemm
    got = call(*a, rows, *w, cu(offsets_of(counts)))
    av, wv = F.mxfp4_restore(*a).double(), F.mxfp4_restore(*w).double()
    offs = offsets_of(counts)
    for e in range(E):
        lo, hi = int(offs[e]), int(offs[e + 1])
        if lo == hi:
            continue
        ae = av[rows[lo:hi].long()] if gather else av[lo:hi]
        we = wv[e].t().contiguous()
        y, mag = ae @ we, ae.abs() @ we.abs()
        d = K * 2.0 ** -23 * mag
        if glu:                                          # (swiglu_limits)
            (gt, u), (dg, du) = y.chunk(2, 1), d.chunk(2, 1)
            y = gt * torch.sigmoid(gt) * u
            rel = 2.0 ** -21 + 1.45 * gt.abs() * 2.0 ** -24
            d = 1.1 * u.abs() * dg + (gt.abs() + 1.1 * dg) * du + rel * y.abs()
        lim = d + 2.0 ** -8 * (y.abs() + d) + 2.0 ** -120
        off = (got[lo:hi].double() - y).abs()
        assert bool((off <= lim).all()), (e, int((off > lim).sum()))
