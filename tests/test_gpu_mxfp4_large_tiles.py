"""The edges of grouped_mxfp4_gemm's large tiles: NaN scales, rows out of range,
memory that is aligned to 4 bytes only, column tiles that end early, counters
in replayed graphs and on two streams.  Every case asserts that the call's rule
sends it to that kernel, and where counters matter, that they are used.

Tolerances as in test_gpu_mxfp4.py: a sum of K exact products is off by at most
K 2^-23 of the sum of magnitudes, the output's rounding by 2^-8 of its value."""
import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from tests.test_gpu_mxfp4 import cu, offsets_of, operands, say
from tests.test_gpu_mxfp4_block import same

pytestmark = pytest.mark.gpu

CALLS = {False: F.grouped_mxfp4_gemm, True: F.grouped_mxfp4_gemm_swiglu}


def up(a, b):
    return -(-a // b)


def is_large(P, E, N, glu):
    """More than 512 tiles of 16 rows x 64 columns, by the call's estimate."""
    active = min(P, E)
    return up(N // 2 if glu else N, 64) * max(up(P, 16) + active // 2, active) > 512


def is_counted(P, E, N, K):
    """More than 72 steps of K for a workgroup: tiles taken as they get free."""
    tiles = (up(P, 128) + E) * up(N, 256)
    groups = min(up(tiles, 8) * 8, up(2 * torch.cuda.get_device_properties(0).multi_processor_count, 8) * 8)
    return tiles * up(K, 256) > 72 * groups


# K / 128 modulo 4 from 0 to 3, rows of scales shorter than 16 bytes among them
KS = [128, 256, 384, 512, 640, 768, 896]


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("glu", [False, True])
def test_nan_stays_in_its_row_and_column(dev, K, glu):
    """Of two experts with 1300 and 20 rows (tiles of 128 and of 64 rows): a NaN
    scale, first or last of its row, whatever the codes are, makes its row or
    its column NaN, and every other element keeps its bits."""
    N, counts = (2080, [1300, 20]) if glu else (1040, [1300, 20])
    P, E, NO = sum(counts), 2, N // 2 if glu else N
    assert is_large(P, E, N, glu)
    say(f"large tiles nan K={K} glu={glu}")
    rng = np.random.default_rng(K)
    ac, asc, wc, wsc = operands(rng, P, E, N, K)
    od = cu(offsets_of(counts))
    clean = CALLS[glu](cu(ac), cu(asc), None, cu(wc), cu(wsc), od)
    rows, last = [2, 127, 128, 1299, 1303], NO - 1
    for i, r in enumerate(rows):
        asc[r, -1 if i % 2 else 0] = 255
    ac[2], ac[1303] = 0x77, 0                            # (0 times NaN is NaN)
    cols = {0: [7, 255, 256, last], 1: [0, last]}        # by expert, of the output
    for e, cs in cols.items():
        for i, c in enumerate(cs):
            wsc[e, c + (NO if glu and i % 2 else 0), -1 if i % 2 else 0] = 255
    got = CALLS[glu](cu(ac), cu(asc), None, cu(wc), cu(wsc), od)
    torch.cuda.synchronize()
    want = torch.zeros((P, NO), dtype=torch.bool)
    want[rows] = True
    for e, cs in cols.items():
        want[sum(counts[:e]):sum(counts[:e + 1]), cs] = True
    nan = torch.isnan(got).cpu()
    assert torch.equal(nan, want)
    keep = ~want.cuda()
    assert bool((got.view(torch.int16) == clean.view(torch.int16))[keep].all())


@pytest.mark.parametrize("K", [384, 512, 640, 768])
@pytest.mark.parametrize("glu", [False, True])
def test_rows_and_offsets_out_of_range(dev, K, glu):
    """Rows beyond the source read its first or last, offsets beyond the output
    count as its ends: the bits of the call with those."""
    N, M = 2080 if glu else 1040, 2000
    assert is_large(M, 3, N, glu)
    say(f"large tiles out of range K={K} glu={glu}")
    rng = np.random.default_rng(K + 1)
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, M // 2, 3, N, K))
    rows = rng.integers(0, M // 2, M).astype(np.int32)
    at = np.concatenate([[0, 7, 127, 128, M - 1], rng.integers(0, M, 200)])
    far = rows.copy()
    far[at] = rng.choice(np.array([-1, -5, -2 ** 31, M // 2, M, 2 ** 31 - 1, 1 << 24], np.int64), at.size)
    near = np.clip(far.astype(np.int64), 0, M // 2 - 1).astype(np.int32)
    a = CALLS[glu](ac, asc, cu(far), wc, wsc, cu(np.array([-9, 1400, 1450, 1 << 30], np.int32)))
    b = CALLS[glu](ac, asc, cu(near), wc, wsc, cu(np.array([0, 1400, 1450, M], np.int32)))
    torch.cuda.synchronize()
    assert same(a, b)


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("glu", [False, True])
def test_unaligned_scales_rows_and_views(dev, K, glu):
    """Scales, row list and offsets that begin 4 bytes into their memory, codes 16
    bytes, an output that is a view: the bits of the aligned call, and nothing
    beside it."""
    N, counts = 2080 if glu else 1040, [200, 300, 0, 1500]
    P, E, NO = sum(counts), 4, N // 2 if glu else N
    assert is_large(P, E, N, glu)
    say(f"large tiles views K={K} glu={glu}")
    rng = np.random.default_rng(K + 2)
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, P, E, N, K))
    rows, od = cu(rng.integers(0, P, P).astype(np.int32)), cu(offsets_of(counts))

    def at(t, skip):
        m = torch.empty(t.numel() + skip, dtype=t.dtype, device="cuda")
        v = m[skip:].view(t.shape)
        v.copy_(t)
        return v

    want = CALLS[glu](ac, asc, rows, wc, wsc, od)
    out = torch.full((P + 2, NO), 9.0, dtype=torch.bfloat16, device="cuda")
    CALLS[glu](at(ac, 16), at(asc, 4), at(rows, 1), at(wc, 16), at(wsc, 4), at(od, 1), out=out[1:-1])
    torch.cuda.synchronize()
    assert same(out[1:-1], want) and bool((out[0] == 9).all()) and bool((out[-1] == 9).all())


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("N", [2064, 2080, 2112, 2144, 2272])
@pytest.mark.parametrize("glu", [False, True])
def test_column_tiles_that_end_early(dev, N, K, glu):
    """Widths that leave 16, 32, .. columns of a tile, a wave or half a wave's,
    with tiles of 128 and of 64 rows, gathered, and rows behind the last expert."""
    if glu and N % 32:
        N += 16
    counts = [700, 0, 31, 129, 64, 1100]
    P, E, NO = sum(counts), len(counts), N // 2 if glu else N
    assert is_large(P + 3, E, N, glu)
    say(f"large tiles columns N={N} K={K} glu={glu}")
    g = torch.Generator("cuda").manual_seed(N + K)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    M_src = 900
    a, w = F.mxfp4_quantize(rand(M_src, K)), F.mxfp4_quantize(rand(E, N, K))
    rows = torch.randint(0, M_src, (P + 3,), generator=g, device="cuda", dtype=torch.int32)
    offs = offsets_of(counts)
    got = torch.full((P + 3, NO), 3.0, dtype=torch.bfloat16, device="cuda")
    CALLS[glu](*a, rows, *w, cu(offs), out=got)
    assert bool((got[P:] == 3).all())
    av, wv = F.mxfp4_restore(*a).double(), F.mxfp4_restore(*w).double()
    for e in range(E):
        lo, hi = int(offs[e]), int(offs[e + 1])
        if lo == hi:
            continue
        ae, we = av[rows[lo:hi].long()], wv[e].t().contiguous()
        y, d = ae @ we, K * 2.0 ** -23 * (ae.abs() @ we.abs())
        if glu:                                          # (test_gpu_mxfp4.swiglu_limits)
            (gt, u), (dg, du) = y.chunk(2, 1), d.chunk(2, 1)
            y = gt * torch.sigmoid(gt) * u
            rel = 2.0 ** -21 + 1.45 * gt.abs() * 2.0 ** -24
            d = 1.1 * u.abs() * dg + (gt.abs() + 1.1 * dg) * du + rel * y.abs()
        lim = d + 2.0 ** -8 * (y.abs() + d) + 2.0 ** -120
        off = (got[lo:hi].double() - y).abs()
        assert bool((off <= lim).all()), (e, int((off > lim).sum()))


# ---------------------------------------------------------------- counters
COUNTED = dict(counts=[3000, 1, 70, 2500, 0, 130], N=12288, K=4096)


def counted_set(seed, gather):
    counts, N, K = COUNTED["counts"], COUNTED["N"], COUNTED["K"]
    P, E = sum(counts), len(counts)
    assert is_large(P, E, N, True) and is_counted(P, E, N, K)
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    M_src = 4000 if gather else P
    rows = torch.randint(0, M_src, (P,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    return [*F.mxfp4_quantize(rand(M_src, K)), rows, *F.mxfp4_quantize(rand(E, N, K)), cu(offsets_of(counts))]


@pytest.mark.parametrize("glu", [False, True])
def test_counters_in_replayed_graphs(dev, glu):
    """Two graphs of the same call, replayed several times with eager calls
    between, also for other rows and offsets in place: every replay has to find
    its counters at nought."""
    say(f"large tiles graphs glu={glu}")
    s = counted_set(5, True)
    CALLS[glu](*s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = CALLS[glu](*s)
        graphs.append((g, got))
    for i in range(5):
        if i == 3:
            s[2].copy_(s[2].flip(0))
            s[5].copy_(cu(offsets_of([100, 2900, 1, 70, 2600, 30])))
        want = CALLS[glu](*s).clone()
        for _, got in graphs:
            got.zero_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(same(got, want) for _, got in graphs), f"replay {i}"


def test_counters_on_two_streams(dev):
    """Calls on two streams at once, each with its own counters."""
    say("large tiles streams")
    sets = [counted_set(7, True), counted_set(8, False)]
    want = [CALLS[glu](*s) for s in sets for glu in (False, True)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        got = []
        for s, q in zip(sets, streams):
            with torch.cuda.stream(q):
                got += [CALLS[glu](*s) for glu in (False, True)]
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want)), i
