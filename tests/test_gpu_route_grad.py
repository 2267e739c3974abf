"""GPU parity of the routing's gradients (moe_unpermute_combine_backward,
moe_permute_backward) against the float64 oracle.

Tolerances, from the arithmetic.  dy is one float32 product (2^-24) rounded to
bf16 (2^-8).  d_topk_w is a float32 sum of N exact products: N * 2^-24 of the
sum of magnitudes.  A logit's gradient w (dw - sum w dw) has tk + 1 terms, each
a product: (tk + 3) * 2^-24 of w (|dw| + sum |w dw|).  d_bias adds
ceil(T / 2048) of them in float32 and rounds the float64 sums of those three
times (a wave's, a workgroup's, the whole): 4 ceil(T / 4096) roundings or fewer."""
import sys

import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from oracle import formats as OF
from oracle import moe as OM
from oracle import mxfp4 as OX
from tests.gpu_util import heavy_bf16, host_vals, to_dev_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_vals(v):
    return to_dev_bf16(OF.f64_to_bf16_bits(v))


def close(got, ref, lim):
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], ref[bad][:3], lim[bad][:3])


@pytest.mark.parametrize("T,E,tk,N", [(1, 1, 1, 8), (1, 8, 8, 512), (3, 4, 2, 72), (65, 16, 5, 520),
                                      (300, 60, 8, 1000), (17, 64, 32, 264), (33, 8, 2, 8192)])
def test_combine_backward(dev, T, E, tk, N):
    say(f"combine backward T={T} tk={tk} N={N}")
    rng = np.random.default_rng(T + N)
    P = T * tk
    d, y = OF.round_to_bf16(rng.standard_normal((T, N)) * 1e-3), heavy_bf16(rng, (P, N))
    inv = rng.permutation(P).reshape(T, tk).astype(np.int32)
    w = rng.random((T, tk)).astype(np.float32)
    w[0, 0] = 0.0
    dy, dw = F.moe_unpermute_combine_backward(dev_vals(d), dev_vals(y), cu(inv), cu(w))
    dy2, none = F.moe_unpermute_combine_backward(dev_vals(d), None, cu(inv), cu(w))
    torch.cuda.synchronize()
    rdy, rdw = OX.combine_backward(d, y, inv, w)
    mag = OX.combine_backward(np.abs(d), np.abs(y), inv, w)[1]
    close(host_vals(dy), rdy, np.abs(rdy) * (2.0 ** -8 + 2 * U) + 2.0 ** -133)
    close(dw.cpu().numpy().astype(np.float64), rdw, N * U * mag + 2.0 ** -149)
    assert none is None and torch.equal(dy, dy2)


def test_combine_backward_skips_entries_out_of_range(dev):
    say("combine backward out of range")
    T, tk, N = 6, 2, 64
    rng = np.random.default_rng(0)
    inv = rng.permutation(T * tk).reshape(T, tk).astype(np.int32)
    inv[1, 0], inv[4, 1] = -1, T * tk
    d, y, w = (dev_vals(rng.standard_normal(s)) for s in ((T, N), (T * tk, N), (T, tk)))
    w = w.float()
    dy = torch.full((T * tk, N), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, tk), 5.0, device="cuda")
    F._call("moe_unpermute_combine_backward", d.device, d.data_ptr(), y.data_ptr(), cu(inv).data_ptr(),
            w.data_ptr(), T, tk, N, dy.data_ptr(), dw.data_ptr())
    torch.cuda.synchronize()
    assert dw[1, 0] == 5 and dw[4, 1] == 5
    unnamed = sorted(set(range(T * tk)) - set(inv.ravel().tolist()))
    assert len(unnamed) == 2 and bool((dy[unnamed] == 5).all())
    assert int((dw == 5).sum()) == 2


@pytest.mark.parametrize("T,E,tk", [(0, 4, 2), (1, 1, 1), (1, 2, 1), (3, 128, 8), (257, 60, 4), (64, 65, 32),
                                    (40, 1024, 32), (4097, 64, 6), (9000, 128, 8), (5000, 300, 2)])
def test_permute_backward(dev, T, E, tk):
    say(f"permute backward T={T} E={E} tk={tk}")
    rng = np.random.default_rng(T + E)
    ids, w = OM.route(rng.standard_normal((T, E)).astype(np.float32), tk)
    dw = (rng.standard_normal((T, tk)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32)
    dl, db = F.moe_permute_backward(cu(ids), cu(w), cu(dw), E, want_bias=True)
    dl2, none = F.moe_permute_backward(cu(ids), cu(w), cu(dw), E)
    torch.cuda.synchronize()
    rl, rb = OX.permute_backward(ids, w, dw, E)
    w64, d64 = w.astype(np.float64), dw.astype(np.float64)
    one = (tk + 3) * U * w64 * (np.abs(d64) + np.abs(w64 * d64).sum(axis=1, keepdims=True))
    lim = np.zeros((T, E))
    np.put_along_axis(lim, ids.astype(np.int64), one, axis=1)
    close(dl.cpu().numpy().astype(np.float64), rl, lim)
    per = 4 * max(1, -(-T // 4096))
    mag = np.abs(rl) + lim
    close(db.cpu().numpy().astype(np.float64), rb, lim.sum(0) + per * U * mag.sum(0) + U * np.abs(rb) + 1e-300)
    assert none is None and torch.equal(dl, dl2)
    if E > tk and T:
        assert int((dl != 0).sum()) <= T * tk


def test_permute_backward_same_expert_twice_and_none(dev):
    say("permute backward twice")
    ids = np.array([[2, 2], [-1, 1], [3, 4]], dtype=np.int32)    # 4 = E: nowhere
    w = np.array([[0.25, 0.75], [0.5, 0.5], [0.5, 0.5]], dtype=np.float32)
    dw = np.array([[1, 2], [1, 3], [2, 0]], dtype=np.float32)
    dl, db = F.moe_permute_backward(cu(ids), cu(w), cu(dw), 4, want_bias=True)
    g = w * (dw - (w * dw).sum(1, keepdims=True))
    want = np.zeros((3, 4), np.float32)
    want[0, 2], want[1, 1], want[2, 3] = g[0].sum(), g[1, 1], g[2, 0]
    assert np.array_equal(dl.cpu().numpy(), want) and np.array_equal(db.cpu().numpy(), want.sum(0))


def test_permute_backward_nan_stays_in_its_token(dev):
    rng = np.random.default_rng(1)
    ids, w = OM.route(rng.standard_normal((70, 16)).astype(np.float32), 4)
    dw = rng.standard_normal((70, 4)).astype(np.float32)
    dw[13, 2] = np.nan
    dl, _ = F.moe_permute_backward(cu(ids), cu(w), cu(dw), 16)
    nan = np.isnan(dl.cpu().numpy())
    assert nan[13, ids[13]].all() and nan.sum() == 4
