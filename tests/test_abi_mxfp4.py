"""Refusals of the MXFP4 calls and of the routing's gradients, on the CPU: every
call below fails its argument checks before it touches memory or launches
anything."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import fp4_quantized_gemm_amd as F
from tests.test_abi_train import SIZES, there

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_UNSUP = 0, 1, 2, 3, 4, 5
A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10002)
U8, I32, F32 = torch.uint8, torch.int32, torch.float32


def quant(x=A, M=4, K=64, ld=64, c=A, s=A):
    return F.lib().mxfp4_quantize(x, M, K, ld, c, s, None)


def quant_t(x=A, E=2, M=64, K=24, ld=24, c=A, s=A):
    return F.lib().mxfp4_quantize_transposed(x, E, M, K, ld, c, s, None)


def restore(c=A, s=A, M=4, K=64, x=A, ld=64):
    return F.lib().mxfp4_restore(c, s, M, K, x, ld, None)


@pytest.mark.parametrize("call", [quant, restore])
@pytest.mark.parametrize("kw,want", [
    (dict(K=48), ERR_SHAPE), (dict(K=0, ld=0), ERR_SHAPE), (dict(M=-1), ERR_SHAPE),
    (dict(M=1 << 40), ERR_SHAPE), (dict(ld=56), ERR_SHAPE), (dict(ld=68), ERR_SHAPE),
    (dict(K=1 << 22, ld=1 << 22), ERR_SHAPE), (dict(ld=1 << 22), ERR_SHAPE),
    (dict(x=None), ERR_NULL), (dict(c=None), ERR_NULL), (dict(s=None), ERR_NULL),
    (dict(x=MIS), ERR_ALIGN), (dict(c=MIS), ERR_ALIGN), (dict(M=0, x=None, c=None, s=None), OK),
])
def test_quantize_and_restore_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(E=-1), ERR_SHAPE), (dict(E=65536), ERR_SHAPE), (dict(M=48), ERR_SHAPE), (dict(M=0), ERR_SHAPE),
    (dict(M=1 << 22), ERR_SHAPE), (dict(K=12, ld=16), ERR_SHAPE), (dict(K=0), ERR_SHAPE),
    (dict(ld=16), ERR_SHAPE), (dict(ld=28), ERR_SHAPE), (dict(ld=1 << 22), ERR_SHAPE),
    (dict(x=None), ERR_NULL), (dict(c=None), ERR_NULL), (dict(s=None), ERR_NULL),
    (dict(x=MIS), ERR_ALIGN), (dict(c=MIS), ERR_ALIGN), (dict(E=0, x=None), OK),
])
def test_quantize_transposed_refusals(kw, want):
    assert quant_t(**kw) == want


def gemm(name="grouped_mxfp4_gemm", a=A, sa=A, rows=A, M=64, w=A, sw=A, off=A, E=2, P=128, N=64, K=128, y=A,
         ws=A, wb=1 << 30):
    return getattr(F.lib(), name)(a, sa, rows, M, w, sw, off, E, P, N, K, y, ws, wb, None)


@pytest.mark.parametrize("name", ["grouped_mxfp4_gemm", "grouped_mxfp4_gemm_swiglu"])
@pytest.mark.parametrize("kw,want", [
    (dict(E=0), ERR_SHAPE), (dict(E=1025), ERR_SHAPE), (dict(P=-1), ERR_SHAPE), (dict(P=1 << 31), ERR_SHAPE),
    (dict(N=24), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(N=(1 << 20) + 32), ERR_SHAPE),
    (dict(K=64), ERR_SHAPE), (dict(K=192), ERR_SHAPE), (dict(K=(1 << 20) + 128), ERR_SHAPE),
    (dict(rows=None), ERR_SHAPE), (dict(M=0), ERR_SHAPE), (dict(M=-1), ERR_SHAPE),
    (dict(M=1 << 26), ERR_UNSUP), (dict(M=(1 << 63) - 1), ERR_UNSUP), (dict(N=1 << 17, K=1 << 17), ERR_UNSUP),
    (dict(a=None), ERR_NULL), (dict(sa=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(sw=None), ERR_NULL),
    (dict(off=None), ERR_NULL), (dict(y=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(a=MIS), ERR_ALIGN), (dict(sa=MIS), ERR_ALIGN), (dict(w=MIS), ERR_ALIGN), (dict(sw=MIS), ERR_ALIGN),
    (dict(y=MIS), ERR_ALIGN), (dict(rows=MIS), ERR_ALIGN), (dict(off=MIS), ERR_ALIGN), (dict(ws=MIS), ERR_ALIGN),
    (dict(wb=4), ERR_WS), (dict(P=0, M=0, a=None, sa=None, y=None), OK),
])
def test_gemm_refusals(name, kw, want):
    assert gemm(name, **kw) == want
    if want != OK:
        assert name.encode() + b":" in F.lib().nvfp4_last_error()


def test_gemm_columns():
    assert gemm(N=16, wb=4) == ERR_WS and gemm("grouped_mxfp4_gemm_swiglu", N=16, wb=4) == ERR_SHAPE
    assert gemm("grouped_mxfp4_gemm_swiglu", N=48, wb=4) == ERR_SHAPE
    assert gemm("grouped_mxfp4_gemm_swiglu", N=32, wb=4) == ERR_WS


@pytest.mark.parametrize("K,last", [(128, (1 << 26) - 1), (384, 22369621)])
def test_gemm_takes_operands_up_to_the_stated_limit(K, last):
    """The activation's codes are below 4 GiB, exactly."""
    assert last * K // 2 < 1 << 32 <= (last + 1) * K // 2
    assert gemm(M=last, K=K, wb=4) == ERR_WS
    assert gemm(M=last + 1, K=K, wb=4) == ERR_UNSUP


def combine(d=A, y=A, inv=A, w=A, T=8, tk=2, N=64, dy=A, dw=A):
    return F.lib().moe_unpermute_combine_backward(d, y, inv, w, T, tk, N, dy, dw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ERR_SHAPE), (dict(T=1 << 31), ERR_SHAPE), (dict(T=1 << 30), ERR_SHAPE), (dict(tk=0), ERR_SHAPE),
    (dict(tk=33), ERR_SHAPE), (dict(N=12), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(N=1 << 31), ERR_SHAPE),
    (dict(d=None), ERR_NULL), (dict(y=None), ERR_NULL), (dict(dw=None), ERR_NULL), (dict(inv=None), ERR_NULL),
    (dict(w=None), ERR_NULL), (dict(dy=None), ERR_NULL),
    (dict(d=MIS), ERR_ALIGN), (dict(y=MIS), ERR_ALIGN), (dict(dy=MIS), ERR_ALIGN), (dict(inv=MIS), ERR_ALIGN),
    (dict(w=MIS), ERR_ALIGN), (dict(dw=MIS), ERR_ALIGN), (dict(T=0, d=None), OK),
])
def test_combine_backward_refusals(kw, want):
    assert combine(**kw) == want


def router(ids=A, w=A, dw=A, T=8, E=16, tk=2, dl=A, db=A, ws=A, wb=1 << 30):
    return F.lib().moe_permute_backward(ids, w, dw, T, E, tk, dl, db, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ERR_SHAPE), (dict(T=1 << 31), ERR_SHAPE), (dict(T=1 << 30), ERR_SHAPE), (dict(E=0), ERR_SHAPE),
    (dict(E=1025), ERR_SHAPE), (dict(tk=0), ERR_SHAPE), (dict(tk=17), ERR_SHAPE), (dict(E=64, tk=33), ERR_SHAPE),
    (dict(ids=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(dw=None), ERR_NULL), (dict(dl=None), ERR_NULL),
    (dict(ws=None), ERR_NULL), (dict(ids=MIS), ERR_ALIGN), (dict(w=MIS), ERR_ALIGN), (dict(dw=MIS), ERR_ALIGN),
    (dict(dl=MIS), ERR_ALIGN), (dict(db=MIS), ERR_ALIGN), (dict(ws=MIS), ERR_ALIGN), (dict(wb=4), ERR_WS),
    (dict(T=0, ids=None, w=None, dw=None, dl=None, db=None, ws=None, wb=0), OK),
])
def test_permute_backward_refusals(kw, want):
    assert router(**kw) == want


@pytest.mark.parametrize("query,n", [("grouped_mxfp4_gemm_workspace_size", 4),
                                     ("moe_permute_backward_workspace_size", 2)])
def test_workspace_queries_survive_every_size(query, n):
    """(In a process of its own: a division by zero there ends it.)"""
    code = ("import itertools, sys, fp4_quantized_gemm_amd as F\n"
            f"q = F.lib().{query}\n"
            "for a in itertools.product(%r, repeat=%d):\n"
            "    n = q(*a)\n"
            "    assert 256 <= n < 1 << 62, (a, n)\n" % (SIZES, n))
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


@pytest.fixture
def calls(monkeypatch):
    """The library calls the binding makes, recorded instead of made."""
    made = []
    monkeypatch.setattr(F, "_call", lambda name, dev, *a: made.append((name, a)))
    return made


def good():
    """Operands of a product of 6 rows, 2 experts, N = 32, K = 128."""
    return dict(a_codes=there(6, 64, dtype=U8), a_scales=there(6, 4, dtype=U8), a_rows=None,
                w_codes=there(2, 32, 64, dtype=U8), w_scales=there(2, 32, 4, dtype=U8),
                expert_offsets=there(3, dtype=I32))


@pytest.mark.parametrize("kw", [
    dict(a_codes=torch.zeros(6, 64, dtype=U8)), dict(a_codes=there(6, 64)), dict(a_codes=there(6, 32, dtype=U8)),
    dict(a_codes=there(6, 128, dtype=U8)[:, ::2]), dict(a_scales=there(6, 3, dtype=U8)),
    dict(a_scales=there(5, 4, dtype=U8)), dict(a_rows=there(6, dtype=torch.int64)),
    dict(a_rows=there(2, 3, dtype=I32)), dict(w_codes=there(2, 32, 32, dtype=U8)),
    dict(w_codes=there(32, 64, dtype=U8)), dict(w_scales=there(2, 32, 8, dtype=U8)),
    dict(w_scales=there(2, 4, 32, dtype=U8)), dict(expert_offsets=there(2, dtype=I32)),
    dict(expert_offsets=there(3, dtype=torch.int64)), dict(out=there(6, 33)), dict(out=there(6, 32, dtype=F32)),
    dict(M_total=-1), dict(a_rows=there(6, dtype=I32), M_total=7), dict(a_codes=None), dict(w_codes=None),
])
def test_binding_refuses_what_does_not_fit(calls, kw):
    for f in (F.grouped_mxfp4_gemm, F.grouped_mxfp4_gemm_swiglu):
        with pytest.raises(F.NvfpError):
            f(**{**good(), **kw})
    assert not calls


def test_binding_passes_good_operands_on(calls):
    assert F.grouped_mxfp4_gemm(**good()).shape == (6, 32)
    assert F.grouped_mxfp4_gemm_swiglu(**good()).shape == (6, 16)
    assert F.grouped_mxfp4_gemm(**{**good(), "a_rows": there(9, dtype=I32)}).shape == (9, 32)
    assert [c[0] for c in calls] == ["grouped_mxfp4_gemm", "grouped_mxfp4_gemm_swiglu", "grouped_mxfp4_gemm"]


def test_binding_refuses_other_operands(calls):
    for f in (lambda: F.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16)),
              lambda: F.mxfp4_quantize(there(4, 64, dtype=F32)), lambda: F.mxfp4_quantize(there(64)),
              lambda: F.mxfp4_quantize(there(2, 2, 4, 64)), lambda: F.mxfp4_quantize(there(4, 64).t()),
              lambda: F.mxfp4_quantize(there(2, 8, 64)[:, ::2]), lambda: F.mxfp4_quantize(None),
              lambda: F.mxfp4_restore(there(4, 32, dtype=U8), there(4, 1, dtype=U8)),
              lambda: F.mxfp4_restore(there(4, 32), there(4, 2, dtype=U8)),
              lambda: F.mxfp4_restore(there(4, 32, dtype=U8), there(4, 2, dtype=U8), out=there(4, 32)),
              lambda: F.moe_unpermute_combine_backward(there(4, 64), there(8, 64), there(4, 2, dtype=I32), there(4, 2)),
              lambda: F.moe_unpermute_combine_backward(there(4, 64), there(7, 64), there(4, 2, dtype=I32),
                                                       there(4, 2, dtype=F32)),
              lambda: F.moe_unpermute_combine_backward(there(4, 64), None, there(3, 2, dtype=I32),
                                                       there(3, 2, dtype=F32)),
              lambda: F.moe_permute_backward(there(4, 2, dtype=I32), there(4, 2, dtype=F32),
                                             there(4, 3, dtype=F32), 8),
              lambda: F.moe_permute_backward(there(4, 2, dtype=torch.int64), there(4, 2, dtype=F32),
                                             there(4, 2, dtype=F32), 8),
              lambda: F.moe_permute_backward(there(4, 2, dtype=I32), there(4, 2, dtype=F32),
                                             there(4, 2, dtype=F32), 0),
              lambda: F.moe_permute_backward(there(4, 2, dtype=I32), there(4, 2, dtype=F32),
                                             there(4, 2, dtype=F32), -1)):
        with pytest.raises(F.NvfpError):
            f()
    assert not calls
