"""Refusals of the training-step calls, on the CPU: every call below fails its
argument checks before it touches memory or launches anything."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import fp4_quantized_gemm_amd as F

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_UNSUP = 0, 1, 2, 3, 4, 5
A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10002)


def test_checkpoint_refusals():
    L = F.lib()
    ck = L.mxfp8_checkpoint
    assert ck(A, 4, 48, 48, A, A, None, None) == ERR_SHAPE           # K % 32
    assert ck(A, 4, 0, 0, A, A, None, None) == ERR_SHAPE
    assert ck(A, -1, 64, 64, A, A, None, None) == ERR_SHAPE
    assert ck(A, 4, 64, 56, A, A, None, None) == ERR_SHAPE           # ldx < K
    assert ck(A, 4, 64, 68, A, A, None, None) == ERR_SHAPE           # ldx % 8
    assert ck(A, 4, 96, 96, A, A, A, None) == ERR_SHAPE              # h needs K % 64
    assert ck(A, 4, 64, 64, A, None, None, None) == ERR_NULL
    assert ck(A, 4, 64, 64, None, None, None, None) == ERR_NULL
    assert ck(None, 4, 64, 64, A, A, None, None) == ERR_NULL
    assert ck(MIS, 4, 64, 64, A, A, None, None) == ERR_ALIGN
    assert ck(A, 4, 64, 64, MIS, A, None, None) == ERR_ALIGN
    assert ck(None, 0, 64, 64, A, A, None, None) == OK
    rs = L.mxfp8_restore
    assert rs(A, A, 4, 40, A, 40, None) == ERR_SHAPE
    assert rs(A, A, 4, 64, A, 32, None) == ERR_SHAPE
    assert rs(A, None, 4, 64, A, 64, None) == ERR_NULL
    assert rs(A, A, 4, 64, MIS, 64, None) == ERR_ALIGN
    assert rs(None, None, 0, 64, None, 64, None) == OK


def dgrad(dy=A, rows=A, M=64, wc=A, ws=A, g=A, off=A, E=2, P=128, N=64, K=128, dx=A, w=A,
          wb=1 << 30):
    return F.lib().grouped_w4a16_dgrad(dy, rows, M, wc, ws, g, off, E, P, N, K, dx, w, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), ERR_SHAPE), (dict(E=1025), ERR_SHAPE), (dict(N=24), ERR_SHAPE),
    (dict(K=96), ERR_SHAPE), (dict(N=(1 << 20) + 16, M=1, P=1), ERR_SHAPE),
    (dict(K=(1 << 20) + 64), ERR_SHAPE), (dict(P=-1), ERR_SHAPE), (dict(P=1 << 31), ERR_SHAPE),
    (dict(rows=None), ERR_SHAPE),                       # 64 rows for 128
    (dict(M=0), ERR_SHAPE), (dict(M=-3), ERR_SHAPE),
    (dict(M=1 << 26), ERR_UNSUP),                       # dy of 8 GiB
    (dict(dy=None), ERR_NULL), (dict(wc=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(g=None), ERR_NULL), (dict(off=None), ERR_NULL), (dict(dx=None), ERR_NULL),
    (dict(w=None), ERR_NULL), (dict(dy=MIS), ERR_ALIGN), (dict(dx=MIS), ERR_ALIGN),
    (dict(wc=MIS), ERR_ALIGN), (dict(wb=4), ERR_WS), (dict(P=0, M=0), OK),
])
def test_dgrad_refusals(kw, want):
    assert dgrad(**kw) == want
    if want != OK:
        assert b"grouped_w4a16_dgrad" in F.lib().nvfp4_last_error()


def wgrad(dy=A, dyr=None, Md=128, x=A, xs=None, xr=None, Mx=128, off=A, E=2, P=128, N=64, K=64,
          dw=A, bf=0, acc=0, w=A, wb=1 << 30):
    return F.lib().grouped_wgrad(dy, dyr, Md, x, xs, xr, Mx, off, E, P, N, K, dw, bf, acc, w, wb,
                                 None)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), ERR_SHAPE), (dict(E=1025), ERR_SHAPE), (dict(N=12), ERR_SHAPE),
    (dict(K=4), ERR_SHAPE), (dict(K=40, xs=A), ERR_SHAPE), (dict(P=-1), ERR_SHAPE),
    (dict(Md=127), ERR_SHAPE), (dict(Mx=127), ERR_SHAPE),
    (dict(Md=0, dyr=A), ERR_SHAPE), (dict(Mx=0, xr=A), ERR_SHAPE),
    (dict(Md=1 << 25), ERR_UNSUP), (dict(Mx=1 << 25), ERR_UNSUP),
    (dict(Mx=1 << 26, xs=A), ERR_UNSUP), (dict(P=1 << 30, Md=1 << 30, Mx=1 << 30), ERR_SHAPE),
    (dict(N=(1 << 20) + 8), ERR_SHAPE), (dict(N=1 << 16, K=1 << 14), ERR_UNSUP),
    (dict(bf=2), ERR_UNSUP), (dict(bf=1, acc=1), ERR_UNSUP),
    (dict(dy=None), ERR_NULL), (dict(x=None), ERR_NULL), (dict(off=None), ERR_NULL),
    (dict(dw=None), ERR_NULL), (dict(w=None), ERR_NULL),
    (dict(dy=MIS), ERR_ALIGN), (dict(x=MIS), ERR_ALIGN), (dict(dw=MIS), ERR_ALIGN),
    (dict(wb=8), ERR_WS),
])
def test_wgrad_refusals(kw, want):
    assert wgrad(**kw) == want
    assert b"grouped_wgrad" in F.lib().nvfp4_last_error()


def swiglu(y=A, ys=None, dh=A, inv=A, w=A, T=8, tk=2, I=64, dy=A, hw=A, dw=A):
    return F.lib().moe_swiglu_backward(y, ys, dh, inv, w, T, tk, I, dy, hw, dw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ERR_SHAPE), (dict(tk=0), ERR_SHAPE), (dict(tk=33), ERR_SHAPE),
    (dict(I=12), ERR_SHAPE), (dict(I=40, ys=A), ERR_SHAPE), (dict(T=1 << 30), ERR_SHAPE),
    (dict(y=None), ERR_NULL), (dict(dh=None), ERR_NULL), (dict(dy=None), ERR_NULL),
    (dict(w=None), ERR_NULL), (dict(inv=None), ERR_NULL),
    (dict(y=MIS), ERR_ALIGN), (dict(dh=MIS), ERR_ALIGN), (dict(hw=MIS), ERR_ALIGN),
    (dict(T=0), OK),
])
def test_swiglu_backward_refusals(kw, want):
    assert swiglu(**kw) == want


def test_workspace_queries_take_any_sizes():
    L = F.lib()
    for q in (L.grouped_w4a16_dgrad_workspace_size, L.grouped_wgrad_workspace_size):
        assert q(128, 131072, 4096, 1536) > 0
        assert q(0, -1, -1, -1) > 0


def test_binding_refuses_host_tensors():
    b = torch.zeros(4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(F.NvfpError, match="device tensor"):
        F.mxfp8_checkpoint(b)
    with pytest.raises(F.NvfpError, match="device tensor"):
        F.mxfp8_restore(b.view(torch.uint8), b.view(torch.uint8))
    with pytest.raises(F.NvfpError, match="device tensor"):
        F.grouped_wgrad(b, None, b, None, i)
    with pytest.raises(F.NvfpError, match="device tensor"):
        F.moe_swiglu_backward(b, b)
    with pytest.raises(F.NvfpError, match="device tensor"):
        F.grouped_w4a16_dgrad(b, None, b, b, b, i)


SIZES = [-(1 << 63), -1, 0, 1, 8, 16, 32, 63, 64, 65, 96, 1024, 1025, (1 << 20), (1 << 20) + 64, 1 << 22,
         1 << 24, 1 << 30, 1 << 31, 1 << 40, 1 << 62, (1 << 63) - 1]


@pytest.mark.parametrize("query", ["grouped_w4a16_dgrad_workspace_size",
                                   "grouped_wgrad_workspace_size"])
def test_workspace_queries_survive_every_size(query):
    """A caller asks before the call that would refuse its sizes.  (In a process
    of its own: a division by zero there ends it.)"""
    code = ("import itertools, sys, fp4_quantized_gemm_amd as F\n"
            f"q = F.lib().{query}\n"
            "for a in itertools.product(%r, repeat=4):\n"
            "    n = q(*a)\n"
            "    assert 256 <= n < 1 << 62, (a, n)\n" % (SIZES,))
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


@pytest.mark.parametrize("E,M,N,K", [(1, 1, 16, 32), (1, 1, 24, 64), (1, 1, 16, 96), (1025, 8, 16, 64),
                                     (1, 1 << 31, 16, 64), (1, 1, (1 << 20) + 16, 64),
                                     (1, 1, 16, (1 << 20) + 64)])
def test_dgrad_query_of_refused_sizes(E, M, N, K):
    assert F.lib().grouped_w4a16_dgrad_workspace_size(E, M, N, K) == 256
    assert dgrad(E=E, P=M, N=N, K=K) == ERR_SHAPE


@pytest.mark.parametrize("E,M,N,K", [(1, 1, 4, 64), (1, 1, 64, 12), (1025, 8, 16, 64),
                                     (1, 1 << 30, 16, 64), (1, 1, (1 << 20) + 8, 64),
                                     (1, 1, 16, (1 << 20) + 8)])
def test_wgrad_query_of_refused_sizes(E, M, N, K):
    assert F.lib().grouped_wgrad_workspace_size(E, M, N, K) == 256
    assert wgrad(E=E, P=M, N=N, K=K) == ERR_SHAPE


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the device, for what the binding
    checks before it calls the library."""
    is_cuda = True


def there(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    """The library calls the binding makes, recorded instead of made."""
    made = []
    monkeypatch.setattr(F, "_call", lambda name, dev, *a: made.append((name, a)))
    return made


@pytest.mark.parametrize("K", [8, 16, 24, 40])
def test_binding_refuses_8_bit_x_of_part_blocks(calls, K):
    """Under 32 columns the scales have no elements, hence no address: the
    library would take the codes for bf16 values and read past their end."""
    with pytest.raises(F.NvfpError, match="32"):
        F.grouped_wgrad(there(4, 64), None, there(4, K, dtype=torch.uint8), None,
                        there(2, dtype=torch.int32), x_scales=there(4, K // 32, dtype=torch.uint8))
    assert not calls


@pytest.mark.parametrize("I", [8, 24, 40])
def test_binding_refuses_8_bit_y_of_part_blocks(calls, I):
    with pytest.raises(F.NvfpError, match="32"):
        F.moe_swiglu_backward(there(4, 2 * I, dtype=torch.uint8), there(4, I),
                              y_scales=there(4, 2 * I // 32, dtype=torch.uint8))
    assert not calls


def test_binding_passes_8_bit_operands_on(calls):
    u8 = torch.uint8
    F.grouped_wgrad(there(4, 64), None, there(4, 32, dtype=u8), None, there(2, dtype=torch.int32),
                    x_scales=there(4, 1, dtype=u8))
    F.moe_swiglu_backward(there(4, 64, dtype=u8), there(4, 32), y_scales=there(4, 2, dtype=u8))
    assert [c[0] for c in calls] == ["grouped_wgrad", "moe_swiglu_backward"]
    assert calls[0][1][4] and calls[1][1][1]                         # the scales' addresses


@pytest.mark.parametrize("N,last", [(48, 44739242), (80, 26843545), (16, (1 << 27) - 1)])
def test_dgrad_takes_dy_up_to_its_stated_limit(N, last):
    """M_src * N * 2 < 2^32, exactly: a workspace of 4 bytes stops the call
    after the check of sizes."""
    assert last * N * 2 < 1 << 32 <= (last + 1) * N * 2
    assert dgrad(M=last, N=N, wb=4) == ERR_WS
    assert dgrad(M=last + 1, N=N, wb=4) == ERR_UNSUP
    assert dgrad(M=(1 << 63) - 1, N=N, wb=4) == ERR_UNSUP


@pytest.mark.parametrize("C,xs,last", [(24, None, 89478485), (8, None, (1 << 28) - 1), (96, A, 44739242),
                                       (32, A, (1 << 27) - 1)])
def test_wgrad_takes_operands_up_to_their_stated_limit(C, xs, last):
    size = 1 if xs else 2
    assert last * C * size < 1 << 32 <= (last + 1) * C * size
    assert wgrad(xr=A, Mx=last, K=C, xs=xs, wb=4) == ERR_WS
    assert wgrad(xr=A, Mx=last + 1, K=C, xs=xs, wb=4) == ERR_UNSUP
    if not xs:
        assert wgrad(dyr=A, Md=last, N=C, wb=4) == ERR_WS
        assert wgrad(dyr=A, Md=last + 1, N=C, wb=4) == ERR_UNSUP
        assert wgrad(dyr=A, Md=(1 << 63) - 1, N=C, wb=4) == ERR_UNSUP


def test_stated_limits():
    """Sizes refused for a limit that the header and the message name."""
    L = F.lib()

    def said():
        return L.nvfp4_last_error().decode()
    # row tiles of 256 rows times column tiles of 256
    assert dgrad(E=1, P=1 << 30, N=16, K=64) == ERR_UNSUP and "2^22" in said()
    assert dgrad(E=1, P=(1 << 30) - 256 * 15, N=16, K=64) == ERR_UNSUP and "2^22" in said()
    assert dgrad(E=1024, P=1 << 20, N=16, K=1 << 20) == ERR_UNSUP and "2^22" in said()
    assert L.mxfp8_checkpoint(A, 1, 1 << 22, 1 << 22, A, A, None, None) == ERR_SHAPE
    assert "2^22" in said()
    assert L.mxfp8_restore(A, A, 1, 1 << 22, A, 1 << 22, None) == ERR_SHAPE and "2^22" in said()
    assert L.mxfp8_checkpoint(A, 1 << 40, 64, 64, A, A, None, None) == ERR_SHAPE
    assert "2^40" in said()
    assert L.mxfp8_restore(A, A, 1 << 40, 64, A, 64, None) == ERR_SHAPE and "2^40" in said()
    assert swiglu(T=1, tk=1, I=1 << 31) == ERR_SHAPE and "I < 2^31" in said()
