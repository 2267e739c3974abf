"""NVFP4 W4A4 MoE expert GEMM with Residual Activation Compensation for
AMD MI355X (gfx950): Python binding of libnvfp4rac.so.

The binding only marshals arguments: it allocates outputs and workspaces as
torch tensors on the current device, passes raw device pointers and the
current HIP stream to the C ABI declared in include/nvfp4rac.h, and raises on
a non-OK status.  Every step of the path runs in the library's HIP kernels;
there is no fallback: importing the library fails loudly if it is missing.

Calls (same names as the C ABI):
    nvfp4_qdq_weights, nvfp4_quantize_act, select_residual_channels,
    moe_permute, grouped_w4a4_gemm_rac, moe_unpermute_combine
the GEMMs' weight pre-pack for row-major codes quantized elsewhere,
    nvfp4_pack_weights
and, for the variants of the correction, the fused SwiGLU and the
trainer-side W4A16 product,
    nvfp4_qdq_residual, select_residual_channels_per_expert,
    grouped_w4a4_gemm_rac_per_expert, grouped_w4a4_gemm_rac_swiglu,
    grouped_w4a16_gemm
and the FP8 (E4M3) W8A8 baseline the method is compared with,
    fp8_quantize, grouped_fp8_gemm
and the training step around the W4A16 product: 8-bit activation checkpoints,
the product's input and weight gradients, the SwiGLU's backward pass,
    mxfp8_checkpoint, mxfp8_restore, grouped_w4a16_dgrad, grouped_wgrad,
    moe_swiglu_backward
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

from .build import LIB as LIB_PATH

__all__ = ["lib", "nvfp4_qdq_weights", "nvfp4_pack_weights", "QdqWeights",
           "nvfp4_e2m1_encode_f32", "nvfp4_quantize_act", "nvfp4_quantize_act_noalloc", "select_residual_channels",
           "moe_permute", "grouped_w4a4_gemm_rac", "moe_unpermute_combine", "nvfp4_qdq_residual",
           "grouped_w4a16_gemm", "select_residual_channels_per_expert",
           "grouped_w4a4_gemm_rac_per_expert", "grouped_w4a4_gemm_rac_swiglu",
           "nvfp4_quantize_act_amax", "fp8_quantize", "grouped_fp8_gemm",
           "mxfp8_checkpoint", "mxfp8_restore", "grouped_w4a16_dgrad", "grouped_wgrad",
           "moe_swiglu_backward", "NvfpError", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = [
    "nvfp4_version", "nvfp4_status_str", "nvfp4_last_error",
    "nvfp4_qdq_weights_workspace_size", "nvfp4_qdq_weights", "nvfp4_pack_weights",
    "nvfp4_e2m1_encode_f32",
    "nvfp4_quantize_act_workspace_size", "nvfp4_quantize_act", "nvfp4_quantize_act_noalloc",
    "select_residual_channels_workspace_size", "select_residual_channels",
    "moe_permute_workspace_size", "moe_permute",
    "grouped_w4a4_gemm_rac_workspace_size", "grouped_w4a4_gemm_rac",
    "moe_unpermute_combine",
    "nvfp4_qdq_residual_workspace_size", "nvfp4_qdq_residual",
    "grouped_w4a16_gemm_workspace_size", "grouped_w4a16_gemm",
    "select_residual_channels_per_expert_workspace_size", "select_residual_channels_per_expert",
    "grouped_w4a4_gemm_rac_per_expert",
    "grouped_w4a4_gemm_rac_swiglu_workspace_size", "grouped_w4a4_gemm_rac_swiglu",
    "nvfp4_quantize_act_amax",
    "fp8_quantize_workspace_size", "fp8_quantize",
    "grouped_fp8_gemm_workspace_size", "grouped_fp8_gemm",
    "mxfp8_checkpoint", "mxfp8_restore",
    "grouped_w4a16_dgrad_workspace_size", "grouped_w4a16_dgrad",
    "grouped_wgrad_workspace_size", "grouped_wgrad",
    "moe_swiglu_backward",
]


# measurement-only exports (include/nvfp4rac_bench.h)
BENCH_SYMBOLS = ["nvfp4_ceiling_mfma_flops", "nvfp4_ceiling_mfma", "nvfp4_ceiling_mfma_operands",
                 "nvfp4_ceiling_read"]


class NvfpError(RuntimeError):
    pass


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise NvfpError(f"{LIB_PATH} is not built; run python -m fp4_quantized_gemm_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    L.nvfp4_version.restype = ctypes.c_int
    L.nvfp4_status_str.restype = ctypes.c_char_p
    L.nvfp4_status_str.argtypes = [ctypes.c_int]
    L.nvfp4_last_error.restype = ctypes.c_char_p
    for name, args in {
        "nvfp4_qdq_weights_workspace_size": [_I64],
        "nvfp4_quantize_act_workspace_size": [_I64, _I64],
        "select_residual_channels_workspace_size": [_I64, _I64, _I64],
        "moe_permute_workspace_size": [_I64, _I64],
        "grouped_w4a4_gemm_rac_workspace_size": [_I64, _I64, _I64, _I64, _I64, _I64],
        "nvfp4_qdq_residual_workspace_size": [_I64, _I64],
        "grouped_w4a16_gemm_workspace_size": [_I64],
        "select_residual_channels_per_expert_workspace_size": [_I64, _I64],
        "grouped_w4a4_gemm_rac_swiglu_workspace_size": [_I64, _I64, _I64, _I64, _I64, _I64],
        "fp8_quantize_workspace_size": [_I64],
        "grouped_fp8_gemm_workspace_size": [_I64],
        "grouped_w4a16_dgrad_workspace_size": [_I64, _I64, _I64, _I64],
        "grouped_wgrad_workspace_size": [_I64, _I64, _I64, _I64],
    }.items():
        f = getattr(L, name)
        f.restype = _SZ
        f.argtypes = args
    sigs = {
        "nvfp4_qdq_weights": [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "nvfp4_pack_weights": [_P, _P, _I64, _I64, _I64, _P, _P, _P],
        "nvfp4_e2m1_encode_f32": [_P, _I64, _P, _P],
        "nvfp4_quantize_act": [_P, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "nvfp4_quantize_act_noalloc": [_P, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P],
        "select_residual_channels": [_P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _SZ, _P],
        "moe_permute": [_P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "grouped_w4a4_gemm_rac": [_P, _P, _P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P, _I64, _I64,
                                  _I64, _I64, _P, _P, _SZ, _P],
        "moe_unpermute_combine": [_P, _P, _P, _I64, _I64, _I64, _P, _P],
        "nvfp4_qdq_residual": [_P, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P],
        "grouped_w4a16_gemm": [_P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _SZ,
                               _P],
        "select_residual_channels_per_expert": [_P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64,
                                                _I64, _I64, _P, _P, _P, _SZ, _P],
        "grouped_w4a4_gemm_rac_per_expert": [_P, _P, _P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P,
                                             _I64, _I64, _I64, _I64, _P, _P, _SZ, _P],
        "grouped_w4a4_gemm_rac_swiglu": [_P, _P, _P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P, _I64,
                                         _I64, _I64, _I64, _P, _P, _P, _SZ, _P],
        "nvfp4_quantize_act_amax": [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "fp8_quantize": [_P, _I64, _I64, _I64, _P, _P, _P, _SZ, _P],
        "grouped_fp8_gemm": [_P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P],
        "mxfp8_checkpoint": [_P, _I64, _I64, _I64, _P, _P, _P, _P],
        "mxfp8_restore": [_P, _P, _I64, _I64, _P, _I64, _P],
        "grouped_w4a16_dgrad": [_P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _SZ,
                                _P],
        "grouped_wgrad": [_P, _P, _I64, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _I64, _P,
                          ctypes.c_int, ctypes.c_int, _P, _SZ, _P],
        "moe_swiglu_backward": [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    L.nvfp4_ceiling_mfma_flops.restype = ctypes.c_double
    L.nvfp4_ceiling_mfma_flops.argtypes = [ctypes.c_int]
    L.nvfp4_ceiling_mfma.restype = ctypes.c_int
    L.nvfp4_ceiling_mfma.argtypes = [ctypes.c_int, _I64, _I64, _P, _P]
    L.nvfp4_ceiling_mfma_operands.restype = ctypes.c_int
    L.nvfp4_ceiling_mfma_operands.argtypes = [ctypes.c_int, _P, _I64, _I64, _P, _P]
    L.nvfp4_ceiling_read.restype = ctypes.c_int
    L.nvfp4_ceiling_read.argtypes = [_P, _I64, _P, _P]
    _lib = L
    return L


def lib():
    return _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev=None):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(status, name):
    if status != 0:
        L = _load()
        raise NvfpError(f"{name}: {L.nvfp4_status_str(status).decode()}: "
                        f"{L.nvfp4_last_error().decode()}")


def _wshape(w_codes):
    """(E, N) of packed weight codes [E][2][N/16][K/64][16][32] (the shape the
    packed outputs of nvfp4_qdq_weights and nvfp4_pack_weights carry: per
    expert the code tiles, then the same bytes' worth of channel-major
    codes)."""
    if w_codes.dim() != 6 or w_codes.shape[1] != 2 or tuple(w_codes.shape[4:]) != (16, 32):
        raise NvfpError("weight codes must be the packed copy [E][2][N/16][K/64][16][32] "
                        "(nvfp4_qdq_weights' packed outputs or nvfp4_pack_weights)")
    return int(w_codes.shape[0]), int(w_codes.shape[2]) * 16


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _need(t, dtype, name):
    if not t.is_cuda:
        raise NvfpError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise NvfpError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise NvfpError(f"{name} must be contiguous")


def _arg(t, dtype, name, dev, shape=None, optional=False, strided=False):
    """Check one tensor argument: on dev, of the dtype, of the shape (None
    entries are free), contiguous (strided: rows may be padded).  Returns its
    address (None for an optional tensor that is not there)."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise NvfpError(f"{name} must be a device tensor")
    if t.device != dev:
        raise NvfpError(f"{name} is on {t.device}, the call is on {dev}")
    if t.dtype is not dtype:
        raise NvfpError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape and \
            (t.dim() != len(shape) or
             any(w is not None and w != n for w, n in zip(shape, t.shape))):
        raise NvfpError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        if not strided:
            raise NvfpError(f"{name} must be contiguous")
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or \
                (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise NvfpError(f"{name} must have contiguous rows")
    return t.data_ptr()


def _ld(t):
    """Row stride of a 2-D tensor with contiguous rows (one row: its width)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _call(name, dev, *args):
    """One library call on dev's current stream, with dev the current device."""
    fn = getattr(_lib or _load(), name)
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        _check(st, name)


class QdqWeights(NamedTuple):
    """Outputs of nvfp4_qdq_weights."""
    codes: torch.Tensor                    # [E][N][K/2] u8, row-major E2M1 pairs
    scales: torch.Tensor                   # [E][N][K/16] u8, row-major E4M3 block scales
    g: torch.Tensor                        # [E] f32 tensor scales
    qdq: Optional[torch.Tensor]            # [E][N][K] bf16 fake-quantized weight, or None
    # the GEMMs' packed copy: per expert [0] the 512-byte code tiles [N/16][K/64]
    # (bytes ordered [2 column halves][16 rows][16]; viewed as [16][32])
    # (codes) and [..][16][4] (scales), [1] the same sizes holding the
    # channel-major codes [K][N/2] and scales [K/16][N]
    packed_codes: Optional[torch.Tensor]   # [E][2][N/16][K/64][16][32]
    packed_scales: Optional[torch.Tensor]  # [E][2][N/16][K/64][16][4]


def _packed_like(E, N, K, dev):
    return (torch.empty((E, 2, N // 16, K // 64, 16, 32), dtype=torch.uint8, device=dev),
            torch.empty((E, 2, N // 16, K // 64, 16, 4), dtype=torch.uint8, device=dev))


def nvfp4_qdq_weights(w, want_qdq=True, want_packed=True) -> QdqWeights:
    """w [E][N][K] bf16 -> QdqWeights: row-major codes [E][N][K/2] and block
    scales [E][N][K/16], g [E], the bf16 fake-quantized weight (want_qdq),
    and the packed copy the grouped GEMMs take (want_packed)."""
    L = _load()
    _need(w, torch.bfloat16, "w")
    E, N, K = w.shape
    dev = w.device
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((E, N, K // 16), dtype=torch.uint8, device=dev)
    g_w = torch.empty(E, dtype=torch.float32, device=dev)
    w_qdq = torch.empty_like(w) if want_qdq else None
    pc, ps = _packed_like(E, N, K, dev) if want_packed else (None, None)
    ws = _ws(L.nvfp4_qdq_weights_workspace_size(E), dev)
    _check(L.nvfp4_qdq_weights(_ptr(w), E, N, K, _ptr(codes), _ptr(scales), _ptr(g_w),
                               _ptr(w_qdq), _ptr(pc), _ptr(ps), _ptr(ws), ws.numel(),
                               _stream(dev)),
           "nvfp4_qdq_weights")
    return QdqWeights(codes, scales, g_w, w_qdq, pc, ps)


def nvfp4_e2m1_encode_f32(v):
    """E2M1 codes (one per byte) of float32 values v with unit scale: the
    element conversion of every quantizer in the library."""
    L = _load()
    _need(v, torch.float32, "v")
    codes = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(L.nvfp4_e2m1_encode_f32(_ptr(v), v.numel(), _ptr(codes), _stream(v.device)),
           "nvfp4_e2m1_encode_f32")
    return codes


def nvfp4_pack_weights(codes, scales):
    """Row-major codes [E][N][K/2] and scales [E][N][K/16] (u8) -> the
    grouped GEMMs' packed copy (packed_codes, packed_scales)."""
    L = _load()
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.uint8, "scales")
    E, N, Kh = codes.shape
    K = 2 * Kh
    if tuple(scales.shape) != (E, N, K // 16):
        raise NvfpError("scales must be [E][N][K/16]")
    pc, ps = _packed_like(E, N, K, codes.device)
    _check(L.nvfp4_pack_weights(_ptr(codes), _ptr(scales), E, N, K, _ptr(pc), _ptr(ps),
                                _stream(codes.device)), "nvfp4_pack_weights")
    return pc, ps


def nvfp4_quantize_act(x, glu=False, want_score=True):
    """x [M][K] bf16 (glu: [M][2K] = [gate | up]) -> dict(codes, scales, g,
    score, x_used).  x_used is x itself for glu=False, else h."""
    L = _load()
    _need(x, torch.bfloat16, "x")
    M, C = x.shape
    K = C // 2 if glu else C
    dev = x.device
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    score = torch.empty(K, dtype=torch.uint64, device=dev) if want_score else None
    h = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if glu else None
    ws = _ws(L.nvfp4_quantize_act_workspace_size(M, K), dev)
    _check(L.nvfp4_quantize_act(_ptr(x), M, K, C, int(bool(glu)), _ptr(codes), _ptr(scales),
                                _ptr(g), _ptr(score), _ptr(h), _ptr(ws), ws.numel(), _stream(dev)),
           "nvfp4_quantize_act")
    return dict(codes=codes, scales=scales, g=g, score=score, x_used=h if glu else x)


def nvfp4_quantize_act_noalloc(x, glu=False, want_score=True, out=None):
    """nvfp4_quantize_act on the library's fixed device scratch (no
    workspace).  out: optional dict of preallocated codes, scales, g, score
    (and h for glu) tensors to write into, so the call allocates nothing."""
    L = _load()
    _need(x, torch.bfloat16, "x")
    M, C = x.shape
    K = C // 2 if glu else C
    dev = x.device
    o = out or {}
    codes = o.get("codes", None)
    codes = codes if codes is not None else torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    scales = o.get("scales", None)
    scales = scales if scales is not None else torch.empty((M, K // 16), dtype=torch.uint8,
                                                           device=dev)
    g = o.get("g", None)
    g = g if g is not None else torch.empty(1, dtype=torch.float32, device=dev)
    score = o.get("score", None)
    if score is None and want_score:
        score = torch.empty(K, dtype=torch.uint64, device=dev)
    h = o.get("x_used", None) if glu else None
    if glu and h is None:
        h = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    _check(L.nvfp4_quantize_act_noalloc(_ptr(x), M, K, C, int(bool(glu)), _ptr(codes),
                                        _ptr(scales), _ptr(g), _ptr(score), _ptr(h),
                                        _stream(dev)),
           "nvfp4_quantize_act_noalloc")
    return dict(codes=codes, scales=scales, g=g, score=score, x_used=h if glu else x)


def select_residual_channels(x_used, codes, scales, g, score, k):
    """-> (S [k] int32 ascending, R_S [M][k] bf16)."""
    L = _load()
    M, K = x_used.shape
    dev = x_used.device
    S = torch.empty(k, dtype=torch.int32, device=dev)
    R = torch.empty((M, k), dtype=torch.bfloat16, device=dev)
    ws = _ws(L.select_residual_channels_workspace_size(M, K, k), dev)
    _check(L.select_residual_channels(_ptr(x_used), x_used.stride(0), _ptr(codes), _ptr(scales),
                                      _ptr(g), _ptr(score), M, K, k, _ptr(S), _ptr(R), _ptr(ws),
                                      ws.numel(), _stream(dev)),
           "select_residual_channels")
    return S, R


def nvfp4_qdq_residual(R_S):
    """Second-pass NVFP4 quantization of the selected residual R_S [M][k]
    bf16 -> (codes [M][k/2] u8, scales [M][k/16] u8, g_r [1] f32, r_qdq
    [M][k] bf16).  Pass r_qdq as R_S to grouped_w4a4_gemm_rac."""
    L = _load()
    _need(R_S, torch.bfloat16, "R_S")
    M, k = R_S.shape
    dev = R_S.device
    codes = torch.empty((M, k // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((M, k // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    r_qdq = torch.empty_like(R_S)
    ws = _ws(L.nvfp4_qdq_residual_workspace_size(M, k), dev)
    _check(L.nvfp4_qdq_residual(_ptr(R_S), M, k, _ptr(codes), _ptr(scales), _ptr(g), _ptr(r_qdq),
                                _ptr(ws), ws.numel(), _stream(dev)),
           "nvfp4_qdq_residual")
    return codes, scales, g, r_qdq


def moe_permute(logits, topk, bias=None):
    """logits [T][E] f32 -> (topk_ids [T][tk] i32, topk_w [T][tk] f32,
    expert_offsets [E+1] i32, perm_token [T*tk] i32, inv_perm [T][tk] i32)."""
    L = _load()
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    w = torch.empty((T, topk), dtype=torch.float32, device=dev)
    offs = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * topk, dtype=torch.int32, device=dev)
    inv = torch.empty((T, topk), dtype=torch.int32, device=dev)
    ws = _ws(L.moe_permute_workspace_size(T, E), dev)
    _check(L.moe_permute(_ptr(logits), _ptr(bias), T, E, topk, _ptr(ids), _ptr(w), _ptr(offs),
                         _ptr(perm), _ptr(inv), _ptr(ws), ws.numel(), _stream(dev)),
           "moe_permute")
    return ids, w, offs, perm, inv


def select_residual_channels_per_expert(x_used, codes, scales, g, score_unused, k, a_rows,
                                        expert_offsets, M_total=None):
    """Per-expert selection -> (S [E][k] int32, R [M_total][k] bf16 by
    permuted row).  score_unused is accepted for symmetry with
    select_residual_channels and ignored (the per-expert scores are formed
    from the activation itself)."""
    L = _load()
    M_src, K = x_used.shape
    E = int(expert_offsets.numel()) - 1
    if M_total is None:
        M_total = int(a_rows.numel()) if a_rows is not None else M_src
    dev = x_used.device
    S = torch.empty((E, k), dtype=torch.int32, device=dev)
    R = torch.empty((M_total, k), dtype=torch.bfloat16, device=dev)
    ws = _ws(L.select_residual_channels_per_expert_workspace_size(E, K), dev)
    _check(L.select_residual_channels_per_expert(
        _ptr(x_used), x_used.stride(0), _ptr(codes), _ptr(scales), _ptr(g), _ptr(a_rows),
        _ptr(expert_offsets), E, M_src, M_total, K, k, _ptr(S), _ptr(R), _ptr(ws), ws.numel(),
        _stream(dev)), "select_residual_channels_per_expert")
    return S, R


def _gemm_rac(fn_name, a_codes, a_scales, g_x, a_rows, R, S, w_codes, w_scales, g_w,
              expert_offsets, M_total, out, glu=False, h_amax=None):
    L = _load()
    M_src, Kh = a_codes.shape
    K = Kh * 2
    E, N = _wshape(w_codes)
    k = 0 if S is None else int(S.shape[-1])
    if M_total is None:
        M_total = int(a_rows.numel()) if a_rows is not None else M_src
    dev = a_codes.device
    cols = N // 2 if glu else N
    y = out if out is not None else torch.empty((M_total, cols), dtype=torch.bfloat16, device=dev)
    wsq = (L.grouped_w4a4_gemm_rac_swiglu_workspace_size if glu
           else L.grouped_w4a4_gemm_rac_workspace_size)
    ws = _ws(wsq(E, M_src, M_total, N, K, k), dev)
    tail = [_ptr(y), _ptr(h_amax)] if glu else [_ptr(y)]
    _check(getattr(L, fn_name)(_ptr(a_codes), _ptr(a_scales), _ptr(g_x), _ptr(a_rows), M_src,
                               _ptr(R) if k else None, _ptr(S) if k else None, k,
                               _ptr(w_codes), _ptr(w_scales), _ptr(g_w), _ptr(expert_offsets),
                               E, M_total, N, K, *tail, _ptr(ws), ws.numel(), _stream(dev)),
           fn_name)
    return y


def grouped_w4a4_gemm_rac_swiglu(a_codes, a_scales, g_x, a_rows, R_S, S, w_codes, w_scales, g_w,
                                 expert_offsets, M_total=None, out=None, with_amax=False):
    """h [M_total][N/2] bf16 = SwiGLU of the grouped W4A4 GEMM plus correction,
    whose weights' N rows are [gate | up].  with_amax=True returns (h, amax)
    with amax [1] int32 holding max |h| as bf16 bits."""
    amax = torch.empty(1, dtype=torch.int32, device=a_codes.device) if with_amax else None
    h = _gemm_rac("grouped_w4a4_gemm_rac_swiglu", a_codes, a_scales, g_x, a_rows, R_S, S,
                  w_codes, w_scales, g_w, expert_offsets, M_total, out, glu=True, h_amax=amax)
    return (h, amax) if with_amax else h


def nvfp4_quantize_act_amax(x, amax, want_score=True):
    """nvfp4_quantize_act (glu=False) with the tensor amax given as bf16 bits
    in a [1] int32 device tensor (from grouped_w4a4_gemm_rac_swiglu)."""
    L = _load()
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    dev = x.device
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    score = torch.empty(K, dtype=torch.uint64, device=dev) if want_score else None
    ws = _ws(L.nvfp4_quantize_act_workspace_size(M, K), dev)
    _check(L.nvfp4_quantize_act_amax(_ptr(x), M, K, x.stride(0), _ptr(amax), _ptr(codes),
                                     _ptr(scales), _ptr(g), _ptr(score), _ptr(ws), ws.numel(),
                                     _stream(dev)),
           "nvfp4_quantize_act_amax")
    return dict(codes=codes, scales=scales, g=g, score=score, x_used=x)


def grouped_w4a4_gemm_rac_per_expert(a_codes, a_scales, g_x, a_rows, R_P, S_E, w_codes,
                                     w_scales, g_w, expert_offsets, M_total=None, out=None):
    """grouped_w4a4_gemm_rac with S_E [E][k] and R_P [M_total][k] by permuted row."""
    return _gemm_rac("grouped_w4a4_gemm_rac_per_expert", a_codes, a_scales, g_x, a_rows, R_P,
                     S_E, w_codes, w_scales, g_w, expert_offsets, M_total, out)


def grouped_w4a4_gemm_rac(a_codes, a_scales, g_x, a_rows, R_S, S, w_codes, w_scales, g_w,
                          expert_offsets, M_total=None, out=None):
    """Y [M_total][N] bf16 for the expert-grouped W4A4 GEMM plus the residual
    correction on the channels S (k = len(S), 0 disables it)."""
    return _gemm_rac("grouped_w4a4_gemm_rac", a_codes, a_scales, g_x, a_rows, R_S, S, w_codes,
                     w_scales, g_w, expert_offsets, M_total, out)


def grouped_w4a16_gemm(x, a_rows, w_codes, w_scales, g_w, expert_offsets, M_total=None,
                       out=None):
    """Y [M_total][N] bf16 = x (bf16, gathered by a_rows) times the
    dequantized NVFP4 weights of each row's expert: the trainer-side W4A16
    product."""
    L = _load()
    _need(x, torch.bfloat16, "x")
    M_src, K = x.shape
    E, N = _wshape(w_codes)
    if M_total is None:
        M_total = int(a_rows.numel()) if a_rows is not None else M_src
    dev = x.device
    y = out if out is not None else torch.empty((M_total, N), dtype=torch.bfloat16, device=dev)
    ws = _ws(L.grouped_w4a16_gemm_workspace_size(E), dev)
    _check(L.grouped_w4a16_gemm(_ptr(x), _ptr(a_rows), M_src, _ptr(w_codes), _ptr(w_scales),
                                _ptr(g_w), _ptr(expert_offsets), E, M_total, N, K, _ptr(y),
                                _ptr(ws), ws.numel(), _stream(dev)),
           "grouped_w4a16_gemm")
    return y


def fp8_quantize(x, stacked=False):
    """FP8 (E4M3) codes of x with one float32 scale per tensor.
    x bf16 [M][K], or with stacked=True [E][N][K] with one scale per x[e]
    (the weights of one expert).  Returns (codes uint8 of x's shape,
    g float32 [1] or [E])."""
    L = _load()
    _need(x, torch.bfloat16, "x")
    if not x.is_contiguous():
        raise NvfpError("x must be contiguous")
    if stacked:
        E, M, K = x.shape
    else:
        (M, K), E = x.shape, 1
    dev = x.device
    codes = torch.empty(x.shape, dtype=torch.uint8, device=dev)
    g = torch.empty(E, dtype=torch.float32, device=dev)
    ws = _ws(L.fp8_quantize_workspace_size(E), dev)
    _check(L.fp8_quantize(_ptr(x), E, M, K, _ptr(codes), _ptr(g), _ptr(ws), ws.numel(),
                          _stream(dev)), "fp8_quantize")
    return codes, g


def grouped_fp8_gemm(a, g_x, a_rows, w, g_w, expert_offsets, M_total=None, out=None):
    """Y [M_total][N] bf16 = g_x g_w[e] (a gathered by a_rows) times the
    E4M3 weights w [E][N][K] of each row's expert: the FP8 W8A8 baseline."""
    L = _load()
    _need(a, torch.uint8, "a")
    _need(w, torch.uint8, "w")
    M_src, K = a.shape
    E, N, _ = w.shape
    if M_total is None:
        M_total = int(a_rows.numel()) if a_rows is not None else M_src
    dev = a.device
    y = out if out is not None else torch.empty((M_total, N), dtype=torch.bfloat16, device=dev)
    ws = _ws(L.grouped_fp8_gemm_workspace_size(E), dev)
    _check(L.grouped_fp8_gemm(_ptr(a), _ptr(g_x), _ptr(a_rows), M_src, _ptr(w), _ptr(g_w),
                              _ptr(expert_offsets), E, M_total, N, K, _ptr(y), _ptr(ws),
                              ws.numel(), _stream(dev)),
           "grouped_fp8_gemm")
    return y


def moe_unpermute_combine(y, inv_perm, topk_w, out=None):
    L = _load()
    T, tk = inv_perm.shape
    N = y.shape[1]
    o = out if out is not None else torch.empty((T, N), dtype=torch.bfloat16, device=y.device)
    _check(L.moe_unpermute_combine(_ptr(y), _ptr(inv_perm), _ptr(topk_w), T, tk, N, _ptr(o),
                                   _stream(y.device)),
           "moe_unpermute_combine")
    return o


def mxfp8_checkpoint(x, glu=False, want_codes=True):
    """8-bit checkpoint of x [M][K] bf16 (rows may be strided) -> dict(codes
    [M][K] u8 E4M3, scales [M][K/32] u8 E8M0, h).  glu=True: x = [gate | up]
    and h [M][K/2] bf16 = silu(gate) * up from the same read; h is None
    otherwise.  want_codes=False (with glu): h alone."""
    dev = getattr(x, "device", None)
    xp = _arg(x, torch.bfloat16, "x", dev, (None, None), strided=True)
    M, K = x.shape
    codes = scales = h = cp = sp = hp = None
    if want_codes:
        codes = torch.empty((M, K), dtype=torch.uint8, device=dev)
        scales = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
        cp, sp = codes.data_ptr(), scales.data_ptr()
    if glu:
        h = torch.empty((M, K // 2), dtype=torch.bfloat16, device=dev)
        hp = h.data_ptr()
    _call("mxfp8_checkpoint", dev, xp, M, K, _ld(x), cp, sp, hp)
    return dict(codes=codes, scales=scales, h=h)


def mxfp8_restore(codes, scales, out=None):
    """The bf16 values [M][K] that a checkpoint's codes and scales stand for
    (exact).  out: a bf16 tensor to write, whose rows may be strided."""
    dev = getattr(codes, "device", None)
    cp = _arg(codes, torch.uint8, "codes", dev, (None, None))
    M, K = codes.shape
    sp = _arg(scales, torch.uint8, "scales", dev, (M, K // 32))
    xp = _arg(out, torch.bfloat16, "out", dev, (M, K), optional=True, strided=True)
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        xp = out.data_ptr()
    _call("mxfp8_restore", dev, cp, sp, M, K, xp, _ld(out))
    return out


def _whole_blocks(scales, cols, name):
    """An 8-bit operand has whole blocks of 32 columns.  (The scales of fewer
    than 32 have no elements and so no address, and without one the library
    reads the operand as bf16.)"""
    if scales is not None and (cols < 32 or cols % 32):
        raise NvfpError(f"8-bit {name} must have a multiple of 32 columns, got {cols}")


def _m_total(M_total, default, *row_lists):
    """Rows of the permuted side: as given, else a row list's length, else
    the default."""
    for rows in row_lists:
        if rows is not None:
            n = rows.shape[0]
            if M_total is None:
                M_total = n
            elif n < M_total:
                raise NvfpError("a row list is shorter than M_total")
    if M_total is not None and M_total < 0:
        raise NvfpError("M_total must not be negative")
    return default if M_total is None else M_total


def grouped_w4a16_dgrad(dy, dy_rows, w_codes, w_scales, g_w, expert_offsets, M_total=None,
                        out=None):
    """dX [M_total][K] bf16 = dy (bf16 [M_src][N], gathered by dy_rows) times
    the dequantized NVFP4 weights of each row's expert, contracted over N: the
    input gradient of grouped_w4a16_gemm.  Rows outside the experts' are left
    as they were (uninitialised without out)."""
    if not isinstance(dy, torch.Tensor) or not dy.is_cuda:
        raise NvfpError("dy must be a device tensor")
    dev = dy.device
    E, N = _wshape(w_codes)
    K = w_codes.shape[3] * 64
    dyp = _arg(dy, torch.bfloat16, "dy", dev, (None, N))
    M_src = dy.shape[0]
    rp = _arg(dy_rows, torch.int32, "dy_rows", dev, (None,), optional=True)
    wp = _arg(w_codes, torch.uint8, "w_codes", dev)
    wsp = _arg(w_scales, torch.uint8, "w_scales", dev, (E, 2, N // 16, K // 64, 16, 4))
    gp = _arg(g_w, torch.float32, "g_w", dev, (E,))
    op = _arg(expert_offsets, torch.int32, "expert_offsets", dev, (E + 1,))
    M_total = _m_total(M_total, M_src, dy_rows)
    xp = _arg(out, torch.bfloat16, "out", dev, (M_total, K), optional=True)
    if out is None:
        out = torch.empty((M_total, K), dtype=torch.bfloat16, device=dev)
        xp = out.data_ptr()
    nb = (_lib or _load()).grouped_w4a16_dgrad_workspace_size(E, M_total, N, K)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _call("grouped_w4a16_dgrad", dev, dyp, rp, M_src, wp, wsp, gp, op, E, M_total, N, K, xp,
          ws.data_ptr(), nb)
    return out


def grouped_wgrad(dy, dy_rows, x, x_rows, expert_offsets, x_scales=None, M_total=None,
                  dtype=torch.float32, out=None, accumulate=False):
    """dW [E][N][K] = for each expert, dy^T x over its rows (dy [M_dy][N] bf16
    gathered by dy_rows; x [M_x][K] bf16, or a checkpoint's codes with
    x_scales, gathered by x_rows).  dtype float32 or bfloat16; out: a tensor
    to write, with accumulate=True (float32) to add to."""
    dev = getattr(dy, "device", None)
    dyp = _arg(dy, torch.bfloat16, "dy", dev, (None, None))
    xp = _arg(x, torch.bfloat16 if x_scales is None else torch.uint8, "x", dev, (None, None))
    (M_dy, N), (M_x, K) = dy.shape, x.shape
    sp = _arg(x_scales, torch.uint8, "x_scales", dev, (M_x, K // 32), optional=True)
    _whole_blocks(x_scales, K, "x")
    drp = _arg(dy_rows, torch.int32, "dy_rows", dev, (None,), optional=True)
    xrp = _arg(x_rows, torch.int32, "x_rows", dev, (None,), optional=True)
    op = _arg(expert_offsets, torch.int32, "expert_offsets", dev, (None,))
    E = expert_offsets.shape[0] - 1
    M_total = _m_total(M_total, min(M_dy, M_x), dy_rows, x_rows)
    if out is not None:
        dtype = out.dtype
    elif accumulate:
        raise NvfpError("accumulate needs out")
    if dtype not in (torch.float32, torch.bfloat16):
        raise NvfpError(f"dw must be float32 or bfloat16, not {dtype}")
    wp = _arg(out, dtype, "out", dev, (E, N, K), optional=True)
    nb = (_lib or _load()).grouped_wgrad_workspace_size(E, M_total, N, K)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((max(E, 0), N, K), dtype=dtype, device=dev)
        wp = out.data_ptr()
    _call("grouped_wgrad", dev, dyp, drp, M_dy, xp, sp, xrp, M_x, op, E, M_total, N, K, wp,
          int(dtype is torch.bfloat16), int(bool(accumulate)), ws.data_ptr(), nb)
    return out


def moe_swiglu_backward(y, dh, inv_perm=None, topk_w=None, y_scales=None, want_h=True):
    """Backward of h = silu(gate) * up with the routing weights -> (dy
    [P][2I] bf16, hw [P][I] bf16 = routing weight times h (None with
    want_h=False), d_topk_w [T][tk] f32 (None without topk_w)).  y [P][2I] =
    [gate | up] bf16, or a checkpoint's codes with y_scales; dh [P][I] bf16 is
    h's gradient without the routing weight; inv_perm [T][tk] i32 and topk_w
    [T][tk] f32 as moe_permute returns them (both None: one slot per row,
    weight 1).  inv_perm is a permutation of the rows: an entry out of range is
    skipped, and what it would have written stays uninitialised."""
    dev = getattr(y, "device", None)
    yp = _arg(y, torch.bfloat16 if y_scales is None else torch.uint8, "y", dev, (None, None))
    P, I2 = y.shape
    I = I2 // 2
    if I2 != 2 * I:
        raise NvfpError("y must be [gate | up]")
    sp = _arg(y_scales, torch.uint8, "y_scales", dev, (P, I2 // 32), optional=True)
    _whole_blocks(y_scales, I, "gate and up")
    dhp = _arg(dh, torch.bfloat16, "dh", dev, (P, I))
    ip = _arg(inv_perm, torch.int32, "inv_perm", dev, (None, None), optional=True)
    T, tk = (P, 1) if inv_perm is None else inv_perm.shape
    if T * tk != P:
        raise NvfpError(f"inv_perm must have one entry for each of the {P} rows")
    wp = _arg(topk_w, torch.float32, "topk_w", dev, (T, tk), optional=True)
    dy = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
    hw = dw = hp = dwp = None
    if want_h:
        hw = torch.empty((P, I), dtype=torch.bfloat16, device=dev)
        hp = hw.data_ptr()
    if topk_w is not None:
        dw = torch.empty((T, tk), dtype=torch.float32, device=dev)
        dwp = dw.data_ptr()
    _call("moe_swiglu_backward", dev, yp, sp, dhp, ip, wp, T, tk, I, dy.data_ptr(), hp, dwp)
    return dy, hw, dw
