"""The rollout-side MoE expert block as a chain of library calls.

Weights go through the shared QDQ path once (per weight sync); each forward
routes and permutes tokens, quantizes the activation online, selects the
high-residual channels, runs the grouped W4A4 GEMM with the residual added
back, forms and quantizes the SwiGLU activation for the down projection the
same way, and combines the expert outputs (QUADS: arXiv abstract;
gist.science technical summary §2.1-§2.2).  Nothing here computes: every
step is one call into libnvfp4rac.

The trainer's side of the same block (asymmetric W4A16 QAT, summary §2.2 A):
moe_train_forward keeps what the backward pass needs, by default in 8 bits,
and moe_train_backward returns the gradients.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import (NvfpError, _arg, _wshape, grouped_w4a16_dgrad, grouped_w4a16_gemm, grouped_w4a4_gemm_rac,
               grouped_w4a4_gemm_rac_per_expert, grouped_w4a4_gemm_rac_swiglu, grouped_wgrad,
               moe_permute, moe_swiglu_backward, mxfp8_checkpoint, nvfp4_quantize_act_amax,
               moe_unpermute_combine, nvfp4_qdq_residual, nvfp4_qdq_weights, nvfp4_quantize_act,
               select_residual_channels, select_residual_channels_per_expert)


@dataclass
class QuantWeights:
    codes: torch.Tensor      # [E][N][K/2] u8, row-major E2M1 pairs
    scales: torch.Tensor     # [E][N][K/16] u8, row-major E4M3 block scales
    g: torch.Tensor          # [E] f32
    qdq: torch.Tensor        # [E][N][K] bf16 or None
    packed_codes: torch.Tensor    # the grouped GEMMs' packed copy of codes ...
    packed_scales: torch.Tensor   # ... and block scales


def prepare_weights(w, want_qdq=False) -> QuantWeights:
    return QuantWeights(*nvfp4_qdq_weights(w, want_qdq=want_qdq, want_packed=True))


def quantized_linear_rac(x, wq: QuantWeights, k, a_rows=None, offsets=None, M_total=None,
                         glu=False, rac="bf16", select="shared", swiglu_out=False, amax=None):
    """Quantize x (or SwiGLU of x), select k channels, grouped GEMM.
    rac="bf16" adds the bf16 residual of the selected channels back;
    rac="nvfp4" quantizes that residual a second time to NVFP4 first and adds
    its fake-quantized value back.  select="shared" picks one channel set
    for the whole call; select="per_expert" one per expert, from the rows
    routed to it.  swiglu_out=True returns h = SwiGLU of the [gate | up]
    product instead of the product (fused into the GEMM; shared selection
    only).  amax: x's tensor amax as bf16 bits (from the fused SwiGLU), so the
    quantizer reads x once.  Returns (y or h, stage dict)."""
    if rac not in ("bf16", "nvfp4"):
        raise ValueError(f"rac must be 'bf16' or 'nvfp4', not {rac!r}")
    if select not in ("shared", "per_expert"):
        raise ValueError(f"select must be 'shared' or 'per_expert', not {select!r}")
    per_expert = select == "per_expert"
    if amax is not None:
        q = nvfp4_quantize_act_amax(x, amax, want_score=k > 0 and not per_expert)
    else:
        q = nvfp4_quantize_act(x, glu=glu, want_score=k > 0 and not per_expert)
    if offsets is None:
        offsets = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
    S = R = None
    if k > 0:
        if per_expert:
            S, R = select_residual_channels_per_expert(q["x_used"], q["codes"], q["scales"],
                                                       q["g"], None, k, a_rows, offsets,
                                                       M_total=M_total)
        else:
            S, R = select_residual_channels(q["x_used"], q["codes"], q["scales"], q["g"],
                                            q["score"], k)
        if rac == "nvfp4":
            R = nvfp4_qdq_residual(R)[3]
    if swiglu_out and per_expert:
        raise ValueError("the fused SwiGLU output takes the shared channel selection")
    args = (q["codes"], q["scales"], q["g"], a_rows, R, S, wq.packed_codes, wq.packed_scales, wq.g,
            offsets)
    if swiglu_out:
        y, amax = grouped_w4a4_gemm_rac_swiglu(*args, M_total=M_total, with_amax=True)
        return y, dict(q=q, S=S, R=R, h_amax=amax)
    gemm = grouped_w4a4_gemm_rac_per_expert if per_expert else grouped_w4a4_gemm_rac
    y = gemm(*args, M_total=M_total)
    return y, dict(q=q, S=S, R=R)


def moe_forward(x, logits, topk, w_first: QuantWeights, w_down: QuantWeights, k_first, k_down,
                bias=None, keep=False, rac="bf16", select="shared", fuse_swiglu=False):
    """x [T][H] bf16, logits [T][E] f32.  w_first [E][N1][H] (N1 = 2I for
    gate+up, I for an up-only block); w_down [E][H][I] or None.  Returns the
    combined output [T][H] (or the first GEMM's permuted output when there is
    no down projection) and, with keep=True, every intermediate.
    fuse_swiglu=True forms h inside the gate+up GEMM (y1 is then h)."""
    ids, tw, offs, perm, inv = moe_permute(logits, topk, bias)
    rows = perm.numel()
    fuse = fuse_swiglu and w_down is not None
    y1, st1 = quantized_linear_rac(x, w_first, k_first, a_rows=perm, offsets=offs, M_total=rows,
                                   rac=rac, select=select, swiglu_out=fuse)
    out = dict(topk_ids=ids, topk_w=tw, offsets=offs, perm_token=perm, inv_perm=inv, y1=y1,
               st1=st1) if keep else {}
    if w_down is None:
        return y1, out
    y2, st2 = quantized_linear_rac(y1, w_down, k_down, a_rows=None, offsets=offs, M_total=rows,
                                   glu=not fuse, rac=rac, select=select,
                                   amax=st1.get("h_amax") if fuse else None)
    o = moe_unpermute_combine(y2, inv, tw)
    if keep:
        out.update(y2=y2, st2=st2, out=o)
    return o, out


@dataclass
class TrainState:
    """What moe_train_forward keeps for moe_train_backward."""
    x: torch.Tensor          # the block's input: bf16, or its checkpoint's codes
    x_scales: torch.Tensor   # ... and scales (None: bf16)
    y1: torch.Tensor         # [gate | up] products by permuted row, likewise
    y1_scales: torch.Tensor
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    offsets: torch.Tensor
    perm_token: torch.Tensor
    inv_perm: torch.Tensor
    w_first: QuantWeights
    w_down: QuantWeights


def _check_block(x, logits, bias, w_first, w_down):
    """The operands of a block fit together: the products take their sizes
    from one operand and index the others with them on the device."""
    dev = getattr(x, "device", None)
    if not getattr(x, "is_cuda", False) or x.dtype is not torch.bfloat16 or x.dim() != 2:
        _arg(x, torch.bfloat16, "x", dev, (None, None))
    T, H = x.shape
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.shape[0] != T:
        _arg(logits, torch.float32, "logits", dev, (T, None))
    E = logits.shape[1]
    if bias is not None:
        _arg(bias, torch.float32, "bias", dev)
        if bias.numel() != E:
            raise NvfpError(f"bias must have {E} elements, got {bias.numel()}")
    c = w_first.packed_codes
    n = c.shape[2] * 16 if c.dim() == 6 else _wshape(c)[1]
    for name, w, N, K in (("w_first", w_first, n, H), ("w_down", w_down, H, n // 2)):
        c, s, g = w.packed_codes, w.packed_scales, w.g
        tiles = (E, 2, N // 16, K // 64, 16)
        # one comparison for all of it; _arg names what is wrong
        if c.shape != tiles + (32,) or s.shape != tiles + (4,) or g.shape != (E,) or \
                not (c.device == s.device == g.device == dev):
            _arg(c, torch.uint8, name + "'s codes", dev, tiles + (32,))
            _arg(s, torch.uint8, name + "'s scales", dev, tiles + (4,))
            _arg(g, torch.float32, name + "'s tensor scales", dev, (E,))


_HERE = nullcontext()


def _where(x):
    """The calls of a step with x's device as the current one: those of the
    rollout side launch on the current device."""
    dev = x.device
    if dev.type != "cuda" or dev.index == torch._C._cuda_getDevice():
        return _HERE
    return torch.cuda.device(dev)


def moe_train_forward(x, logits, topk, w_first: QuantWeights, w_down: QuantWeights, bias=None,
                      checkpoint="mxfp8"):
    """The block with the trainer's W4A16 products (bf16 activations): x [T][H]
    bf16, logits [T][E] f32, w_first [E][2I][H], w_down [E][H][I] -> (out
    [T][H] bf16, TrainState).  checkpoint="mxfp8" keeps x and the gate and up
    products in 8 bits (1.03 bytes per element instead of 2): out is the same,
    and the backward pass sees values off by up to 2^-4 of themselves (of a
    block of 32, those under 2^-13 of its largest by more), which moves
    gradients of random data by 3 to 4% in norm.  "bf16" keeps them as they
    are, x itself and not a copy: it is not to be overwritten before the
    backward pass."""
    if checkpoint not in ("mxfp8", "bf16"):
        raise ValueError(f"checkpoint must be 'mxfp8' or 'bf16', not {checkpoint!r}")
    _check_block(x, logits, bias, w_first, w_down)
    with _where(x):
        return _train_forward(x, logits, topk, w_first, w_down, bias, checkpoint == "mxfp8")


def _train_forward(x, logits, topk, w_first, w_down, bias, mx):
    ids, tw, offs, perm, inv = moe_permute(logits, topk, bias)
    rows = perm.numel()
    y1 = grouped_w4a16_gemm(x, perm, w_first.packed_codes, w_first.packed_scales, w_first.g, offs,
                            M_total=rows)
    c1 = mxfp8_checkpoint(y1, glu=True, want_codes=mx)
    y2 = grouped_w4a16_gemm(c1["h"], None, w_down.packed_codes, w_down.packed_scales, w_down.g,
                            offs, M_total=rows)
    out = moe_unpermute_combine(y2, inv, tw)
    kept_x, x_scales, kept_y, y_scales = x, None, y1, None
    if mx:
        c0 = mxfp8_checkpoint(x)
        kept_x, x_scales, kept_y, y_scales = c0["codes"], c0["scales"], c1["codes"], c1["scales"]
    return out, TrainState(kept_x, x_scales, kept_y, y_scales, ids, tw, offs, perm, inv, w_first,
                           w_down)


def moe_train_backward(st: TrainState, d_out, dw_dtype=torch.float32, dw_first=None, dw_down=None):
    """Gradients of moe_train_forward for d_out [T][H] bf16 -> dict(dx [T][H]
    bf16, dw_first [E][2I][H], dw_down [E][H][I] (dw_dtype float32 or
    bfloat16), d_topk_w [T][tk] f32).  dw_first, dw_down: float32 tensors that
    the weight gradients are added to (gradient accumulation).  The routing
    weight enters in the SwiGLU's backward pass, so d_out goes into both of the
    down projection's products as it is, gathered by token."""
    # (d_out is gathered by token, a token past its end as its last row)
    T, H = st.topk_w.shape[0], st.w_down.packed_codes.shape[2] * 16
    if getattr(d_out, "shape", None) != (T, H):
        raise NvfpError(f"d_out must be a device tensor of shape {[T, H]}")
    # all that the weight gradients could refuse, before one of them has been
    # added to (their own limits are the stricter for the first product's,
    # which has twice the columns: it comes first)
    for name, out, w in (("dw_first", dw_first, st.w_first), ("dw_down", dw_down, st.w_down)):
        if out is not None:
            E, N = _wshape(w.packed_codes)
            _arg(out, torch.float32, name, d_out.device, (E, N, w.packed_codes.shape[3] * 64))
    if (dw_first is None or dw_down is None) and dw_dtype not in (torch.float32, torch.bfloat16):
        raise NvfpError(f"dw_dtype must be float32 or bfloat16, not {dw_dtype}")
    with _where(d_out):
        return _train_backward(st, d_out, dw_dtype, dw_first, dw_down)


def _train_backward(st, d_out, dw_dtype, dw_first, dw_down):
    acc1, acc2 = dw_first is not None, dw_down is not None
    rows = st.perm_token.numel()
    dh = grouped_w4a16_dgrad(d_out, st.perm_token, st.w_down.packed_codes, st.w_down.packed_scales,
                             st.w_down.g, st.offsets, M_total=rows)
    dy1, hw, d_tw = moe_swiglu_backward(st.y1, dh, st.inv_perm, st.topk_w, y_scales=st.y1_scales)
    g_first = grouped_wgrad(dy1, None, st.x, st.perm_token, st.offsets, x_scales=st.x_scales,
                            M_total=rows, dtype=dw_dtype, out=dw_first, accumulate=acc1)
    g_down = grouped_wgrad(d_out, st.perm_token, hw, None, st.offsets, M_total=rows,
                           dtype=dw_dtype, out=dw_down, accumulate=acc2)
    dxp = grouped_w4a16_dgrad(dy1, None, st.w_first.packed_codes, st.w_first.packed_scales,
                              st.w_first.g, st.offsets, M_total=rows)
    dx = moe_unpermute_combine(dxp, st.inv_perm, torch.ones_like(st.topk_w))
    return dict(dx=dx, dw_first=g_first, dw_down=g_down, d_topk_w=d_tw)
