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

The block also runs with MXFP4 products: moe_forward_mxfp4 for serving, and the
training pair with prepare_mxfp4_weights' weights instead of the W4A16 ones.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import (NvfpError, _arg, _wshape, grouped_mxfp4_gemm, grouped_mxfp4_gemm_swiglu,
               grouped_w4a16_dgrad, grouped_w4a16_gemm, grouped_w4a4_gemm_rac,
               grouped_w4a4_gemm_rac_per_expert, grouped_w4a4_gemm_rac_swiglu, grouped_wgrad,
               moe_permute, moe_permute_backward, moe_swiglu_backward, moe_unpermute_combine,
               moe_unpermute_combine_backward, mxfp4_quantize, mxfp8_checkpoint,
               nvfp4_qdq_residual, nvfp4_qdq_weights, nvfp4_quantize_act, nvfp4_quantize_act_amax,
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


@dataclass
class MxWeights:
    codes: torch.Tensor      # [E][N][K/2] u8, row-major E2M1 pairs
    scales: torch.Tensor     # [E][N][K/32] u8, row-major E8M0 block scales
    t_codes: torch.Tensor    # [E][K][N/2], of the transposes (input gradients) or None
    t_scales: torch.Tensor   # [E][K][N/32] or None


def prepare_mxfp4_weights(w, want_transposed=False) -> MxWeights:
    """w [E][N][K] bf16.  want_transposed: also what the input gradient takes,
    quantized along the transposes' rows."""
    _arg(w, torch.bfloat16, "w", getattr(w, "device", None), (None, None, None))
    return MxWeights(*mxfp4_quantize(w), *(mxfp4_quantize(w, transpose=True) if want_transposed
                                           else (None, None)))


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


def moe_forward_mxfp4(x, logits, topk, w_first: MxWeights, w_down: MxWeights, bias=None, keep=False):
    """The block with MXFP4 activations and weights and no compensation: x [T][H]
    bf16, logits [T][E] f32, w_first [E][2I][H] (gate rows, then up rows),
    w_down [E][H][I] -> (out [T][H] bf16, dict: with keep=True every
    intermediate).  H and I multiples of 128."""
    for name, w in (("w_first", w_first), ("w_down", w_down)):
        if not isinstance(w, MxWeights):
            raise NvfpError(f"{name} must be MxWeights (prepare_mxfp4_weights)")
    _check_block(x, logits, bias, w_first, w_down)
    with _where(x):
        ids, tw, offs, perm, inv = moe_permute(logits, topk, bias)
        rows = perm.numel()
        h = grouped_mxfp4_gemm_swiglu(*mxfp4_quantize(x), perm, w_first.codes, w_first.scales, offs,
                                      M_total=rows)
        y2 = grouped_mxfp4_gemm(*mxfp4_quantize(h), None, w_down.codes, w_down.scales, offs,
                                M_total=rows)
        out = moe_unpermute_combine(y2, inv, tw)
    return out, dict(topk_ids=ids, topk_w=tw, offsets=offs, perm_token=perm, inv_perm=inv, h=h, y2=y2,
                     out=out) if keep else {}


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
    has_bias: bool = False
    y2: torch.Tensor = None  # the down projection's output by permuted row, if asked for


def _out_features(w):
    """N of prepared weights [E][N][K]."""
    if isinstance(w, MxWeights):
        return w.codes.shape[1]
    c = w.packed_codes
    return c.shape[2] * 16 if c.dim() == 6 else _wshape(c)[1]


def _check_block(x, logits, bias, w_first, w_down, train=False):
    """The operands of a block fit together: the products take their sizes
    from one operand and index the others with them on the device."""
    dev = getattr(x, "device", None)
    if not getattr(x, "is_cuda", False) or x.dtype is not torch.bfloat16 or x.dim() != 2:
        _arg(x, torch.bfloat16, "x", dev, (None, None))
    T, H = x.shape
    if not isinstance(logits, torch.Tensor) or logits.dtype is not torch.float32 or \
            logits.dim() != 2 or logits.shape[0] != T:
        _arg(logits, torch.float32, "logits", dev, (T, None))
    E = logits.shape[1]
    if bias is not None:
        _arg(bias, torch.float32, "bias", dev)
        if bias.numel() != E:
            raise NvfpError(f"bias must have {E} elements, got {bias.numel()}")
    if isinstance(w_first, MxWeights) != isinstance(w_down, MxWeights):
        raise NvfpError("w_first and w_down must be of one format")
    n = _out_features(w_first)
    for name, w, N, K in (("w_first", w_first, n, H), ("w_down", w_down, H, n // 2)):
        if isinstance(w, MxWeights):
            _arg(w.codes, torch.uint8, name + "'s codes", dev, (E, N, K // 2))
            _arg(w.scales, torch.uint8, name + "'s scales", dev, (E, N, K // 32))
            if train:
                # (the products take strided rows, the weight gradients do not)
                _arg(x, torch.bfloat16, "x", dev, (T, H))
                _arg(w.t_codes, torch.uint8, name + "'s transposed codes", dev, (E, K, N // 2))
                _arg(w.t_scales, torch.uint8, name + "'s transposed scales", dev, (E, K, N // 32))
            continue
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


def _product(a, rows, w, offs, M_total):
    """y = a w^T by expert, in the weights' format."""
    if isinstance(w, MxWeights):
        return grouped_mxfp4_gemm(*mxfp4_quantize(a), rows, w.codes, w.scales, offs, M_total=M_total)
    return grouped_w4a16_gemm(a, rows, w.packed_codes, w.packed_scales, w.g, offs, M_total=M_total)


def _dgrad(d, rows, w, offs, M_total):
    """dx = d w by expert, in the weights' format."""
    if isinstance(w, MxWeights):
        return grouped_mxfp4_gemm(*mxfp4_quantize(d), rows, w.t_codes, w.t_scales, offs, M_total=M_total)
    return grouped_w4a16_dgrad(d, rows, w.packed_codes, w.packed_scales, w.g, offs, M_total=M_total)


def moe_train_forward(x, logits, topk, w_first: QuantWeights, w_down: QuantWeights, bias=None,
                      checkpoint="mxfp8", keep_y2=False):
    """The block with the trainer's W4A16 products (bf16 activations): x [T][H]
    bf16, logits [T][E] f32, w_first [E][2I][H], w_down [E][H][I] -> (out
    [T][H] bf16, TrainState).  With MxWeights (both, with their transposes; H
    and I multiples of 128) the products and their input gradients take MXFP4
    operands instead, and gradients pass the rounding as if it were not there.
    checkpoint="mxfp8" keeps x and the gate and up
    products in 8 bits (1.03 bytes per element instead of 2): out is the same,
    and the backward pass sees values off by up to 2^-4 of themselves (of a
    block of 32, those under 2^-13 of its largest by more), which moves
    gradients of random data by 3 to 4% in norm.  "bf16" keeps them as they
    are, x itself and not a copy: it is not to be overwritten before the
    backward pass.  keep_y2=True keeps the down projection's output too, 2
    bytes for each of its T*tk*H elements: d_topk_w is then the gradient of out
    (see moe_train_backward)."""
    if checkpoint not in ("mxfp8", "bf16"):
        raise ValueError(f"checkpoint must be 'mxfp8' or 'bf16', not {checkpoint!r}")
    _check_block(x, logits, bias, w_first, w_down, train=True)
    with _where(x):
        return _train_forward(x, logits, topk, w_first, w_down, bias, checkpoint == "mxfp8", keep_y2)


def _train_forward(x, logits, topk, w_first, w_down, bias, mx, keep_y2):
    ids, tw, offs, perm, inv = moe_permute(logits, topk, bias)
    rows = perm.numel()
    y1 = _product(x, perm, w_first, offs, rows)
    c1 = mxfp8_checkpoint(y1, glu=True, want_codes=mx)
    y2 = _product(c1["h"], None, w_down, offs, rows)
    out = moe_unpermute_combine(y2, inv, tw)
    kept_x, x_scales, kept_y, y_scales = x, None, y1, None
    if mx:
        c0 = mxfp8_checkpoint(x)
        kept_x, x_scales, kept_y, y_scales = c0["codes"], c0["scales"], c1["codes"], c1["scales"]
    return out, TrainState(kept_x, x_scales, kept_y, y_scales, ids, tw, offs, perm, inv, w_first,
                           w_down, bias is not None, y2 if keep_y2 else None)


def moe_train_backward(st: TrainState, d_out, dw_dtype=torch.float32, dw_first=None, dw_down=None,
                       want_d_logits=False):
    """Gradients of moe_train_forward for d_out [T][H] bf16 -> dict(dx [T][H]
    bf16, dw_first [E][2I][H], dw_down [E][H][I] (dw_dtype float32 or
    bfloat16), d_topk_w [T][tk] f32).  dw_first, dw_down: float32 tensors that
    the weight gradients are added to (gradient accumulation).  want_d_logits:
    also d_logits [T][E] f32 and, if the block had a bias, d_bias [E] f32.  The routing
    weight enters in the SwiGLU's backward pass, so d_out goes into both of the
    down projection's products as it is, gathered by token.

    d_topk_w, and with it d_logits and d_bias, is <dh, h> of the backward pass's
    own dh = W_down^T d_out and h.  out's gradient is <d_out, y2>; with W4A16
    products the two differ by the rounding of dh and the checkpoint of h.  With
    MXFP4 they do not take the same operands (d_out and the weights' transposes
    are rounded to 4 bits in the one, h and the weights in the other), and
    <dh, h> is 15 to 19% in norm off <d_out, y2> for random data (of the block
    without any rounding both are about as far, 27 and 29%, like dx, 29%).  The
    state of keep_y2=True has y2, and d_topk_w is <d_out, y2>."""
    # (d_out is gathered by token, a token past its end as its last row)
    T, H = st.topk_w.shape[0], _out_features(st.w_down)
    if getattr(d_out, "shape", None) != (T, H):
        raise NvfpError(f"d_out must be a device tensor of shape {[T, H]}")
    # (MXFP4 products take strided rows, the weight gradients and y2's not)
    if isinstance(st.w_down, MxWeights) or st.y2 is not None:
        _arg(d_out, torch.bfloat16, "d_out", d_out.device, (T, H))
    # all that the weight gradients could refuse, before one of them has been
    # added to (their own limits are the stricter for the first product's,
    # which has twice the columns: it comes first)
    for name, out, w in (("dw_first", dw_first, st.w_first), ("dw_down", dw_down, st.w_down)):
        if out is not None:
            if isinstance(w, MxWeights):
                E, N, half = w.codes.shape
                K = 2 * half
            else:
                (E, N), K = _wshape(w.packed_codes), w.packed_codes.shape[3] * 64
            _arg(out, torch.float32, name, d_out.device, (E, N, K))
    if (dw_first is None or dw_down is None) and dw_dtype not in (torch.float32, torch.bfloat16):
        raise NvfpError(f"dw_dtype must be float32 or bfloat16, not {dw_dtype}")
    with _where(d_out):
        return _train_backward(st, d_out, dw_dtype, dw_first, dw_down, want_d_logits)


def _train_backward(st, d_out, dw_dtype, dw_first, dw_down, want_d_logits):
    acc1, acc2 = dw_first is not None, dw_down is not None
    rows = st.perm_token.numel()
    exact_tw = None
    if st.y2 is not None:
        # (y2's own gradient, w d_out by row, is not used: the products take d_out)
        exact_tw = moe_unpermute_combine_backward(d_out, st.y2, st.inv_perm, st.topk_w)[1]
    dh = _dgrad(d_out, st.perm_token, st.w_down, st.offsets, rows)
    dy1, hw, d_tw = moe_swiglu_backward(st.y1, dh, st.inv_perm, st.topk_w, y_scales=st.y1_scales)
    if exact_tw is not None:
        d_tw = exact_tw
    g_first = grouped_wgrad(dy1, None, st.x, st.perm_token, st.offsets, x_scales=st.x_scales,
                            M_total=rows, dtype=dw_dtype, out=dw_first, accumulate=acc1)
    g_down = grouped_wgrad(d_out, st.perm_token, hw, None, st.offsets, M_total=rows,
                           dtype=dw_dtype, out=dw_down, accumulate=acc2)
    dxp = _dgrad(dy1, None, st.w_first, st.offsets, rows)
    dx = moe_unpermute_combine(dxp, st.inv_perm, torch.ones_like(st.topk_w))
    grads = dict(dx=dx, dw_first=g_first, dw_down=g_down, d_topk_w=d_tw)
    if want_d_logits:
        E = st.offsets.numel() - 1
        grads["d_logits"], d_bias = moe_permute_backward(st.topk_ids, st.topk_w, d_tw, E,
                                                         want_bias=st.has_bias)
        if st.has_bias:
            grads["d_bias"] = d_bias
    return grads
