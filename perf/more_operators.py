"""Operators around an expert block with microscaled 4-bit (MXFP4) products, as
cases that can be timed: the quantisation, along the rows or of the transpose;
the expert-grouped product, plain and with the SwiGLU in its epilogue; and the
gradients of the routing, of the weighted combine and of the softmax over the
chosen experts.

`run` computes an operator in its plain form (elementary torch operations in
float32, rounded once at the end), or, with `own` set, through this package.
"""
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a dense layer's input: latency
        dict(name="quantize_dense", op="quantize", E=0, M=64, K=512, transpose=False),
        # the input of a large prefill-sized block, once per layer and forward
        dict(name="quantize_block_input", op="quantize", E=0, M=16384, K=4096, transpose=False),
        # down projection's weights for the product of its input gradient, once per optimizer step
        dict(name="quantize_transposed_weights", op="quantize", E=128, M=2048, K=768, transpose=True),
        # a dense layer at its smallest: latency
        dict(name="gemm_dense", op="gemm", T=64, topk=1, E=1, N=512, K=512, gather=False, skew=0.0, swiglu=False),
        # one token of a serving step: its experts' weights and nothing else
        dict(name="gemm_one_token", op="gemm", T=1, topk=8, E=128, N=4096, K=1536, gather=True, skew=0.0, swiglu=False),
        # a serving step of many sequences, few rows per expert: the weights' bytes count
        dict(name="gemm_few_rows", op="gemm", T=256, topk=8, E=128, N=4096, K=1536, gather=False, skew=0.0,
             swiglu=False),
        # gate and up projection, SwiGLU in the epilogue, a router that prefers some experts
        dict(name="gemm_gate_up", op="gemm", T=4096, topk=8, E=128, N=1536, K=2048, gather=True, skew=0.5, swiglu=True),
        # down projection of a large prefill
        dict(name="gemm_down", op="gemm", T=16384, topk=8, E=128, N=4096, K=1536, gather=False, skew=0.0, swiglu=False),
        # a small step through the combine
        dict(name="combine_few_tokens", op="combine", T=256, topk=8, E=128, N=4096),
        # a large block's combine
        dict(name="combine_block", op="combine", T=16384, topk=8, E=128, N=4096),
        # the router of a small step: latency
        dict(name="router_few_tokens", op="router", T=256, topk=8, E=128, bias=False),
        # the router of a large block, with the gradient of its bias
        dict(name="router_block", op="router", T=16384, topk=8, E=128, bias=True),
    ]


def draw(rng):
    def logu(lo, hi, step=1):
        v = lo * (hi / lo) ** rng.random()
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["quantize", "quantize", "gemm", "gemm", "gemm", "combine", "router"])
    if op == "quantize":
        if rng.random() < 0.5:
            return dict(op=op, E=0, M=logu(1, 32768), K=logu(32, 4096, 32), transpose=False)
        E = rng.choice([0, 1, 8, 60, 128])
        return dict(op=op, E=E, M=logu(32, 2048, 32), K=logu(32, 768, 8), transpose=True)
    E = rng.choice([1, 2, 8, 16, 60, 64, 128])
    topk = 1 if E == 1 else rng.choice([1, 2, 4, 8] if E >= 8 else [1, 2])
    T = logu(1, 65536 // topk)
    if op == "combine":
        return dict(op=op, T=T, topk=topk, E=E, N=logu(8, 4096, 8))
    if op == "router":
        return dict(op=op, T=T, topk=topk, E=E, bias=rng.random() < 0.5)
    return dict(op=op, T=T, topk=topk, E=E, N=logu(32, 4096, 32), K=logu(128, 1536, 128), gather=rng.random() < 0.5,
                skew=rng.choice([0.0, 0.5, 1.0]), swiglu=rng.random() < 0.4)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=F32)


def _activation(gen, M, K):
    # channels of different size, as activations have them
    return (_randn(gen, M, K) * torch.exp(0.5 * _randn(gen, K))).to(BF16)


def _gradient(gen, M, N):
    # small, tokens of different size
    return (_randn(gen, M, N) * (1e-3 * torch.exp(0.5 * _randn(gen, M, 1)))).to(BF16)


def _routing(gen, T, topk, E, skew):
    """Expert-major rows of a top-k routing: offsets [E+1], the token of each
    row, the row of each (token, slot), the experts and their weights."""
    logits = _randn(gen, T, E) + skew * _randn(gen, E)
    top, ids = logits.topk(topk, dim=1)
    flat = ids.reshape(-1)
    order = torch.sort(flat * (T * topk) + torch.arange(T * topk, device="cuda")).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * topk, device="cuda")
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return dict(offsets=offsets, longest=int(counts.max()), rows=(order // topk).to(torch.int32),
                inv=inv.view(T, topk).to(torch.int32), w=torch.softmax(top, 1), ids=ids.to(torch.int32))


def _kept(x):
    """MXFP4 codes [..., K/2] and scale bytes [..., K/32] of x [..., K]: per 32
    elements the smallest power of two 2^E with max |x| <= 7 * 2^E (E from -125
    to 125), and x * 2^-E rounded to E2M1, ties to the even code."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m == 0, torch.full_like(e, -125), torch.clamp(e - 3 + (m > 0.875), -125, 125))
    v = torch.ldexp(b, -e)
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (c | (torch.signbit(v).to(torch.uint8) << 3)).view(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), (e[..., 0] + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "quantize":
        M, K, E = case["M"], case["K"], case["E"]
        s["x"] = (0.02 * _randn(gen, E, M, K)).to(BF16) if E else _activation(gen, M, K)
        return s
    T, topk, E = case["T"], case["topk"], case["E"]
    P = T * topk
    s.update(_routing(gen, T, topk, E, case.get("skew", 0.0)))
    if op == "gemm":
        N, K = case["N"], case["K"]
        s["a_rows"] = s["rows"] if case["gather"] else None
        s["a_codes"], s["a_scales"] = _kept(_activation(gen, T if case["gather"] else P, K))
        s["w_codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        s["w_scales"] = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
        for e in range(E):
            s["w_codes"][e], s["w_scales"][e] = _kept((0.02 * _randn(gen, N, K)).to(BF16))
    elif op == "combine":
        s["d_out"] = _gradient(gen, T, case["N"])
        s["y"] = _activation(gen, P, case["N"])
    else:
        s["dw"] = 1e-2 * _randn(gen, T, topk)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _value(codes, scales):
    """What MXFP4 codes and scales stand for, in float32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()]
    v = v.view(*codes.shape[:-1], scales.shape[-1], 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).flatten(-2)


def _plain_quantize(s):
    x = s["x"].transpose(-1, -2) if s["case"]["transpose"] else s["x"]
    return _value(*_kept(x)).to(BF16)


def _plain_gemm(s):
    first, count = s["offsets"][:-1].long(), s["offsets"].diff().long()
    at = torch.arange(s["longest"], device="cuda")
    there = at < count[:, None]
    row = torch.where(there, first[:, None] + at, 0)
    row = row if s["a_rows"] is None else s["a_rows"].long()[row]
    a = torch.where(there[..., None], _value(s["a_codes"], s["a_scales"])[row], 0)
    y = torch.bmm(a, _value(s["w_codes"], s["w_scales"]).transpose(1, 2))[there]
    if s["case"]["swiglu"]:
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(BF16)


def _plain_combine(s):
    T, topk = s["w"].shape
    inv = s["inv"].long().view(-1)
    d = s["d_out"].float().repeat_interleave(topk, 0)
    dy = torch.empty_like(s["y"])
    dy[inv] = (s["w"].view(-1, 1) * d).to(BF16)
    return dy, (d * s["y"].float()[inv]).sum(1).view(T, topk)


def _plain_router(s):
    w, dw = s["w"], s["dw"]
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    out = torch.zeros(w.shape[0], s["case"]["E"], device="cuda").scatter_(1, s["ids"].long(), dl)
    return (out, out.double().sum(0).float()) if s["case"]["bias"] else out


_PLAIN = dict(quantize=_plain_quantize, gemm=_plain_gemm, combine=_plain_combine, router=_plain_router)


def run(state):
    s, case = state, state["case"]
    if not own:
        return _PLAIN[case["op"]](s)
    import fp4_quantized_gemm_amd as F
    if case["op"] == "quantize":
        return F.mxfp4_restore(*F.mxfp4_quantize(s["x"], transpose=case["transpose"]))
    if case["op"] == "gemm":
        product = F.grouped_mxfp4_gemm_swiglu if case["swiglu"] else F.grouped_mxfp4_gemm
        return product(s["a_codes"], s["a_scales"], s["a_rows"], s["w_codes"], s["w_scales"], s["offsets"],
                       M_total=case["T"] * case["topk"])
    if case["op"] == "combine":
        return F.moe_unpermute_combine_backward(s["d_out"], s["y"], s["inv"], s["w"])
    dl, db = F.moe_permute_backward(s["ids"], s["w"], s["dw"], case["E"], want_bias=case["bias"])
    return (dl, db) if case["bias"] else dl


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        n = max(1, case["E"]) * case["M"] * case["K"]
        return dict(bytes=n * (2 + 2 * 0.53125 + 2), flops=4 * n)
    T, topk, E = case["T"], case["topk"], case["E"]
    P = T * topk
    if op == "combine":
        N = case["N"]
        return dict(bytes=2 * T * N + 4 * P * N + 12 * P, flops=3 * P * N)
    if op == "router":
        return dict(bytes=12 * P + 4 * T * E + (4 * E if case["bias"] else 0), flops=4 * P + (P if case["bias"] else 0))
    N, K = case["N"], case["K"]
    return dict(bytes=0.53125 * K * ((T if case["gather"] else P) + min(E, P) * N)
                + 2 * P * (N // 2 if case["swiglu"] else N), flops=2 * P * N * K)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_quantized(x):
    """x on its blocks' E2M1 grids: steps of 2^E / 2 up to 2 * 2^E, of 2^E up
    to 4 * 2^E, of 2 * 2^E above, at most 6 * 2^E."""
    v = x.double().reshape(-1, 32)
    top = v.abs().max(1, keepdim=True).values
    E = torch.ceil(torch.log2(top / 7))                        # -inf for a block of zeros
    E = torch.where(7 * torch.exp2(E - 1) >= top, E - 1, E).clamp(-125, 125)
    u = v / torch.exp2(E)
    step = torch.exp2(torch.floor(torch.log2(u.abs())).clamp(0, 2) - 1)
    return ((torch.round(u / step) * step).clamp(-6, 6) * torch.exp2(E)).reshape(x.shape)


def _exact_values(codes, scales):
    """E2M1 codes by their fields, the lower one first, times 2^(byte - 127)."""
    c = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.long, device="cuda")
    c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
    e, m = (c // 2) % 4, (c % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    v = torch.where(c >= 8, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"]
        return _exact_quantized(x.transpose(-1, -2).contiguous() if case["transpose"] else x)
    P = case["T"] * case["topk"]
    if op == "combine":
        rows = s["inv"].long()
        dy = torch.empty(P, case["N"], dtype=F64, device="cuda")
        dw = torch.empty(case["T"], case["topk"], dtype=F64, device="cuda")
        d = s["d_out"].double()
        for j in range(case["topk"]):
            dy[rows[:, j]] = d * s["w"][:, j:j + 1].double()
            dw[:, j] = torch.einsum("tn,tn->t", d, s["y"][rows[:, j]].double())
        return dy, dw
    if op == "router":
        w, dw = s["w"].double(), s["dw"].double()
        # row by row the softmax's Jacobian, diag(w) - w w^T
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        dl = (jac * dw[:, None, :]).sum(2)
        out = torch.zeros(case["T"], case["E"], dtype=F64, device="cuda")
        out[torch.arange(case["T"], device="cuda")[:, None], s["ids"].long()] = dl
        return (out, out.sum(0)) if case["bias"] else out
    off = s["offsets"].tolist()
    N = case["N"]
    out = torch.empty(P, N // 2 if case["swiglu"] else N, dtype=F64, device="cuda")
    for e in range(case["E"]):
        at = slice(off[e], off[e + 1])
        pick = at if s["a_rows"] is None else s["a_rows"][at].long()
        y = _exact_values(s["a_codes"][pick], s["a_scales"][pick]) @ \
            _exact_values(s["w_codes"][e], s["w_scales"][e]).t()
        out[at] = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:] if case["swiglu"] else y
    return out
