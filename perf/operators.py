"""The operators of one training step through the expert block, as cases that
can be timed: 8-bit activation checkpoints, the input and weight gradients of
the W4A16 expert product, and the SwiGLU's backward pass with the gradient of
the routing weights.

`run` computes an operator in its plain form (elementary torch operations in
float32, rounded once at the end), or, with `own` set, through this package.
"""
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a dense layer's input, kept for the backward pass: latency
        dict(name="checkpoint_dense", op="checkpoint", M=64, K=512, glu=False),
        # the input of a large prefill-sized block, once per layer and step
        dict(name="checkpoint_block_input", op="checkpoint", M=16384, K=4096, glu=False),
        # gate and up products of a 4096-token, top-8 block, kept while h is formed
        dict(name="checkpoint_gate_up", op="checkpoint", M=32768, K=1536, glu=True),
        # a dense layer at its smallest: latency
        dict(name="dgrad_dense", op="dgrad", T=64, topk=1, E=1, N=512, K=512, gather=False, skew=0.0),
        # few rows per expert: the weights' bytes count
        dict(name="dgrad_few_rows", op="dgrad", T=256, topk=8, E=128, N=4096, K=1536, gather=True, skew=0.0),
        # gate and up projection's input gradient, a router that prefers some experts
        dict(name="dgrad_gate_up", op="dgrad", T=4096, topk=8, E=128, N=1536, K=2048, gather=False, skew=0.5),
        # down projection's input gradient of a large block, the output's gradient gathered by token
        dict(name="dgrad_down", op="dgrad", T=16384, topk=8, E=128, N=4096, K=1536, gather=True, skew=0.0),
        # a dense layer at its smallest
        dict(name="wgrad_dense", op="wgrad", T=64, topk=1, E=1, N=512, K=512, gather="", skew=0.0, fp8=False, out="f32"),
        # gate and up projection's weight gradient from the 8-bit block input, float32 master gradients
        dict(name="wgrad_gate_up_fp8", op="wgrad", T=4096, topk=8, E=128, N=1536, K=2048, gather="x", skew=0.5,
             fp8=True, out="f32"),
        # down projection's weight gradient of a large block, bf16 gradients
        dict(name="wgrad_down", op="wgrad", T=16384, topk=8, E=128, N=4096, K=1536, gather="dy", skew=0.0,
             fp8=False, out="bf16"),
        # few tokens, activations kept in bf16
        dict(name="swiglu_few_rows", op="swiglu", T=256, topk=8, E=128, I=768, fp8=False),
        # a large block, gate and up kept in 8 bits
        dict(name="swiglu_fp8", op="swiglu", T=16384, topk=8, E=128, I=1024, fp8=True),
    ]


def draw(rng):
    def logu(lo, hi, step=1):
        v = lo * (hi / lo) ** rng.random()
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["checkpoint", "dgrad", "dgrad", "wgrad", "wgrad", "swiglu"])
    if op == "checkpoint":
        glu = rng.random() < 0.5
        return dict(op=op, M=logu(1, 16384), K=logu(64, 4096, 64 if glu else 32), glu=glu)
    E = rng.choice([1, 2, 8, 16, 60, 64, 128])
    topk = 1 if E == 1 else rng.choice([1, 2, 4, 8] if E >= 8 else [1, 2])
    if op == "swiglu":
        fp8 = rng.random() < 0.5
        return dict(op=op, T=logu(1, 65536 // topk), topk=topk, E=E, I=logu(32, 1536, 32 if fp8 else 8), fp8=fp8)
    T = logu(1, 65536 // topk)
    skew = rng.choice([0.0, 0.5, 1.0])
    if op == "dgrad":
        return dict(op=op, T=T, topk=topk, E=E, N=logu(16, 4096, 16), K=logu(64, 1536, 64),
                    gather=rng.random() < 0.5, skew=skew)
    fp8 = rng.random() < 0.5
    return dict(op=op, T=T, topk=topk, E=E, N=logu(8, 2048, 8), K=logu(32, 2048, 32 if fp8 else 8),
                gather=rng.choice(["", "x", "dy"]), skew=skew, fp8=fp8, out=rng.choice(["f32", "bf16"]))


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
    row, the row of each (token, slot), the routing weights."""
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
                inv=inv.view(T, topk).to(torch.int32), w=torch.softmax(top, 1))


def _weights(gen, E, N, K):
    """NVFP4 weights: row-major codes and block scales, the tensor scales, and
    the expert products' packed copy of the same bytes (per expert the tiles of
    16 rows x 64 columns, then the channel-major copy)."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 16, dtype=torch.uint8, device="cuda")
    g = torch.empty(E, device="cuda")
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for e in range(E):
        w = 0.02 * _randn(gen, N, K // 16, 16)
        g[e] = w.abs().amax() / 2688
        s = (w.abs().amax(2) / (6 * g[e])).to(torch.float8_e4m3fn)
        v = w / (s.float() * g[e])[..., None]
        c = torch.bucketize(v.abs(), steps).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        c = c.view(N, K // 2, 2)
        codes[e], scales[e] = c[..., 0] | (c[..., 1] << 4), s.view(torch.uint8)
    nt, kt = N // 16, K // 64
    pc = torch.empty(E, 2, nt, kt, 16, 32, dtype=torch.uint8, device="cuda")
    ps = torch.empty(E, 2, nt, kt, 16, 4, dtype=torch.uint8, device="cuda")
    pc[:, 0] = codes.view(E, nt, 16, kt, 2, 16).permute(0, 1, 3, 4, 2, 5).reshape(E, nt, kt, 16, 32)
    ps[:, 0] = scales.view(E, nt, 16, kt, 4).permute(0, 1, 3, 2, 4)
    cols = torch.stack([codes & 15, codes >> 4], 3).view(E, N, K).transpose(1, 2)
    pc[:, 1] = (cols[..., 0::2] | (cols[..., 1::2] << 4)).reshape(E, nt, kt, 16, 32)
    ps[:, 1] = scales.transpose(1, 2).reshape(E, nt, kt, 16, 4)
    return dict(codes=codes, scales=scales, g=g, packed_codes=pc, packed_scales=ps)


def _kept(x):
    """A tensor's 8-bit checkpoint, made as the operator's definition says."""
    M, K = x.shape
    b = x.view(M, K // 32, 32).float()
    m, e = torch.frexp(b.abs().amax(2))
    e = torch.clamp(e - 9 + (m > 0.875), min=-117)
    e = torch.where(m == 0, torch.full_like(e, -117), e)
    codes = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(M, K)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "checkpoint":
        s["x"] = _activation(gen, case["M"], case["K"])
        return s
    T, topk, E = case["T"], case["topk"], case["E"]
    r = _routing(gen, T, topk, E, case.get("skew", 0.0))
    P = T * topk
    s.update(r)
    if op == "dgrad":
        s["dy"] = _gradient(gen, T if case["gather"] else P, case["N"])
        s["dy_rows"] = r["rows"] if case["gather"] else None
        s.update(_weights(gen, E, case["N"], case["K"]))
    elif op == "wgrad":
        s["dy"] = _gradient(gen, T if case["gather"] == "dy" else P, case["N"])
        s["x"] = _activation(gen, T if case["gather"] == "x" else P, case["K"])
        s["dy_rows"] = r["rows"] if case["gather"] == "dy" else None
        s["x_rows"] = r["rows"] if case["gather"] == "x" else None
        s["x_scales"] = None
        if case["fp8"]:
            s["x"], s["x_scales"] = _kept(s["x"])
    else:
        s["y"] = _activation(gen, P, 2 * case["I"])
        s["y_scales"] = None
        if case["fp8"]:
            s["y"], s["y_scales"] = _kept(s["y"])
        s["dh"] = _gradient(gen, P, case["I"])
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _value(codes, scales):
    """What E4M3 codes with one power-of-two scale per 32 stand for."""
    M, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(M, K // 32, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).view(M, K)


def _padded(a, rows, offsets, longest):
    """Rows of `a` (gathered by `rows`) as [E][longest][...] in float32, zero
    behind each expert's last row, and the places of the real rows."""
    first, count = offsets[:-1].long(), offsets.diff().long()
    at = torch.arange(longest, device=a.device)
    there = at < count[:, None]
    row = torch.where(there, first[:, None] + at, 0)
    row = row if rows is None else rows.long()[row]
    return torch.where(there[..., None], a[row].float(), 0), there


def _weight_values(codes, scales):
    E, N, half = codes.shape
    table = torch.tensor(E2M1, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 3).int()
    q = table[c & 7] * (1 - 2 * (c >> 3))
    s = scales.view(torch.float8_e4m3fn).float()
    return (q.view(E, N, half // 8, 16) * s[..., None]).view(E, N, 2 * half)


def _plain_checkpoint(s):
    x, case = s["x"], s["case"]
    M, K = x.shape
    codes, scales = _kept(x)
    if not case["glu"]:
        return _value(codes, scales).to(BF16)
    gate, up = x.float().view(M, 2, K // 2).unbind(1)
    return _value(codes, scales).to(BF16), (gate / (1 + torch.exp(-gate)) * up).to(BF16)


def _plain_dgrad(s):
    dy, there = _padded(s["dy"], s["dy_rows"], s["offsets"], s["longest"])
    w = _weight_values(s["codes"], s["scales"])
    return (torch.bmm(dy, w) * s["g"][:, None, None])[there].to(BF16)


def _plain_wgrad(s):
    x = s["x"] if s["x_scales"] is None else _value(s["x"], s["x_scales"])
    dy, _ = _padded(s["dy"], s["dy_rows"], s["offsets"], s["longest"])
    x, _ = _padded(x, s["x_rows"], s["offsets"], s["longest"])
    return torch.bmm(dy.transpose(1, 2), x).to(F32 if s["case"]["out"] == "f32" else BF16)


def _plain_swiglu(s):
    y = s["y"].float() if s["y_scales"] is None else _value(s["y"], s["y_scales"])
    gate, up = y.view(y.shape[0], 2, -1).unbind(1)
    dh, inv = s["dh"].float(), s["inv"].long().view(-1)
    w = torch.empty(inv.numel(), 1, device=y.device)
    w[inv] = s["w"].view(-1, 1)
    sig = 1 / (1 + torch.exp(-gate))
    silu = gate * sig
    dy = torch.cat([w * dh * up * (sig + silu * (1 - sig)), w * dh * silu], 1)
    h = silu * up
    return dy.to(BF16), (w * h).to(BF16), (dh * h).sum(1)[inv].view(s["w"].shape)


_PLAIN = dict(checkpoint=_plain_checkpoint, dgrad=_plain_dgrad, wgrad=_plain_wgrad, swiglu=_plain_swiglu)


def run(state):
    s, case = state, state["case"]
    if not own:
        return _PLAIN[case["op"]](s)
    import fp4_quantized_gemm_amd as F
    if case["op"] == "checkpoint":
        c = F.mxfp8_checkpoint(s["x"], glu=case["glu"])
        x = F.mxfp8_restore(c["codes"], c["scales"])
        return (x, c["h"]) if case["glu"] else x
    if case["op"] == "dgrad":
        return F.grouped_w4a16_dgrad(s["dy"], s["dy_rows"], s["packed_codes"], s["packed_scales"], s["g"],
                                     s["offsets"], M_total=case["T"] * case["topk"])
    if case["op"] == "wgrad":
        return F.grouped_wgrad(s["dy"], s["dy_rows"], s["x"], s["x_rows"], s["offsets"], x_scales=s["x_scales"],
                               M_total=case["T"] * case["topk"], dtype=F32 if case["out"] == "f32" else BF16)
    return F.moe_swiglu_backward(s["y"], s["dh"], s["inv"], s["w"], y_scales=s["y_scales"])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "checkpoint":
        n = case["M"] * case["K"]
        return dict(bytes=n * (2 + 2 * (1 + 1 / 32) + 2) + (n if case["glu"] else 0), flops=4 * n)
    T, topk, E = case["T"], case["topk"], case["E"]
    P = T * topk
    if op == "swiglu":
        n = P * case["I"]
        return dict(bytes=n * (2 * (1 + 1 / 32 if case["fp8"] else 2) + 2 + 4 + 2) + 12 * P, flops=20 * n)
    N, K = case["N"], case["K"]
    if op == "dgrad":
        return dict(bytes=2 * N * (T if case["gather"] else P) + min(E, P) * N * K * 0.5625 + 2 * P * K,
                    flops=2 * P * N * K)
    return dict(bytes=2 * N * (T if case["gather"] == "dy" else P)
                + K * (T if case["gather"] == "x" else P) * (1 + 1 / 32 if case["fp8"] else 2)
                + E * N * K * (4 if case["out"] == "f32" else 2), flops=2 * P * N * K)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_kept(x):
    """x rounded to a 4-bit significand on each block's grid."""
    v = x.double().reshape(-1, 32)
    top = v.abs().max(1, keepdim=True).values
    E = torch.ceil(torch.log2(top / 448))                      # -inf for a block of zeros
    E = torch.where(448 * torch.exp2(E - 1) >= top, E - 1, E).clamp(min=-117)
    step = torch.exp2(torch.floor(torch.log2(v.abs())).clamp(min=E - 6) - 3)
    return (torch.round(v / step) * step).reshape(x.shape)


def _exact_values(codes, scales):
    """E4M3 bytes by their fields."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = torch.where(c >= 128, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        x = s["x"]
        if not case["glu"]:
            return _exact_kept(x)
        gate, up = x.double().chunk(2, 1)
        return _exact_kept(x), gate * torch.sigmoid(gate) * up
    if op == "swiglu":
        y = s["y"].double() if s["y_scales"] is None else _exact_values(s["y"], s["y_scales"])
        I, dh = case["I"], s["dh"].double()
        a, b = y[:, :I], y[:, I:]
        p = torch.sigmoid(a)
        w = torch.zeros(y.shape[0], dtype=F64, device="cuda").index_put_((s["inv"].long().flatten(),),
                                                                         s["w"].double().flatten())[:, None]
        d = torch.empty_like(y)
        d[:, :I] = dh * w * b * (p + a * p * torch.sigmoid(-a))
        d[:, I:] = dh * w * a * p
        h = a * p * b
        return d, w * h, torch.einsum("pi,pi->p", dh, h)[s["inv"].long()]
    off = s["offsets"].tolist()
    N, K, P = case["N"], case["K"], off[-1]
    pick = lambda a, rows, lo, hi: a[lo:hi] if rows is None else a[rows[lo:hi].long()]  # noqa: E731
    if op == "dgrad":
        out = torch.empty(P, K, dtype=F64, device="cuda")
        grid = torch.tensor([-v for v in E2M1], dtype=F64, device="cuda")
        grid = torch.cat([-grid, grid])
        for e in range(case["E"]):
            c = s["codes"][e].long()
            w = torch.empty(N, K, dtype=F64, device="cuda")
            w[:, 0::2], w[:, 1::2] = grid[c % 16], grid[c // 16]
            sc = s["scales"][e].view(torch.float8_e4m3fn).double()
            w *= sc.repeat_interleave(16, 1) * s["g"][e].double()
            out[off[e]:off[e + 1]] = pick(s["dy"], s["dy_rows"], off[e], off[e + 1]).double() @ w
        return out
    out = torch.empty(case["E"], N, K, dtype=F64, device="cuda")
    for e in range(case["E"]):
        d = pick(s["dy"], s["dy_rows"], off[e], off[e + 1]).double()
        x = pick(s["x"], s["x_rows"], off[e], off[e + 1])
        x = x.double() if s["x_scales"] is None else _exact_values(
            x, pick(s["x_scales"], s["x_rows"], off[e], off[e + 1]))
        out[e] = d.t() @ x
    return out
