"""Microscaled 4-bit (MX4) operators: the cases they are measured on, and their plain forms.

MX4 is the OCP microscaling format with FP4 (E2M1) elements: blocks of 32 consecutive
values along the reduction axis share one power-of-two scale (E8M0, a biased exponent
byte), v = 2^(s - 127) * e2m1(code).

Four operators, each with listed cases:

* ``quantize``  values -> MX4 codes and scales, returned as the values they stand for
* ``gemm``      y = x W^T with x bf16 and W in MX4
* ``gemm_mx``   y = x W^T with x quantized to MX4 in the call, W in MX4
* ``moe``       the sparse mixture-of-experts layer of a few tokens with MX4 experts:
                router, top-k, SwiGLU experts, shared expert, weighted combine

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits;
with ``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
# magnitudes of the eight E2M1 codes; bit 3 of a code is the sign
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's hidden state, quantized before a projection: launch latency
        dict(name="quantize-token", op="quantize", rows=1, K=2048, dtype="bf16", layout="tiles"),
        # the activations of a long prompt, quantized once for the projections that read them
        dict(name="quantize-prompt", op="quantize", rows=4096, K=8192, dtype="bf16", layout="tiles"),
        # a weight matrix of odd shape, quantized at load time from fp32 into row-major blocks
        dict(name="quantize-weight", op="quantize", rows=16390, K=2080, dtype="f32", layout="rows"),
        # the attention output projection of one token
        dict(name="gemm-token", op="gemm", T=1, N=2048, K=2048, y="bf16"),
        # the fused gate/up projection for a small batch of decoding requests
        dict(name="gemm-batch5", op="gemm", T=5, N=16384, K=2048, y="f32"),
        # the down projection for a ragged decode batch
        dict(name="gemm-batch37", op="gemm", T=37, N=2048, K=8192, y="bf16"),
        # the fused gate/up projection of a long prompt
        dict(name="gemm-prompt", op="gemm", T=4096, N=16384, K=2048, y="bf16"),
        # the down projection of three tokens (a verification batch), activations quantized
        dict(name="gemm_mx-batch3", op="gemm_mx", T=3, N=2048, K=8192, y="f32"),
        # the fused gate/up projection of a long prompt, activations quantized
        dict(name="gemm_mx-prompt", op="gemm_mx", T=4096, N=16384, K=2048, y="bf16"),
        # one decoded token through the MoE layer
        dict(name="moe-token", op="moe", T=1, hidden=2048, inter=512, experts=256, top_k=8,
             shared=True, gated=False, bias=False, y="bf16"),
        # a small decode batch, with the sigmoid-gated shared expert
        dict(name="moe-batch7", op="moe", T=7, hidden=2048, inter=512, experts=256, top_k=8,
             shared=True, gated=True, bias=False, y="bf16"),
        # a wider decode batch under a skewed router
        dict(name="moe-batch48", op="moe", T=48, hidden=2048, inter=512, experts=256, top_k=8,
             shared=True, gated=False, bias=True, y="bf16"),
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(int(v / multiple) * multiple, lo), hi)


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm_mx", "moe"))
    if op == "quantize":
        dtype = rng.choice(("bf16", "f16", "f32"))
        K = _log_int(rng, 64, 8192, 32)
        rows = _log_int(rng, 1, 30_000_000 // K)
        return dict(op=op, rows=rows, K=K, dtype=dtype, layout=rng.choice(("tiles", "rows")))
    if op in ("gemm", "gemm_mx"):
        T = _log_int(rng, 1, 4096)
        N = _log_int(rng, 64, 16384, rng.choice((1, 16, 64)))
        K = _log_int(rng, 64, min(8192, 2 ** 37 // (T * N)) if T * N > 2 ** 24 else 8192, 32)
        return dict(op=op, T=T, N=N, K=K, y=rng.choice(("bf16", "f32")))
    shared = rng.random() < 0.75
    experts = _log_int(rng, 8, 256)
    return dict(op=op, T=_log_int(rng, 1, 48), hidden=_log_int(rng, 256, 2048, 64),
                inter=_log_int(rng, 128, 512, 64), experts=experts, top_k=rng.randint(1, min(8, experts)),
                shared=shared, gated=shared and rng.random() < 0.5, bias=rng.random() < 0.5,
                y="bf16")


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, K):
    """N(0, 1) values with a few channels of large magnitude, as hidden states have them."""
    x = _randn(g, rows, K)
    loud = torch.randperm(K, generator=g, device="cuda")[:max(K // 256, 1)]
    x[:, loud] *= 8.0
    return x


def _weights_mx4(g, rows, K):
    """Row-major MX4 codes [rows, K/2] and scales [rows, K/32] of N(0, s^2 / K) rows with
    a spread of row scales s."""
    w = _randn(g, rows, K) * (torch.exp(0.5 * _randn(g, rows, 1)) / math.sqrt(K))
    c, s = _quantize_plain(w)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        x = _activations(g, case["rows"], case["K"]) * torch.exp(_randn(g, case["rows"], 1))
        return dict(x=x.to(_DT[case["dtype"]]))
    if op in ("gemm", "gemm_mx"):
        codes, scales = _weights_mx4(g, case["N"], case["K"])
        return dict(x=_activations(g, case["T"], case["K"]).to(torch.bfloat16), w=(codes, scales))
    H, I, E = case["hidden"], case["inter"], case["experts"]
    d = dict(x=_activations(g, case["T"], H).to(torch.bfloat16),
             router_w=(_randn(g, E, H) / math.sqrt(H)).to(torch.bfloat16),
             gate_up=_weights_mx4(g, E * 2 * I, H), down=_weights_mx4(g, E * H, I))
    d["bias"] = None
    if case["bias"]:
        # a Zipf-like load: a few experts far above the mean
        r = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        d["bias"] = -1.1 * torch.log(r)
    d["shared"] = d["gate_w"] = None
    if case["shared"]:
        d["shared"] = (_weights_mx4(g, 2 * I, H), _weights_mx4(g, H, I))
    if case["gated"]:
        d["gate_w"] = (_randn(g, H) / math.sqrt(H)).to(torch.bfloat16)
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import quantized_sparse_moe_amd as qs
        s["qs"] = qs
        op = case["op"]
        if op in ("gemm", "gemm_mx"):
            # load time: the weights in the product's tile order, and a workspace
            s["w"] = qs.mx4_pack_rows16(*s["w"], case["N"], case["K"])
            s["ws"] = qs.mx4_new_workspace(case["T"], case["N"], case["K"])
        elif op == "moe":
            H, I, E = case["hidden"], case["inter"], case["experts"]
            gu = qs.mx4_pack_rows16(*s["gate_up"], E * 2 * I, H)
            dn = qs.mx4_pack_rows16(*s["down"], E * H, I)
            sh = None
            if s["shared"]:
                sh = (qs.mx4_pack_rows16(*s["shared"][0], 2 * I, H), qs.mx4_pack_rows16(*s["shared"][1], H, I))
            s["gate_up"] = s["down"] = s["shared"] = None
            s["desc"] = qs.LayerDesc.from_mx4(H, I, E, case["top_k"], s["router_w"], gu, dn,
                                              router_bias=s["bias"], shared=sh, shared_gate_w=s["gate_w"])
            s["ws"] = qs.new_workspace(s["desc"], case["T"])
            s["idx"] = torch.empty(case["T"], case["top_k"], dtype=torch.int32, device="cuda")
            s["wt"] = torch.empty(case["T"], case["top_k"], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms
def _pow2(n):
    """2^n in fp32, exact, for integers -127 <= n <= 127 (2^-127 is subnormal)."""
    n = n.to(torch.int32)
    return torch.where(n > -127, (n + 127) << 23, torch.full_like(n, 1 << 22)).view(torch.float32)


def _quantize_plain(x):
    """Codes uint8 [rows, K] (one per value) and scales uint8 [rows, K/32] of fp32 rows:
    the scale is the power of two that puts the block's largest value in [4, 8), elements
    round to the nearest code (ties to the even code) and saturate at 6."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(dim=2)
    e = torch.frexp(amax)[1] - 3                            # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    v = b * _pow2(-e).unsqueeze(2)
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = c + 8 * torch.signbit(v).to(torch.uint8)
    return c.reshape(x.shape), (e + 127).to(torch.uint8)


def _dequantize_plain(c, s):
    """fp32 values of one-per-value codes [..., K] and scales [..., K/32]."""
    table = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=torch.float32, device=c.device)
    v = table[c.int()].unflatten(-1, (-1, BLOCK)) * _pow2(s.int() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _weight_plain(codes, scales):
    """fp32 values of packed row-major codes [..., K/2] (column 2i in the low nibble)."""
    return _dequantize_plain(torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2), scales)


def _moe_plain(s):
    case = s["case"]
    H, I, E, k, T = case["hidden"], case["inter"], case["experts"], case["top_k"], case["T"]
    x = s["x"].float()
    # the logits in 64 bits: the selection is a comparison of neighbouring values
    logits = s["x"].double() @ s["router_w"].double().t()
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    idx = torch.sort(idx, dim=1)[0]
    sel = torch.gather(logits, 1, idx).float()
    w = torch.exp(sel - sel.amax(dim=1, keepdim=True))
    w = w / w.sum(dim=1, keepdim=True)

    def swiglu(v, gu):
        a = v @ gu.transpose(-1, -2)
        g, u = a[..., :I], a[..., I:]
        return g / (1.0 + torch.exp(-g)) * u

    guc, gus = (a.view(E, 2 * I, -1) for a in s["gate_up"])
    dnc, dns = (a.view(E, H, -1) for a in s["down"])
    # every (token, choice) with its expert's weights beside it
    h = swiglu(x.view(T, 1, 1, H).expand(T, k, 1, H), _weight_plain(guc[idx], gus[idx]))
    o = h @ _weight_plain(dnc[idx], dns[idx]).transpose(-1, -2)
    y = (w.unsqueeze(2) * o.view(T, k, H)).sum(dim=1)
    if s["shared"]:
        o = swiglu(x, _weight_plain(*s["shared"][0])) @ _weight_plain(*s["shared"][1]).t()
        if s["gate_w"] is not None:
            z = x @ s["gate_w"].float()
            o = o * (1.0 / (1.0 + torch.exp(-z))).unsqueeze(1)
        y = y + o
    return y.to(_DT[case["y"]]), idx.int(), w


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return _dequantize_plain(*_quantize_plain(s["x"])).to(_DT[case["dtype"]])
    if op == "gemm":
        return (s["x"].float() @ _weight_plain(*s["w"]).t()).to(_DT[case["y"]])
    if op == "gemm_mx":
        x = _dequantize_plain(*_quantize_plain(s["x"]))
        return (x @ _weight_plain(*s["w"]).t()).to(_DT[case["y"]])
    return _moe_plain(s)


# --------------------------------------------------------------------------------- run
def run(state):
    if not own:
        return _plain(state)
    qs, case = state["qs"], state["case"]
    op = case["op"]
    if op == "quantize":
        layout = qs.MX4_TILES if case["layout"] == "tiles" else qs.MX4_ROWS
        codes, scales = qs.mx4_quantize(state["x"], layout=layout)
        return qs.mx4_dequantize(codes, scales, case["rows"], case["K"], y_dtype=_DT[case["dtype"]], layout=layout)
    if op == "gemm":
        return qs.mx4_gemm(*state["w"], case["N"], case["K"], state["x"], y_dtype=_DT[case["y"]],
                           workspace=state["ws"])
    if op == "gemm_mx":
        xc, xs = qs.mx4_quantize(state["x"], layout=qs.MX4_TILES)
        return qs.mx4_gemm_mx4x(*state["w"], case["N"], case["K"], xc, xs, case["T"], y_dtype=_DT[case["y"]],
                                workspace=state["ws"])
    y = qs.moe_layer_forward(state["desc"], state["x"], y_dtype=_DT[case["y"]], topk_idx=state["idx"],
                             topk_w=state["wt"], workspace=state["ws"])
    return y, state["idx"], state["wt"]


# ---------------------------------------------------------------------- exact, 64 bits
def _exp2_64(n):
    """2^n in float64, exact, for integral -1022 <= n <= 1023."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _values64(codes, scales):
    """float64 values of packed row-major MX4, from the bits of the format: sign, two
    exponent bits (bias 1, 0 = subnormal) and one mantissa bit."""
    lohi = torch.stack((codes.bitwise_and(0x0F), codes.bitwise_right_shift(4)), -1)
    n = lohi.reshape(*codes.shape[:-1], codes.shape[-1] * 2).to(torch.float64)
    neg = n >= 8
    n = n - 8 * neg
    expo = torch.floor(n / 2)
    mant = n - 2 * expo
    mag = torch.where(expo > 0, (1 + mant / 2) * _exp2_64(expo - 1), mant / 2)
    v = torch.where(neg, -mag, mag)
    return v * torch.repeat_interleave(_exp2_64(scales.to(torch.int64) - 127), BLOCK, dim=-1)


def _nearest64(x):
    """float64 values of x after MX4 quantization: the nearest of the code magnitudes
    under the block's scale, ties to the code whose last bit is 0."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    b = x.double().reshape(-1, BLOCK)
    big = b.abs().max(dim=1, keepdim=True)[0]
    lg = torch.floor(torch.log2(torch.clamp(big, min=2.0 ** -140)))
    lg = torch.where(_exp2_64(lg) > big, lg - 1, lg)                    # log2 next to a power of two
    lg = torch.where(_exp2_64(lg + 1) <= big, lg + 1, lg)
    unit = _exp2_64(torch.clamp(lg - 2, min=-127.0))
    a = (b / unit).abs()
    lo = torch.bucketize(a, mid, right=False)                           # a tie stays with the lower code
    hi = torch.bucketize(a, mid, right=True)                            # a tie goes to the upper code
    code = torch.where(lo % 2 == 0, lo, hi)
    return (torch.sign(b) * grid[code] * unit).reshape(x.shape)


def _moe64(case, d):
    H, I, E, k, T = case["hidden"], case["inter"], case["experts"], case["top_k"], case["T"]
    x = d["x"].double()
    score = (x.unsqueeze(1) * d["router_w"].double()).sum(dim=2)
    if d["bias"] is not None:
        score = score + d["bias"].double()
    score = score.cpu().numpy()
    order = np.argsort(-score, axis=1, kind="stable")[:, :k]
    order.sort(axis=1)
    part = np.take_along_axis(score, order, axis=1)
    wt = np.exp(part - part.max(axis=1, keepdims=True))
    wt /= wt.sum(axis=1, keepdims=True)

    def mlp(v, gate_up, down):
        m = _values64(*gate_up)
        g, u = v @ m[:I].t(), v @ m[I:].t()
        return (torch.sigmoid(g) * g * u) @ _values64(*down).t()

    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = np.nonzero(order == e)
        if len(t):
            o = mlp(x[torch.as_tensor(t, device="cuda")],
                    tuple(a[e * 2 * I:(e + 1) * 2 * I] for a in d["gate_up"]),
                    tuple(a[e * H:(e + 1) * H] for a in d["down"]))
            y[torch.as_tensor(t, device="cuda")] += torch.as_tensor(wt[t, j], device="cuda").unsqueeze(1) * o
    if d["shared"]:
        o = mlp(x, *d["shared"])
        if d["gate_w"] is not None:
            o = o * torch.sigmoid(x @ d["gate_w"].double()).unsqueeze(1)
        y = y + o
    return y, torch.as_tensor(order.astype(np.int32), device="cuda"), torch.as_tensor(wt, device="cuda")


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return _nearest64(d["x"])
    if op == "moe":
        return _moe64(case, d)
    x = d["x"].double() if op == "gemm" else _nearest64(d["x"])
    return x @ _values64(*d["w"]).t()


# -------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    mx = 0.5 + 1.0 / BLOCK                                   # bytes per MX4 value
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": 2 * n * size[case["dtype"]], "flops": 2 * n}
    if op in ("gemm", "gemm_mx"):
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": int(N * K * mx) + 2 * T * K + size[case["y"]] * T * N, "flops": 2 * T * N * K}
    T, H, I, E, k = case["T"], case["hidden"], case["inter"], case["experts"], case["top_k"]
    # distinct experts that T tokens of k choices reach under an even router
    touched = E * (1.0 - (1.0 - k / E) ** T) + (1 if case["shared"] else 0)
    per_token = k + (1 if case["shared"] else 0)
    return {"bytes": int(touched * 3 * H * I * mx) + 2 * E * H + 2 * T * H + size[case["y"]] * T * H + 8 * T * k,
            "flops": 2 * T * E * H + 2 * T * per_token * 3 * H * I}
