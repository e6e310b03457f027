"""Operators around the sparse MoE layer: the cases they are measured on, and their plain forms.

Four operators of a served block, each with listed cases:

* ``select``  experts and weights from router logits: softmax or sigmoid scores, a bias for
              balance, groups of experts, top-k, renormalised and scaled weights
* ``route``   the same rule from hidden states (the router's product included)
* ``norm``    the norm after a block, its gate and residual scale, the residual stream, and the
              norm before the next block, in one pass
* ``lora``    low-rank adapters of many requests added beside a shared projection

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits (scores
and logits that are compared with one another in 64); with ``own`` true it makes the
library's calls.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token: sigmoid scores, a balance bias, 4 of 8 groups by their two best
        dict(name="select-token", op="select", T=1, E=256, k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5),
        # logits of a packed prompt in bf16 (many of them equal), softmax without renormalising
        dict(name="select-packed", op="select", T=4099, E=60, k=4, dtype="bf16", score="softmax", bias=False,
             groups=1, keep=1, group_score="max", renorm=False, scale=1.0),
        # the router logits of a long prompt, grouped and biased
        dict(name="select-prompt", op="select", T=16384, E=256, k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5),
        # one token's hidden state to its experts
        dict(name="route-token", op="route", T=1, H=2048, E=256, k=8, score="sigmoid", bias=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5),
        # a decode batch, softmax over all experts, a group kept by its best expert
        dict(name="route-batch48", op="route", T=48, H=2048, E=256, k=8, score="softmax", bias=False,
             groups=4, keep=2, group_score="max", renorm=True, scale=1.0),
        # one token: a block's output joins the residual stream, norm before the next block
        dict(name="norm-token", op="norm", mode="join", T=1, H=2048, y="bf16", r="bf16", x="bf16", kind="rms",
             post=False, gate="none", act="none", scale=1.0, pre=True, offset=0.0),
        # a ragged decode batch of odd width: norm of the output, gate, residual scale, fp32 stream, next norm
        dict(name="norm-batch37", op="norm", mode="join", T=37, H=2047, y="f16", r="f32", x="f16", kind="layer",
             post=True, gate="token", act="sigmoid", scale=0.22, pre=True, offset=0.0),
        # the gated norm of attention heads over a prompt: 32 heads of 128 per token
        dict(name="norm-heads", op="norm", mode="gated", T=131072, H=128, y="bf16", r="bf16", x="bf16", kind="rms",
             post=True, gate="element", act="silu", scale=1.0, pre=False, offset=0.0),
        # a long prompt through both norms of a wide block
        dict(name="norm-prompt", op="norm", mode="join", T=16384, H=8192, y="bf16", r="bf16", x="bf16", kind="rms",
             post=True, gate="none", act="none", scale=1.0, pre=True, offset=1.0),
        # one token's adapter beside the attention output projection
        dict(name="lora-token", op="lora", T=1, K=2048, N=2048, R=16, adapters=8, order="mixed", ragged=False, y="bf16"),
        # a decode batch in which nearly every request has its own adapter, beside the gate/up projection
        dict(name="lora-batch48", op="lora", T=48, K=2048, N=16384, R=64, adapters=40, order="mixed", ragged=True,
             y="f32"),
        # packed prompts of a few requests, beside the gate/up projection
        dict(name="lora-prompt", op="lora", T=4096, K=2048, N=16384, R=32, adapters=6, order="packed", ragged=True,
             y="bf16"),
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(int(v / multiple) * multiple, lo), hi)


def _draw_rule(rng, E):
    """A rule over E experts and its top_k: groups of at least two experts."""
    fits = [g for g in range(2, 33) if E % g == 0 and E // g >= 2]
    groups = rng.choice(fits) if fits and rng.random() < 0.6 else 1
    k = rng.randint(1, min(8, E))
    least = -(-k // (E // groups))                          # groups that hold k experts
    return dict(E=E, k=k, score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                keep=rng.randint(least, groups), group_score=rng.choice(("max", "top2")), renorm=rng.random() < 0.7,
                scale=rng.choice((1.0, 2.5)))


def draw(rng):
    op = rng.choice(("select", "route", "norm", "lora"))
    if op == "select":
        return dict(op=op, T=_log_int(rng, 1, 16384), dtype=rng.choice(("bf16", "f16", "f32")),
                    **_draw_rule(rng, _log_int(rng, 8, 256)))
    if op == "route":
        return dict(op=op, T=_log_int(rng, 1, 64), H=_log_int(rng, 256, 2048, 64),
                    **_draw_rule(rng, _log_int(rng, 8, 256)))
    if op == "norm":
        mode = rng.choice(("join", "join", "pre", "gated"))
        H = _log_int(rng, 64, 8192, rng.choice((1, 8, 64)))
        gate = "none" if mode == "pre" else rng.choice(("none", "token", "element"))
        post = mode == "gated" or (mode == "join" and rng.random() < 0.5)
        kind = rng.choice(("rms", "rms", "layer"))
        return dict(op=op, mode=mode, T=_log_int(rng, 1, 2 ** 25 // H), H=H, y=rng.choice(("bf16", "f16", "f32")),
                    r=rng.choice(("bf16", "f16", "f32")), x=rng.choice(("bf16", "f16", "f32")), kind=kind, post=post,
                    gate=gate, act="none" if gate == "none" else rng.choice(("none", "sigmoid", "silu")),
                    scale=1.0 if mode == "pre" else rng.choice((1.0, 0.22)), pre=mode == "pre" or rng.random() < 0.8,
                    offset=rng.choice((0.0, 1.0)) if kind == "rms" else 0.0)
    T = _log_int(rng, 1, 4096)
    N = _log_int(rng, 64, 16384, rng.choice((1, 16, 64)))
    return dict(op=op, T=T, K=_log_int(rng, 64, 2048, 32), N=N, R=rng.choice((8, 16, 32, 64)),
                adapters=rng.randint(1, 8 if T > 64 else 40), order=rng.choice(("packed", "mixed")),
                ragged=rng.random() < 0.5, y=rng.choice(("bf16", "f32")))


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


def _adapter_ids(g, case):
    """The adapter of each token, one in eight requests without (-1): runs of tokens of a
    request for packed prompts, any order for decoded tokens."""
    T, n = case["T"], case["adapters"]
    if case["order"] == "packed":
        # as many requests as adapters, of uneven lengths, each with any adapter
        cut = torch.sort(torch.randint(0, T, (n - 1,), generator=g, device="cuda"))[0]
        request = torch.searchsorted(cut, torch.arange(T, device="cuda"), right=True)
        which = torch.randint(0, n, (n,), generator=g, device="cuda")
        without = torch.randint(0, 8, (n,), generator=g, device="cuda") == 0
        ids = torch.where(without, torch.full_like(which, -1), which)[request]
    else:
        ids = torch.randint(0, n, (T,), generator=g, device="cuda")
        if T > 1:
            ids = torch.where(torch.randint(0, 8, (T,), generator=g, device="cuda") == 0, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32)


def _inputs(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    if op in ("select", "route"):
        E = case["E"]
        d = dict(bias=0.1 * _randn(g, E) if case["bias"] else None)
        if op == "select":
            d["logits"] = (1.5 * _randn(g, T, E)).to(_DT[case["dtype"]])
        else:
            d["x"] = _activations(g, T, case["H"]).to(torch.bfloat16)
            d["router_w"] = (_randn(g, E, case["H"]) / math.sqrt(case["H"])).to(torch.bfloat16)
        return d
    if op == "norm":
        H = case["H"]
        d = dict(y=None, r=None, gate=None, post=None, pre=None)
        if case["mode"] != "pre":
            d["y"] = _randn(g, T, H).mul_(torch.exp(0.5 * _randn(g, T, 1))).to(_DT[case["y"]])
        if case["mode"] != "gated":
            r = _activations(g, T, H)
            d["r"] = r.mul_(torch.exp(0.5 * _randn(g, T, 1))).to(_DT[case["r"]])
        if case["gate"] != "none":
            d["gate"] = _randn(g, T, H if case["gate"] == "element" else 1).to(_DT[case["y"]])
        for which in ("post", "pre"):
            if case[which]:
                w = (1.0 - case["offset"] + 0.2 * _randn(g, H)).to(torch.bfloat16)
                d[which] = (w, (0.1 * _randn(g, H)).to(torch.bfloat16) if case["kind"] == "layer" else None)
        return d
    K, N, R, n = case["K"], case["N"], case["R"], case["adapters"]
    d = dict(x=_activations(g, T, K).to(torch.bfloat16), ids=_adapter_ids(g, case),
             a=(_randn(g, n, R, K) / math.sqrt(K)).to(torch.bfloat16),
             b=(_randn(g, n, N, R) / math.sqrt(R)).to(torch.bfloat16),
             scales=0.5 + torch.rand(n, generator=g, device="cuda"),
             base=_randn(g, T, N).to(_DT[case["y"]]), ranks=None)
    if case["ragged"]:
        d["ranks"] = torch.randint(1, R // 4 + 1, (n,), generator=g, device="cuda", dtype=torch.int32) * 4
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import quantized_sparse_moe_amd as qs
        s["qs"] = qs
        op = case["op"]
        if op in ("select", "route"):
            s["rule"] = qs.RouterRule(score=case["score"], renorm=case["renorm"], n_groups=case["groups"],
                                      group_top_k=case["keep"], group_score=case["group_score"], scale=case["scale"],
                                      select_bias=s["bias"])
        if op == "route":
            # the layer's experts (small ones: routing does not read them) and its workspace
            H, E, I = case["H"], case["E"], 64
            gu, dn = (qs.mx4_quantize(torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"))
                      for rows, cols in ((E * 2 * I, H), (E * H, I)))
            s["desc"] = qs.LayerDesc.from_mx4(H, I, E, case["k"], s["router_w"], gu, dn)
            s["ws"] = qs.new_workspace(s["desc"], case["T"])
        elif op == "norm":
            for which in ("post", "pre"):
                if s[which]:
                    w, b = s[which]
                    s[which] = qs.Norm(case["kind"], weight=w, bias=b, eps=EPS, offset=case["offset"])
        elif op == "lora":
            s["adapters"] = qs.LoraAdapters(s["a"], s["b"], scales=s["scales"], ranks=s["ranks"])
            s["ws"] = qs.lora_new_workspace(s["adapters"], case["T"])
    return s


# ------------------------------------------------------------------------- plain forms
def _select_plain(case, logits, bias):
    """The rule on float64 logits: scores are compared with their neighbours."""
    E, k, G = case["E"], case["k"], case["groups"]
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
    c = s if bias is None else s + bias.double()
    if G > 1:
        best = torch.sort(c.view(-1, G, E // G), dim=2, descending=True)[0]
        value = best[:, :, 0] + best[:, :, 1] if case["group_score"] == "top2" else best[:, :, 0]
        kept = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :case["keep"]]
        mask = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(E // G, dim=1), c, torch.full_like(c, -math.inf))
    idx = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :k]
    idx = torch.sort(idx, dim=1)[0]
    w = torch.gather(s, 1, idx)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.int(), (w * case["scale"]).float()


def _norm_rows(v, case, weights):
    if case["kind"] == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    w, b = weights
    v = v * (case["offset"] + w.float())
    return v if b is None else v + b.float()


def _norm_plain(s):
    case = s["case"]
    z = None
    if s["y"] is not None:
        z = s["y"].float()
        if s["post"]:
            z = _norm_rows(z, case, s["post"])
        if s["gate"] is not None:
            g = s["gate"].float()
            if case["act"] == "sigmoid":
                g = 1.0 / (1.0 + torch.exp(-g))
            elif case["act"] == "silu":
                g = g / (1.0 + torch.exp(-g))
            z = z * g
        z = z * case["scale"]
    r = z if s["r"] is None else s["r"].float() if z is None else s["r"].float() + z
    out = []
    if z is not None:
        out.append(r.to(_DT[case["r"]]))
    if s["pre"]:
        out.append(_norm_rows(r, case, s["pre"]).to(_DT[case["x"]]))
    return tuple(out)


def _lora_plain(s):
    case = s["case"]
    x = s["x"].float()
    y = s["base"].float()
    for i in range(case["adapters"]):
        mine = s["ids"] == i
        v = x @ s["a"][i].float().t()
        if s["ranks"] is not None:
            v = v * (torch.arange(case["R"], device="cuda") < s["ranks"][i])
        v = torch.where(mine.unsqueeze(1), v * s["scales"][i], torch.zeros_like(v))
        y = y + v @ s["b"][i].float().t()
    return y.to(_DT[case["y"]])


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "select":
        return _select_plain(case, s["logits"].double(), s["bias"])
    if op == "route":
        return _select_plain(case, s["x"].double() @ s["router_w"].double().t(), s["bias"])
    return _norm_plain(s) if op == "norm" else _lora_plain(s)


# --------------------------------------------------------------------------------- run
def run(state):
    if not own:
        return _plain(state)
    qs, case = state["qs"], state["case"]
    op = case["op"]
    if op == "select":
        return qs.moe_select(state["logits"], case["k"], state["rule"])
    if op == "route":
        return qs.moe_route(state["desc"], state["x"], workspace=state["ws"], rule=state["rule"])
    if op == "norm":
        out = qs.moe_block_norm(state["y"], residual=state["r"], post=state["post"], gate=state["gate"],
                                gate_act=case["act"], scale=case["scale"], pre=state["pre"], r_dtype=_DT[case["r"]],
                                x_dtype=_DT[case["x"]])
        return tuple(t for t in out if t is not None)
    return qs.lora_gemm(state["adapters"], state["ids"], state["x"], base=state["base"], y_dtype=_DT[case["y"]],
                        workspace=state["ws"])


# ---------------------------------------------------------------------- exact, 64 bits
def _select64(case, logits, bias):
    """The rule on a float64 numpy array [T, E]: by rank, an expert at a time."""
    T, E = logits.shape
    G, k = case["groups"], case["k"]
    if case["score"] == "sigmoid":
        score = np.where(logits >= 0, 1 / (1 + np.exp(-np.abs(logits))),
                         np.exp(-np.abs(logits)) / (1 + np.exp(-np.abs(logits))))
    else:
        score = np.exp(logits - logits.max(axis=1)[:, None])
        score /= score.sum(axis=1)[:, None]
    value = score + bias if bias is not None else score.copy()
    if G > 1:
        part = np.sort(value.reshape(T, G, E // G), axis=2)
        rank = part[:, :, -1] + (part[:, :, -2] if case["group_score"] == "top2" else 0.0)
        order = np.argsort(-rank, axis=1, kind="stable")
        for j in range(case["keep"], G):
            for i in range(E // G):
                value[np.arange(T), order[:, j] * (E // G) + i] = -np.inf
    order = np.sort(np.argsort(-value, axis=1, kind="stable")[:, :k], axis=1)
    wt = np.take_along_axis(score, order, axis=1)
    if case["renorm"]:
        wt = wt / wt.sum(axis=1)[:, None]
    return (torch.as_tensor(order.astype(np.int32), device="cuda"),
            torch.as_tensor(wt * case["scale"], device="cuda"))


def _norm64(case, d):
    def scaled(v, weights):
        m = v.mean(dim=1, keepdim=True) if case["kind"] == "layer" else 0.0
        u = torch.var(v, dim=1, correction=0, keepdim=True) if case["kind"] == "layer" else v.pow(2).mean(1, True)
        v = (v - m) * torch.rsqrt(u + EPS) * (weights[0].double() + case["offset"])
        return v if weights[1] is None else v + weights[1].double()

    total = d["r"].double() if d["r"] is not None else 0.0
    out = []
    if d["y"] is not None:
        v = d["y"].double()
        if d["post"]:
            v = scaled(v, d["post"])
        if d["gate"] is not None:
            gate = d["gate"].double()
            act = {"none": lambda t: t, "sigmoid": torch.sigmoid, "silu": lambda t: t * torch.sigmoid(t)}[case["act"]]
            v = v * act(gate)
        total = total + v * case["scale"]
        out.append(total)
    if d["pre"]:
        out.append(scaled(total, d["pre"]))
    return tuple(out)


def _lora64(case, d):
    y = d["base"].double()
    ids = d["ids"].cpu().numpy()
    for i in range(case["adapters"]):
        rows = np.nonzero(ids == i)[0]
        if len(rows):
            rows = torch.as_tensor(rows, device="cuda")
            r = case["R"] if d["ranks"] is None else int(d["ranks"][i])
            low = d["x"][rows].double() @ d["a"][i, :r].double().t()
            y[rows] += float(d["scales"][i]) * (low @ d["b"][i, :, :r].double().t())
    return y


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op in ("select", "route"):
        logits = d["logits"].double() if op == "select" else (d["x"].double() @ d["router_w"].double().t())
        return _select64(case, logits.cpu().numpy(), None if d["bias"] is None else d["bias"].double().cpu().numpy())
    return _norm64(case, d) if op == "norm" else _lora64(case, d)


# -------------------------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["T"]
    if op in ("select", "route"):
        E, k = case["E"], case["k"]
        bias = 4 * E if case["bias"] else 0
        if op == "select":
            return {"bytes": T * E * _SIZE[case["dtype"]] + 8 * T * k + bias, "flops": 20 * T * E}
        return {"bytes": 2 * E * case["H"] + 2 * T * case["H"] + 8 * T * k + bias, "flops": 2 * T * E * case["H"]}
    if op == "norm":
        H, per = case["H"], 0
        if case["mode"] != "pre":
            per += _SIZE[case["y"]] + _SIZE[case["r"]]          # y read, the stream written
        if case["mode"] != "gated":
            per += _SIZE[case["r"]]
        if case["gate"] == "element":
            per += _SIZE[case["y"]]
        if case["pre"]:
            per += _SIZE[case["x"]]
        return {"bytes": T * H * per, "flops": T * H * (2 + 4 * case["post"] + 4 * case["pre"])}
    K, N, R, n = case["K"], case["N"], case["R"], case["adapters"]
    rank = R if not case["ragged"] else (R + 4) / 2             # on average
    live = 1.0 if T == 1 else 7 / 8                             # tokens with an adapter
    used = n * (1.0 - (1.0 - 1.0 / n) ** (n if case["order"] == "packed" else T * live))
    return {"bytes": int(2 * T * K + 2 * _SIZE[case["y"]] * T * N + used * rank * 2 * (K + N)),
            "flops": int(2 * T * live * rank * (K + N))}
