"""Routing rules on the GPU against the plain 64-bit evaluation (rule_ref): the selection from
given logits, and the layers' routing and forward pass under a rule."""
import numpy as np
import pytest

import mx4_ref as ref
import oracle
import qsmoe_synth as syn
import rule_ref
from gpu_util import TAU, check_output, to_dev, y_to_np
from test_gpu_mx4_moe import check, run, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm device"
    return t


@pytest.fixture(scope="module")
def qs():
    import quantized_sparse_moe_amd as q
    q.lib()
    return q


RULES = {
    "plain": dict(),
    "all": dict(renorm=False),
    "sigmoid": dict(score="sigmoid", renorm=False, scale=2.5),
    "bias": dict(score="sigmoid", select_bias=True),
    "softbias": dict(score="softmax", renorm=False, select_bias=True, scale=-0.5),
    "group": dict(score="softmax", groups=(4, 2), group_score="max"),
    "group2": dict(score="sigmoid", groups=(8, 4), group_score="top2", scale=2.5),
    "group2bias": dict(score="sigmoid", groups=(8, 3), group_score="top2", select_bias=True),
    "groupbias": dict(score="softmax", groups=(5, 2), group_score="max", select_bias=True, renorm=False),
    "softgroup2": dict(score="softmax", groups=(3, 1), group_score="top2"),
}


def rule_for(name, E, k, seed=0):
    """The rule's arguments over E experts (groups only where they fit), numpy bias."""
    r = dict(RULES[name])
    g = r.pop("groups", None)
    if g and E % g[0] == 0 and E // g[0] * g[1] >= k:
        r.update(n_groups=g[0], group_top_k=g[1])
    else:
        r.pop("group_score", None)
    if r.get("select_bias"):
        r["select_bias"] = (0.1 * np.random.default_rng(seed + 5).standard_normal(E)).astype(np.float32)
    return r


def to_rule(r, torch, qs):
    r = dict(r)
    if r.get("select_bias") is not None:
        r["select_bias"] = torch.from_numpy(r["select_bias"]).cuda()
    return qs.RouterRule(**r)


def expect(logits, k, r):
    r = dict(r)
    if r.get("select_bias") is not None:
        r["select_bias"] = r["select_bias"].astype(np.float64)
    return rule_ref.select(logits, k, **r)


def check_select(idx, w, logits, k, r, what):
    """Experts equal; weights off by their one rounding to fp32 (half a step, 2^-24 of the
    value, 2^-150 where it is subnormal), the 64-bit evaluations by far less."""
    wi, ww, _ = expect(logits, k, r)
    assert np.array_equal(idx.cpu().numpy(), wi), what
    got = w.cpu().numpy().astype(np.float64)
    assert (np.abs(got - ww) <= 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(ww) + 2.0 ** -149).all(), what


@pytest.mark.parametrize("name", sorted(RULES))
@pytest.mark.parametrize("E,k", [(1, 1), (5, 5), (15, 3), (64, 8), (65, 16), (240, 6), (256, 8)])
@pytest.mark.parametrize("T", [1, 67])
def test_select(torch, qs, name, E, k, T):
    rng = np.random.default_rng(E * 100 + k + T)
    r = rule_for(name, E, k)
    rule = to_rule(r, torch, qs)
    l = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        x = torch.from_numpy(l).to(dt)                      # (bf16 logits: many are equal)
        idx, w = qs.moe_select(x.cuda(), k, rule)
        check_select(idx, w, x.double().numpy(), k, r, (name, E, k, T, dt))


def test_select_long(torch, qs):
    """A prompt: scores of neighbouring ranks lie as close as 1e-7 here and there."""
    r = rule_for("group2bias", 256, 8)
    l = (1.5 * np.random.default_rng(9).standard_normal((5003, 256))).astype(np.float32)
    idx, w = qs.moe_select(torch.from_numpy(l).cuda(), 8, to_rule(r, torch, qs))
    check_select(idx, w, l.astype(np.float64), 8, r, "long")


@pytest.mark.parametrize("name", ["plain", "bias", "group", "group2", "group2bias", "softgroup2"])
def test_close_scores(torch, qs, name):
    """Logits a few fp32 steps apart, and equal ones: the order is that of 64-bit scores.  (Steps of
    2^-21: sums of two scores a step d apart on either side of a third differ from its double by
    d^2 times a curvature of at least 0.03, a hundred times what 64 bits round.)"""
    E, k, T = 240, 7, 64
    rng = np.random.default_rng(4)
    base = (rng.choice([-1, 1], (T, 1)) * rng.uniform(1, 3, (T, 1))).astype(np.float32)
    l = (base * (1 + rng.integers(-3, 4, (T, E)) * 2.0 ** -21)).astype(np.float32)
    l[::2] = np.repeat(l[::2, ::8], 8, axis=1)
    r = rule_for(name, E, k)
    if r.get("select_bias") is not None:
        r["select_bias"] = (rng.integers(0, 2, E) * 2.0 ** -24).astype(np.float32)
    idx, w = qs.moe_select(torch.from_numpy(l).cuda(), k, to_rule(r, torch, qs))
    check_select(idx, w, l.astype(np.float64), k, r, name)


@pytest.mark.parametrize("name", ["bias", "group2", "group2bias", "softbias", "softgroup2", "groupbias"])
@pytest.mark.parametrize("spread", [1e-2, 1e-3, 1e-4, 1e-5])
def test_crowded_scores(torch, qs, name, spread):
    """Rows whose scores all lie close together: the cuts fall on either side of what fp32 scores can
    decide, and the selection is that of 64-bit scores on both."""
    E, k, T = 240, 6, 500
    rng = np.random.default_rng(21)
    l = (rng.uniform(-3, 3, (T, 1)) + spread * rng.standard_normal((T, E))).astype(np.float32)
    r = rule_for(name, E, k)
    if r.get("select_bias") is not None:
        r["select_bias"] = (spread * rng.standard_normal(E) + rng.choice([0.0, 3.0])).astype(np.float32)
    idx, w = qs.moe_select(torch.from_numpy(l).cuda(), k, to_rule(r, torch, qs))
    check_select(idx, w, l.astype(np.float64), k, r, name)


@pytest.mark.parametrize("name", ["bias", "softbias", "group2bias", "groupbias"])
@pytest.mark.parametrize("spread", [1e-1, 1e-3, 1e-5])
def test_disabled_experts(torch, qs, name, spread):
    """Experts disabled by a bias of -infinity or NaN, or by their logit under a huge bias, beside scores on
    either side of what fp32 decides: the cut's error is that of the others."""
    E, k, T = 240, 6, 300
    rng = np.random.default_rng(31)
    l = (rng.uniform(-3, 3, (T, 1)) + spread * rng.standard_normal((T, E))).astype(np.float32)
    r = rule_for(name, E, k)
    b = (spread * rng.standard_normal(E)).astype(np.float32)
    b[[3, 40, 41, 200]] = [-np.inf, -np.inf, np.nan, 3e38]
    l[:, 200] = -np.inf
    r["select_bias"] = b
    idx, w = qs.moe_select(torch.from_numpy(l).cuda(), k, to_rule(r, torch, qs))
    assert not np.isin(idx.cpu().numpy(), [3, 40, 41, 200]).any()
    check_select(idx, w, l.astype(np.float64), k, r, (name, spread))


@pytest.mark.parametrize("name", sorted(RULES))
def test_masked_logits(torch, qs, name):
    """-infinity, NaN, the type's lowest value and +infinity; rows with few live experts or none."""
    E, k, T = 120, 6, 40
    rng = np.random.default_rng(11)
    l = rng.standard_normal((T, E)).astype(np.float32)
    for t in range(T):
        n = rng.integers(0, E + 1)
        l[t, rng.permutation(E)[:n]] = [-np.inf, np.nan, np.finfo(np.float32).min][t % 3]
    l[0] = -np.inf
    l[1] = np.nan
    l[2] = np.finfo(np.float32).min
    l[3] = np.inf
    l[4, :] = -np.inf
    l[4, 77] = 0.25
    l[5, [3, 50]] = np.inf
    l[6] = 0.0
    l[6, ::2] = -0.0
    r = rule_for(name, E, k)
    if r.get("select_bias") is not None:
        r["select_bias"][[7, 9, 100]] = [-np.inf, np.nan, 3.0]
    idx, w = qs.moe_select(torch.from_numpy(l).cuda(), k, to_rule(r, torch, qs))
    check_select(idx, w, l.astype(np.float64), k, r, name)


@pytest.mark.parametrize("scale", [1.0, 2.5, -3.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_of_scores_near_the_end_of_64_bits(torch, qs, score, scale):
    """Selected scores of 6e-310 to 2e-308, one over which is no 64-bit number, beside experts that are not live.
    (64-bit numbers are 4.9e-324 apart there: a score, the sum and the quotient of two evaluations
    differ by some 4 e-15 each, within the slack of 6e-14 that check_select has.)"""
    E, T = 40, 24
    rng = np.random.default_rng(8)
    bias = None
    if score == "softmax":                                  # chosen by their bias, far below the row's largest
        l = rng.uniform(-712.0, -709.9, (T, E)).astype(np.float32)
        l[:, 17] = 0.0
        bias = np.full(E, 4.0, np.float32)
        bias[17] = 0.0
    else:
        l = rng.uniform(-709.5, -708.5, (T, E)).astype(np.float32)
    l[1::2, 3:] = np.where(np.arange(3, E) == 17, l[1::2, 3:], -np.inf)  # (three of them, and the largest)
    for k in (1, 2, 6):
        for b in ([bias] if bias is not None else [None, np.zeros(E, np.float32)]):
            r = dict(score=score, renorm=True, scale=scale, select_bias=b)
            idx, w = qs.moe_select(torch.from_numpy(l).cuda(), k, to_rule(r, torch, qs))
            assert w.isfinite().all()
            if k < 4:
                assert ((w.double().sum(1) / scale - 1).abs() < 1e-6).all()
            check_select(idx, w, l.astype(np.float64), k, r, (score, scale, k))


def test_strided_logits_and_caller_buffers(torch, qs):
    E, k, T = 100, 5, 37
    r = rule_for("bias", E, k)
    wide = torch.randn(T, 3 * E + 1, device="cuda")
    x = wide[:, E + 1:2 * E + 1]
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    qs.moe_select(x, k, to_rule(r, torch, qs), topk_idx=idx[:T], topk_w=w[:T])
    check_select(idx[:T], w[:T], x.double().cpu().numpy(), k, r, "strided")
    assert (idx[T] == -7).all() and (w[T] == -7).all()      # rows behind the last: as they were
    i0, w0 = qs.moe_select(x[:0], k, to_rule(r, torch, qs))
    assert i0.shape == (0, k) and w0.shape == (0, k)


def test_select_past_2_31_elements(torch, qs):
    """Rows so far apart that their offsets pass 32 bits."""
    E, k = 64, 4
    r = rule_for("sigmoid", E, k)
    ld = (1 << 31) // 3 + 5
    buf = torch.empty(4 * ld + E, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((5, E), (ld, 1))
    x.copy_(torch.randn(5, E))
    idx, w = qs.moe_select(x, k, to_rule(r, torch, qs))
    check_select(idx, w, x.double().cpu().numpy(), k, r, "far")


def test_select_on_streams_and_in_a_graph(torch, qs):
    E, k, T = 256, 8, 70
    r = rule_for("group2bias", E, k)
    rule = to_rule(r, torch, qs)
    x = torch.randn(T, E, device="cuda")
    want = qs.moe_select(x, k, rule)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qs.moe_select(x, k, rule, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    idx, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.moe_select(x, k, rule, topk_idx=idx, topk_w=w)
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(T, E))
        g.replay()
        torch.cuda.synchronize()
        want = qs.moe_select(x, k, rule)
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])


# ----------------------------------------------------------------------- the layer
LAYERS = {
    "tiny": dict(hidden=256, inter=128, n_experts=16, top_k=2),
    "ragged": dict(hidden=192, inter=320, n_experts=20, top_k=3, gated=True),
    "many": dict(hidden=576, inter=64, n_experts=240, top_k=16, bias=True, shared=False),
}


_cache = {}


def layer(lname, name=None):
    """A layer under a rule, or (no rule) with its own routing: made once."""
    if (lname, name) not in _cache:
        kw = LAYERS[lname]
        _cache[lname, name] = (ref.Layer(seed=3, **kw) if name is None else
                               rule_ref.RuledLayer(dict(rule_for(name, kw["n_experts"], kw["top_k"])), seed=3, **kw))
    return _cache[lname, name]


@pytest.mark.parametrize("name", ["group2bias", "all"])
@pytest.mark.parametrize("lname", sorted(LAYERS))
@pytest.mark.parametrize("T", [1, 3, 9, 40, 150])
def test_mx4_layer_under_a_rule(torch, qs, name, lname, T):
    """Every path of the MX4 layer: its own check, with the rule's selection and weights (a
    weight's relative error is at most twice its logits' error, as in the softmax over the
    selection: a sigmoid's and a softmax's logarithm have slopes of at most 1 and 2)."""
    kw = LAYERS[lname]
    r = rule_for(name, kw["n_experts"], kw["top_k"])
    L = layer(lname, name)
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=T)
    x = to_dev(xb, torch)
    ws = qs.new_workspace(desc, T)
    rule = to_rule(r, torch, qs)
    for yt in (torch.float32, torch.bfloat16):
        y, idx, w = run(torch, qs, desc, x, y_dtype=yt, workspace=ws, rule=rule)
        check(L, xb, y, idx, w, (name, lname, T, yt))
    ri, rw = qs.moe_route(desc, x, workspace=ws, rule=rule)
    assert torch.equal(ri, idx) and torch.equal(rw, w)
    assert int(qs.moe_workspace_status(ws)) == 0
    # and the layer's own routing afterwards, in the same workspace
    y0, i0, w0 = run(torch, qs, desc, x, workspace=ws)
    check(layer(lname), xb, y0, i0, w0, "own routing")


@pytest.mark.parametrize("name", ["group2bias", "all"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 40])
def test_affine_layer_under_a_rule(torch, qs, orc, name, bits, T):
    """T = 1, 2 to 4, 5 to 8 and the grouped path, against the oracle on the rule's routing."""
    Ly = syn.make_layer(**{**syn.TINY, "bits": bits, "n_experts": 24, "top_k": 3, "shared_gate": T % 2 == 0})
    r = rule_for(name, 24, 3)
    rule = to_rule(r, torch, qs)
    desc = qs.LayerDesc.from_host(Ly, device="cuda:0")
    ol = orc.OracleLayer(Ly)
    xb = syn.make_x(T, Ly.hidden, seed=T)
    x = to_dev(xb, torch)
    ws = qs.new_workspace(desc, T)
    logits = orc.router_logits(ol, xb)
    wi, _, gap = expect(logits, 3, r)
    for yt in (torch.float32, torch.bfloat16):
        y, idx, w = run(torch, qs, desc, x, y_dtype=yt, workspace=ws, rule=rule)
        gi = idx.cpu().numpy()
        clear = gap >= TAU
        assert np.array_equal(gi[clear], wi[clear])
        ww = rule_ref.weights_of(logits, gi, **r)
        assert np.abs(w.cpu().numpy() - ww).max() <= 1e-6 * max(1.0, abs(r.get("scale", 1.0)))
        want = orc.layer_forward_with_routing(ol, xb, gi, ww)
        check_output(y_to_np(y, torch), want, yt == torch.bfloat16, (name, bits, T))
    ri, rw = qs.moe_route(desc, x, workspace=ws, rule=rule)
    assert torch.equal(ri, idx) and torch.equal(rw, w)
    assert int(qs.moe_workspace_status(ws)) == 0


def test_chunked_prompt_under_a_rule(torch, qs):
    kw = LAYERS["tiny"]
    r = rule_for("group2bias", kw["n_experts"], kw["top_k"])
    L = rule_ref.RuledLayer(dict(r), seed=3, **kw)
    desc, rule = upload(L, torch, qs), to_rule(r, torch, qs)
    x = to_dev(syn.make_x(700, L.hidden, seed=1), torch)
    whole, wi, ww = run(torch, qs, desc, x, rule=rule)
    part, pi, pw = run(torch, qs, desc, x, rule=rule, workspace=qs.new_workspace(desc, 700, chunk=200))
    assert torch.equal(whole, part) and torch.equal(wi, pi) and torch.equal(ww, pw)


@pytest.mark.parametrize("T", [1, 6, 150])
def test_layer_under_a_rule_in_a_graph(torch, qs, T):
    kw = LAYERS["ragged"]
    r = rule_for("group2bias", kw["n_experts"], kw["top_k"])
    desc, rule = upload(rule_ref.RuledLayer(dict(r), seed=3, **kw), torch, qs), to_rule(r, torch, qs)
    x = to_dev(syn.make_x(T, 192, seed=1), torch)
    ws, own = qs.new_workspace(desc, T), qs.new_workspace(desc, T)
    y = torch.empty(T, 192, device="cuda")
    qs.moe_layer_forward(desc, x, y=y, workspace=ws, rule=rule)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.moe_layer_forward(desc, x, y=y, workspace=ws, rule=rule)
    for seed in range(3):
        x.copy_(to_dev(syn.make_x(T, 192, seed=seed), torch))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, qs.moe_layer_forward(desc, x, workspace=own, rule=rule))
