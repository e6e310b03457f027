"""The MoE layer with MX4 experts against the plain 64-bit evaluation (mx4_ref.Layer),
through the same entry points as the affine layers."""
import numpy as np
import pytest

import mx4_ref as ref
import qsmoe_synth as syn
from gpu_util import TAU, to_dev

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


def upload(L, torch, qs):
    def pack(m, rows, cols):
        return qs.mx4_pack_rows16(to_dev(ref.pack_rows(m[0]), torch), to_dev(m[1], torch), rows, cols)

    H, I, E = L.hidden, L.inter, L.n_experts
    sh = None if L.shared is None else (pack(L.shared[0], 2 * I, H), pack(L.shared[1], H, I))
    return qs.LayerDesc.from_mx4(H, I, E, L.top_k, to_dev(L.router_bits, torch), pack(L.gate_up, E * 2 * I, H),
                                 pack(L.down, E * H, I), shared=sh,
                                 router_bias=None if L.bias is None else to_dev(L.bias, torch),
                                 shared_gate_w=None if L.gate_bits is None else to_dev(L.gate_bits, torch))


def run(torch, qs, desc, x, **kw):
    T = x.shape[0]
    idx = torch.full((T, desc.top_k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, desc.top_k), -1.0, device="cuda")
    y = qs.moe_layer_forward(desc, x, topk_idx=idx, topk_w=w, **kw)
    torch.cuda.synchronize()
    return y, idx, w


def check(L, xb, y, idx, w, what):
    x = ref.bf16_values(xb)
    want_idx, gap = L.route(x)
    gi, gw = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    clear = gap >= TAU
    assert (np.diff(gi, axis=1) > 0).all(), what
    assert np.array_equal(gi[clear], want_idx[clear]), what
    # the weights: off by the logits' error (twice) and a few fp32 roundings
    dl = ref.product_bound(x, ref.bf16_values(L.router_bits)).max(axis=1, keepdims=True)
    assert (np.abs(gw - L.weights(x, gi)) <= 2 * dl + 2.0 ** -20).all(), what
    # (near ties: the GPU's own selection)
    want, bound = L.forward(x, gi, prompt=len(x) > 128)
    bf16 = str(y.dtype).endswith("bfloat16")
    got = y.float().cpu().numpy().astype(np.float64)
    err = np.abs(got - want)
    lim = bound + (2.0 ** -8 * (np.abs(want) + bound) if bf16 else 0.0)
    assert (err <= lim).all(), (what, float((err / lim).max()))


LAYERS = {
    "tiny": dict(hidden=256, inter=128, n_experts=16, top_k=2),
    "ragged": dict(hidden=192, inter=320, n_experts=20, top_k=3, gated=True),
    "narrow": dict(hidden=64, inter=64, n_experts=5, top_k=5, shared=False),
    "one": dict(hidden=128, inter=64, n_experts=1, top_k=1),
    "many": dict(hidden=576, inter=64, n_experts=256, top_k=16, bias=True, shared=False),
    "skew": dict(hidden=1088, inter=192, n_experts=100, top_k=8, bias=True, gated=True),
    "wide": dict(hidden=4160, inter=576, n_experts=6, top_k=2),
}
_cache = {}


def layer(name):
    if name not in _cache:
        _cache[name] = ref.Layer(seed=len(name), **LAYERS[name])
    return _cache[name]


@pytest.mark.parametrize("name", sorted(LAYERS))
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 17, 33, 64, 65, 127, 129, 150, 700])
def test_layer(torch, qs, name, T):
    L = layer(name)
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=T)
    x = to_dev(xb, torch)
    ws = qs.new_workspace(desc, T)
    for yt in (torch.float32, torch.bfloat16):
        y, idx, w = run(torch, qs, desc, x, y_dtype=yt, workspace=ws)
        check(L, xb, y, idx, w, (name, T, yt))
    # the routing alone, and the entry point that allocates nothing: the same bits
    ri, rw = qs.moe_route(desc, x, workspace=ws)
    assert torch.equal(ri, idx) and torch.equal(rw, w)
    ys = qs.moe_layer_forward_static(desc, x, y_dtype=torch.bfloat16)
    assert torch.equal(ys, y)
    # completion counters are back at zero, and no wait gave up
    assert (ws[(2 << 20) - 4096:2 << 20] == 0).all()
    assert int(qs.moe_workspace_status(ws)) == 0


@pytest.mark.parametrize("T", [1, 5, 20])
@pytest.mark.parametrize("sigma", [1e-12, 300.0])
def test_activation_range(torch, qs, T, sigma):
    L = layer("tiny")
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=T, std=sigma)
    y, idx, w = run(torch, qs, desc, to_dev(xb, torch))
    gi = idx.cpu().numpy()
    x = ref.bf16_values(xb)
    want_idx, gap = L.route(x)
    clear = gap >= TAU * max(1.0, sigma)
    assert np.array_equal(gi[clear], want_idx[clear])
    want, bound = L.forward(x, gi)
    # h and y of products of two activations: what leaves fp32's normal range may be flushed
    assert (np.abs(y.cpu().numpy() - want) <= bound + 2.0 ** -126 * L.inter).all()


@pytest.mark.parametrize("T", [1, 9, 64])
def test_same_tokens_and_all_on_one_expert(torch, qs, T):
    """Every token the same (one set of experts, every operand row live), twice the same bits."""
    L = layer("tiny")
    desc = upload(L, torch, qs)
    xb = np.repeat(syn.make_x(1, L.hidden, seed=77), T, axis=0)
    y, idx, w = run(torch, qs, desc, to_dev(xb, torch))
    check(L, xb, y, idx, w, T)
    assert (y == y[0]).all()
    y2, _, _ = run(torch, qs, desc, to_dev(xb, torch))
    assert torch.equal(y, y2)


@pytest.mark.parametrize("name", ["one", "many", "narrow"])
@pytest.mark.parametrize("T", [65, 96, 128])
@pytest.mark.parametrize("same", [False, True])
def test_largest_few_token_passes(torch, qs, name, T, same):
    """More than 64 tokens in one pass: every token on one expert (eight list entries), 16 experts a
    token (the longest list), the same token in every row."""
    L = layer(name)
    desc = upload(L, torch, qs)
    xb = np.repeat(syn.make_x(1, L.hidden, seed=78), T, axis=0) if same else syn.make_x(T, L.hidden, seed=T)
    ws = qs.new_workspace(desc, T)
    for _ in range(2):                                   # (the counters are back at zero)
        y, idx, w = run(torch, qs, desc, to_dev(xb, torch), workspace=ws)
        check(L, xb, y, idx, w, (name, T, same))


def test_exact_ties_go_to_the_lower_expert(torch, qs):
    L = ref.Layer(hidden=128, inter=64, n_experts=12, top_k=4, seed=3)
    L.router_bits[[1, 5, 9]] = L.router_bits[1]
    L.router_bits[[2, 3]] = L.router_bits[2]
    desc = upload(L, torch, qs)
    xb = syn.make_x(40, 128, seed=1)
    idx, _ = qs.moe_route(desc, to_dev(xb, torch))
    l = L.logits(ref.bf16_values(xb))
    assert np.array_equal(idx.cpu().numpy(), np.sort(np.argsort(-l, axis=1, kind="stable")[:, :4], axis=1))


def test_workspace_shared_with_affine_layers_and_graph_replays(torch, qs):
    """One workspace for an MX4 layer and an affine one, calls of every path in turn, eager
    and in a captured graph replayed with eager calls in between: always the same bits."""
    L = layer("skew")
    mx = upload(L, torch, qs)
    A = syn.make_layer(**syn.TINY)
    af = qs.LayerDesc.from_host(A)
    n = max(qs.moe_workspace_size(mx, 170), qs.moe_workspace_size(af, 40))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    xm = {T: to_dev(syn.make_x(T, L.hidden, seed=T), torch) for T in (1, 3, 6, 30, 100, 170)}
    xa = {T: to_dev(syn.make_x(T, A.hidden, seed=T), torch) for T in (1, 3, 40)}
    rm = {T: qs.moe_layer_forward(mx, x, workspace=qs.new_workspace(mx, T)) for T, x in xm.items()}
    ra = {T: qs.moe_layer_forward(af, x, workspace=qs.new_workspace(af, T)) for T, x in xa.items()}
    outs = {("m", T): torch.empty_like(r) for T, r in rm.items()} | {("a", T): torch.empty_like(r) for T, r in ra.items()}

    def every():
        for T in (1, 30, 3, 6, 100, 170):
            qs.moe_layer_forward(mx, xm[T], y=outs["m", T], workspace=ws)
            Ta = {1: 3, 30: 1, 3: 3, 6: 40, 100: 1, 170: 1}[T]
            qs.moe_layer_forward(af, xa[Ta], y=outs["a", Ta], workspace=ws)

    def same():
        torch.cuda.synchronize()
        for T in rm:
            assert torch.equal(outs["m", T], rm[T]), T
        for T in ra:
            assert torch.equal(outs["a", T], ra[T]), T

    every()
    same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        every()
    for _ in range(4):
        for o in outs.values():
            o.fill_(7.0)
        g.replay()
        same()
        every()
        same()


def test_prompt_in_chunks(torch, qs):
    """A prompt in chunks (a smaller workspace) gives the bits of one chunk, and a token's result
    does not depend on the others."""
    L = layer("skew")
    desc = upload(L, torch, qs)
    T = 333
    xb = syn.make_x(T, L.hidden, seed=12)
    x = to_dev(xb, torch)
    y, idx, w = run(torch, qs, desc, x)
    for chunk in (2, 150, 200):
        ws = torch.zeros(qs.moe_workspace_size(desc, T, chunk), dtype=torch.uint8, device="cuda")
        y2, i2, w2 = run(torch, qs, desc, x, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(idx, i2) and torch.equal(w, w2), chunk
    other = to_dev(syn.make_x(T, L.hidden, seed=13), torch)
    other[200] = x[200]
    y4, _, _ = run(torch, qs, desc, other)
    assert torch.equal(y4[200], y[200])


@pytest.mark.parametrize("T", [1, 30, 129, 400, 1500])
@pytest.mark.parametrize("shape", [(512, 512), (1024, 1536), (1536, 64)])
def test_whole_quads_of_columns(torch, qs, shape, T):
    """Dimensions of whole quads (512 columns): the prompt kernels unroll those."""
    L = ref.Layer(*shape, n_experts=12, top_k=3, seed=T, gated=True)
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=T + 1)
    y, idx, w = run(torch, qs, desc, to_dev(xb, torch))
    check(L, xb, y, idx, w, (shape, T))


def test_prompt_past_32_bit_offsets(torch, qs):
    """A workspace for all of a prompt whose x is larger than 2^31 bytes gives the bits of small chunks."""
    L = ref.Layer(8192, 64, n_experts=4, top_k=1, shared=False, seed=3)
    desc = upload(L, torch, qs)
    T = 140000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, L.hidden, generator=g, device="cuda", dtype=torch.bfloat16)
    idx = torch.empty((T, 1), dtype=torch.int32, device="cuda")
    y = {}
    for chunk in (4096, T):
        ws = torch.zeros(qs.moe_workspace_size(desc, T, chunk), dtype=torch.uint8, device="cuda")
        y[chunk] = qs.moe_layer_forward(desc, x, topk_idx=idx, workspace=ws, y_dtype=torch.bfloat16)
    assert torch.equal(y[4096], y[T])
    rows = [0, 131071, 131072, T - 1]                    # (2^31 bytes into x is row 131072)
    few = qs.moe_layer_forward(desc, x[rows].contiguous().repeat(40, 1), y_dtype=torch.bfloat16)
    assert torch.equal(few[:4], y[T][rows])


def test_prompt_range(torch, qs):
    """Activations whose expert outputs leave fp16's range: the slot rows carry scales."""
    L = layer("ragged")
    desc = upload(L, torch, qs)
    for sigma in (1e-6, 2000.0):
        xb = syn.make_x(140, L.hidden, seed=6, std=sigma)
        y, idx, w = run(torch, qs, desc, to_dev(xb, torch))
        gi = idx.cpu().numpy()
        want, bound = L.forward(ref.bf16_values(xb), gi, prompt=True)
        assert (np.abs(y.cpu().numpy() - want) <= bound + 2.0 ** -126 * L.inter).all()


def test_token_state(torch, qs):
    """The one-token launch waits for tagged logits: many calls on one workspace alternating inputs,
    across the wrap of the tag, give the first results; a bound of a poll or two makes the waits
    give up, every kernel still ends, the error word says so, and the next call is right again."""
    L = ref.Layer(hidden=2048, inter=128, n_experts=256, top_k=8, seed=21, gated=True)
    desc = upload(L, torch, qs)
    xbs = [syn.make_x(1, L.hidden, seed=s) for s in (1, 2, 3)]
    xs = [to_dev(b, torch) for b in xbs]
    want = [run(torch, qs, desc, x) for x in xs]
    for xb, (y, idx, w) in zip(xbs, want):
        check(L, xb, y, idx, w, "token")
    ws = qs.new_workspace(desc, 1)
    w32 = ws[:1024].view(torch.int32)
    w32[64] = -4                                                 # the generation: wraps after four calls
    for i in range(30):
        y, idx, w = run(torch, qs, desc, xs[i % 3], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip((y, idx, w), want[i % 3])), i
    assert int(qs.moe_workspace_status(ws)) == 0
    w32[32] = 1                                                  # at most one more poll
    for i in range(3):
        qs.moe_layer_forward(desc, xs[i], workspace=ws)
    torch.cuda.synchronize()
    st = int(qs.moe_workspace_status(ws, clear=True))
    assert st in (0, qs.MOE_WS_ERR_DECODE_WAIT)
    w32[32] = 0
    y, idx, w = run(torch, qs, desc, xs[1], workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip((y, idx, w), want[1]))
    assert int(qs.moe_workspace_status(ws)) == 0


def test_few_token_state(torch, qs):
    """The same for two to four tokens, which share the copies of the logit words, and calls of other
    sizes in between: one workspace, across the wrap of the tag."""
    L = ref.Layer(hidden=2048, inter=128, n_experts=256, top_k=8, seed=22, gated=True)
    desc = upload(L, torch, qs)
    Ts = (1, 2, 4, 3, 5)
    xbs = [syn.make_x(T, L.hidden, seed=50 + T) for T in Ts]
    xs = [to_dev(b, torch) for b in xbs]
    want = [run(torch, qs, desc, x) for x in xs]
    for T, xb, (y, idx, w) in zip(Ts, xbs, want):
        check(L, xb, y, idx, w, T)
    ws = qs.new_workspace(desc, max(Ts))
    w32 = ws[:1024].view(torch.int32)
    w32[64] = -7                                                 # the generation: wraps in the second turn
    for i in range(40):
        y, idx, w = run(torch, qs, desc, xs[i % 5], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip((y, idx, w), want[i % 5])), i
    assert int(qs.moe_workspace_status(ws)) == 0
    w32[32] = 1                                                  # at most one more poll
    for i in (1, 2, 3):
        qs.moe_layer_forward(desc, xs[i], workspace=ws)
    torch.cuda.synchronize()
    assert int(qs.moe_workspace_status(ws, clear=True)) in (0, qs.MOE_WS_ERR_DECODE_WAIT)
    w32[32] = 0
    for i in (3, 2, 1):
        y, idx, w = run(torch, qs, desc, xs[i], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip((y, idx, w), want[i]))
    assert int(qs.moe_workspace_status(ws)) == 0


@pytest.mark.parametrize("name", sorted(LAYERS))
@pytest.mark.parametrize("T", [2, 3, 4])
def test_few_tokens_share_experts(torch, qs, name, T):
    """Two to four tokens, the first and last alike: experts of one and of several tokens."""
    L = layer(name)
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=60 + T)
    xb[T - 1] = xb[0]
    ws = qs.new_workspace(desc, T)
    for _ in range(2):
        y, idx, w = run(torch, qs, desc, to_dev(xb, torch), workspace=ws)
        check(L, xb, y, idx, w, (name, T))
        assert torch.equal(y[0], y[T - 1])
    i2, w2 = qs.moe_route(desc, to_dev(xb, torch), workspace=ws)
    assert torch.equal(i2, idx) and torch.equal(w2, w)


def test_side_stream_and_empty(torch, qs):
    L = layer("tiny")
    desc = upload(L, torch, qs)
    x = to_dev(syn.make_x(12, L.hidden, seed=4), torch)
    y = qs.moe_layer_forward(desc, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = qs.moe_layer_forward(desc, x, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    assert qs.moe_layer_forward(desc, x[:0]).shape == (0, L.hidden)


def test_guards_around_the_outputs(torch, qs):
    L = layer("ragged")
    desc = upload(L, torch, qs)
    for T in (3, 70, 200):
        x = to_dev(syn.make_x(T, L.hidden, seed=5), torch)
        y = torch.full((T + 2, L.hidden), 7.0, device="cuda")
        idx = torch.full((T + 2, 3), -9, dtype=torch.int32, device="cuda")
        w = torch.full((T + 2, 3), -9.0, device="cuda")
        qs.moe_layer_forward(desc, x, y=y[1:T + 1], topk_idx=idx[1:T + 1], topk_w=w[1:T + 1])
        torch.cuda.synchronize()
        for t, v in ((y, 7.0), (idx, -9), (w, -9.0)):
            assert (t[0] == v).all() and (t[T + 1] == v).all() and not (t[1:T + 1] == v).any()


@pytest.mark.parametrize("T", [1, 2, 21, 64, 100, 150])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_tokens_stay_alone(torch, qs, T, value):
    """A NaN or an infinity in one token's x: the call returns, that token's row of y holds no finite
    value where its experts see it, every other token's row is right."""
    L = layer("skew")
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=31)
    x = to_dev(xb, torch).view(torch.bfloat16).clone()
    bad = T // 2
    x[bad, 5] = value
    ws = qs.new_workspace(desc, T)
    y, idx, w = run(torch, qs, desc, x, workspace=ws)
    assert not torch.isfinite(y[bad]).any()
    gi = idx.cpu().numpy()
    assert (np.diff(gi, axis=1) > 0).all() and gi.min() >= 0 and gi.max() < L.n_experts
    rest = [t for t in range(T) if t != bad]
    if rest:
        want, bound = L.forward(ref.bf16_values(xb)[rest], gi[rest], prompt=T > 128)
        assert (np.abs(y.cpu().numpy()[rest] - want) <= bound).all()
    # and nothing of it stays in the workspace
    y2, i2, w2 = run(torch, qs, desc, to_dev(xb, torch), workspace=ws)
    check(L, xb, y2, i2, w2, T)


@pytest.mark.parametrize("Ts", [(1, 7), (2, 4), (3, 128), (1, 200)])
def test_two_streams_two_workspaces(torch, qs, Ts):
    """Calls that overlap in time, each on its own stream and workspace, give what they give alone."""
    L = layer("skew")
    desc = upload(L, torch, qs)
    xs = [to_dev(syn.make_x(T, L.hidden, seed=40 + T), torch) for T in Ts]
    ws = [qs.new_workspace(desc, x.shape[0]) for x in xs]
    want = [qs.moe_layer_forward(desc, x, workspace=w).clone() for x, w in zip(xs, ws)]
    ys = [torch.empty((20,) + tuple(y.shape), device="cuda") for y in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for r in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                qs.moe_layer_forward(desc, xs[i], y=ys[i][r], workspace=ws[i])
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert (y == w).all()
    assert all(int(qs.moe_workspace_status(w)) == 0 for w in ws)


def test_products_and_layer_run_together(torch, qs):
    """A block as it is used: a projection with MX4 weights makes the layer's input, the layer
    runs, its output is quantized and goes through another projection."""
    L = layer("tiny")
    desc = upload(L, torch, qs)
    rng = np.random.default_rng(9)
    T, H, N = 11, L.hidden, 160
    ws = []
    for shape in ((H, H), (N, H)):
        c, s = ref.quantize(rng.standard_normal(shape) / 16)
        ws.append((ref.values(c, s), qs.mx4_pack_rows16(to_dev(ref.pack_rows(c), torch), to_dev(s, torch), *shape)))
    xb = syn.make_x(T, H, seed=8)
    a = qs.mx4_gemm(*ws[0][1], H, H, to_dev(xb, torch), y_dtype=torch.bfloat16)
    y, idx, w = run(torch, qs, desc, a, y_dtype=torch.bfloat16)
    out = qs.mx4_gemm_mx4x(*ws[1][1], N, H, *qs.mx4_quantize(y), T)
    torch.cuda.synchronize()
    av = a.float().cpu().numpy().astype(np.float64)
    want, bound = ref.bf16_values(xb) @ ws[0][0].T, ref.product_bound(ref.bf16_values(xb), ws[0][0])
    assert (np.abs(av - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()
    check(L, a.view(torch.int16).cpu().numpy().view(np.uint16), y, idx, w, "layer of the projection")
    yq = ref.values(*ref.quantize(y.float().cpu().numpy().astype(np.float64)))
    assert (np.abs(out.cpu().numpy() - yq @ ws[1][0].T) <= ref.product_bound(yq, ws[1][0])).all()


def _list_of(ws, L, T):
    """(nact, act, pos) of the last call of T <= 128 tokens, as views into its workspace: behind the
    2 MiB state, 256-byte aligned, logits, selections, weights, list, its length and rows."""
    up = lambda n: -(-n // 256) * 256
    E, K = L.n_experts, L.top_k
    act = (2 << 20) + up(T * (E + 1) * 4) + 2 * up(T * K * 4)
    nact = act + up(384 * 4)
    pos = nact + up(4)
    return ws[nact:nact + 4], ws[act:act + 384 * 4], ws[pos:pos + E * 256]


@pytest.mark.parametrize("T", [1, 2, 3, 4])
def test_give_up_leaves_a_whole_list(torch, qs, T):
    """Waits that give up over logits that differ from copy to copy: workgroups select differently, and
    the error word says so, but every entry of the list that the next launch reads was written by this
    call and lies in range, and the next call is right again."""
    L = _cache.setdefault("slow route", ref.Layer(hidden=8192, inter=64, n_experts=40, top_k=8, seed=23))
    desc = upload(L, torch, qs)
    xb = syn.make_x(T, L.hidden, seed=80 + T)
    x = to_dev(xb, torch)
    ws = qs.new_workspace(desc, T)
    want = run(torch, qs, desc, x, workspace=ws)
    check(L, xb, *want, T)
    w32 = ws[:1 << 20].view(torch.int32)
    empty = status = 0
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ws[2 << 20:].fill_(0xFF)                             # what lies there is no list
        logits = w32[1216:1216 + 32 * 576]                   # the copies of the tagged logit words
        logits.copy_(torch.randn(logits.shape, generator=g, device="cuda").view(torch.int32))
        logits[1::2] = -1                                    # (of another call's tag)
        torch.empty(1 << 29, dtype=torch.uint8, device="cuda").fill_(seed)   # (weights out of the caches)
        w32[32] = 1                                          # the bound on a wait's polls
        qs.moe_layer_forward(desc, x, workspace=ws)
        torch.cuda.synchronize()
        w32[32] = 0
        status |= int(qs.moe_workspace_status(ws, clear=True))
        nact, act, pos = (v.cpu().numpy().view(t) for v, t in zip(_list_of(ws, L, T), ("i4", "i4", "i2")))
        n = int(nact[0])
        assert L.top_k <= n <= T * L.top_k
        for a in act[:n].tolist():
            e, slot, tile, count = a & 255, a >> 8 & 255, a >> 16 & 15, a >> 20
            assert e < L.n_experts and slot < L.n_experts and tile == 0 and 0 <= count <= T, hex(a)
            rows = pos[slot * 128:slot * 128 + count]
            assert ((rows >= 0) & (rows < T * L.top_k)).all()
        empty += int((act[:n] == 0).any())
        got = run(torch, qs, desc, x, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert int(qs.moe_workspace_status(ws)) == 0
    assert status == qs.MOE_WS_ERR_DECODE_WAIT
    print(f"[state] T = {T}: {empty} of 4 lists with empty entries", flush=True)
