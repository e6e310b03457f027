"""moe_block_norm on the GPU against the plain 64-bit evaluation (norm_ref)."""
import numpy as np
import pytest

import norm_ref as ref

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


def dtypes(torch):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def make(torch, qs, T, H, y="bf16", r="bf16", x="bf16", kind="rms", post=True, pre=True, gate=None, act="none", scale=1.0,
         offset=0.0, bias=False, seed=0, spread=1.0, w="bf16"):
    """Tensors of a case, the call's arguments and the reference's."""
    g = torch.Generator().manual_seed(seed)
    D = dtypes(torch)
    rnd = lambda *s: torch.randn(*s, generator=g)
    rows = torch.exp(spread * rnd(T, 1))
    a = dict(y=None if y is None else (rnd(T, H) * rows).to(D[y]).cuda(),
             residual=None if r is None else (rnd(T, H) * rows.flip(0) + 0.5).to(D[r]).cuda(),
             gate=None if gate is None else (3 * rnd(T, H if gate == "element" else 1)).to(D[y]).cuda(),
             gate_act=act, scale=scale)
    e = {}
    for which, on in (("post", post and y is not None), ("pre", pre)):
        if not on:
            a[which] = e[which] = None
            continue
        wt, bt = (1 - offset + 0.3 * rnd(H)).to(D[w]).cuda(), rnd(H).to(D[w]).cuda() if bias else None
        a[which] = qs.Norm(kind, weight=wt, bias=bt, eps=1e-5, offset=offset)
        e[which] = dict(kind=kind, eps=float(np.float32(1e-5)), offset=offset, weight=np64(wt), bias=np64(bt))
    return a, e, dict(r=r or y, x=x)


def check(torch, a, e, types, out, what):
    (t, bt), (v, bv) = ref.block(np64(a["y"]), np64(a["residual"]), e["post"], np64(a["gate"]), a["gate_act"], a["scale"],
                                 e["pre"])
    for got, want, b, name in ((out[0], t, bt, types["r"]), (out[1], v, bv, types["x"])):
        if got is None:
            continue
        assert got.dtype == dtypes(torch)[name], what
        err, lim = np.abs(np64(got) - want), ref.rounded(want, b, name)
        assert (err <= lim).all(), (what, name, float((err / lim).max()))


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 64), (67, 128), (9, 129), (33, 512), (3, 513), (5, 1024), (6, 1023), (4, 1032),
          (2, 4096), (3, 4095), (2, 16384), (2, 16381), (1, 2048), (600, 2048), (5, 2047),
          (520, 2047), (2, 2056), (4, 8192), (530, 8192), (3, 8191), (2, 8200), (2, 8193), (3, 15), (4, 1001), (3, 16383), (2, 16378), (5, 2041),
          (5, 2042), (9, 505), (9, 506), (17, 121), (17, 122), (40, 9), (30, 5)]


@pytest.mark.parametrize("T,H", SHAPES)
def test_shapes(torch, qs, T, H):
    """Every row length class, from both sides, few rows and many."""
    for kind in ("rms", "layer"):
        a, e, ty = make(torch, qs, T, H, kind=kind, bias=kind == "layer", gate="element", act="sigmoid", scale=0.3, seed=T + H)
        out = qs.moe_block_norm(**a)
        check(torch, a, e, ty, out, (T, H, kind))


@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("r", ["bf16", "f16", "f32", None])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_types(torch, qs, y, r, x):
    for H in (264, 263):
        for w in ("bf16", "f16", "f32"):
            a, e, ty = make(torch, qs, 5, H, y=y, r=r, x=x, w=w, bias=True, spread=0.5)
            out = qs.moe_block_norm(**a, x_dtype=dtypes(torch)[x])
            check(torch, a, e, ty, out, (y, r, x, w, H))


@pytest.mark.parametrize("gate,act", [(None, "none"), ("token", "none"), ("token", "silu"), ("element", "sigmoid"),
                                      ("element", "silu"), ("token", "sigmoid"), ("element", "none")])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_parts(torch, qs, gate, act, post, pre):
    for H in (136, 1001):
        for r in ("f32", None):
            a, e, ty = make(torch, qs, 6, H, r=r, gate=gate, act=act, post=post, pre=pre, scale=-1.5, offset=1.0)
            out = qs.moe_block_norm(**a)
            assert (out[1] is None) == (not pre)
            check(torch, a, e, ty, out, (gate, act, post, pre, H, r))


def test_norm_before_a_block_alone(torch, qs):
    for kind in ("rms", "layer"):
        a, e, ty = make(torch, qs, 7, 640, y=None, r="f16", x="bf16", kind=kind)
        out = qs.moe_block_norm(**a, x_dtype=torch.bfloat16)
        assert out[0] is None
        check(torch, a, e, ty, out, kind)
    # no gain at all
    v = torch.randn(4, 96, device="cuda")
    _, x = qs.moe_block_norm(residual=v, pre=qs.Norm(eps=0.0))
    want, b = ref.norm(np64(v), 0 * np64(v), "rms", 0.0, 0.0, None, None)
    assert (np.abs(np64(x) - want) <= ref.rounded(want, b, "f32")).all()


def test_in_place_and_columns_of_a_wider_matrix(torch, qs):
    T, H = 70, 200
    a, e, ty = make(torch, qs, T, H, gate="element", act="silu")
    want = qs.moe_block_norm(**a)
    # [y | gate | r] as columns of one matrix, r updated in place, x over the gate
    m = torch.cat([a["y"], a["gate"], a["residual"], torch.full((T, 8), 7.0, dtype=torch.bfloat16, device="cuda")], 1)
    b = dict(a, y=m[:, :H], gate=m[:, H:2 * H], residual=m[:, 2 * H:3 * H])
    r, x = qs.moe_block_norm(**b, r_out=b["residual"], x_out=b["gate"])
    assert r.data_ptr() == b["residual"].data_ptr()
    assert torch.equal(m[:, 2 * H:3 * H], want[0]) and torch.equal(m[:, H:2 * H], want[1])
    assert torch.equal(m[:, :H], a["y"]) and (m[:, 3 * H:] == 7).all()
    # an odd column offset: values no longer 16-byte aligned
    m = torch.zeros(T, 3 * H + 3, dtype=torch.bfloat16, device="cuda")
    m[:, 1:H + 1], m[:, H + 1:2 * H + 1], m[:, 2 * H + 1:3 * H + 1] = a["y"], a["gate"], a["residual"]
    b = dict(a, y=m[:, 1:H + 1], gate=m[:, H + 1:2 * H + 1], residual=m[:, 2 * H + 1:3 * H + 1])
    out = qs.moe_block_norm(**b)
    check(torch, a, e, ty, out, "odd offset")
    with pytest.raises(qs.QsmoeError):                       # one column off itself
        qs.moe_block_norm(**b, r_out=m[:, 2 * H:3 * H])


def test_rows_behind_the_last_stay(torch, qs):
    for H in (256, 255, 4096):
        a, e, ty = make(torch, qs, 21, H)
        r = torch.full((25, H), 9.0, dtype=torch.bfloat16, device="cuda")
        x = torch.full((25, H), 9.0, dtype=torch.bfloat16, device="cuda")
        qs.moe_block_norm(**a, r_out=r[:21], x_out=x[:21])
        check(torch, a, e, ty, (r[:21], x[:21]), H)
        assert (r[21:] == 9).all() and (x[21:] == 9).all()
        r0, x0 = qs.moe_block_norm(a["y"][:0], residual=a["residual"][:0], pre=a["pre"])
        assert r0.shape == (0, H) and x0.shape == (0, H)


def test_not_finite_values_stay_in_their_row(torch, qs):
    for H in (200, 77):
        a, e, ty = make(torch, qs, 6, H, gate="element", act="sigmoid", kind="layer")
        clean = qs.moe_block_norm(**a)
        a["y"][1, 3], a["residual"][2, 5], a["gate"][3, 0] = float("nan"), float("inf"), float("nan")
        r, x = qs.moe_block_norm(**a)
        for i in (0, 4, 5):
            assert torch.equal(r[i], clean[0][i]) and torch.equal(x[i], clean[1][i])
        assert r[1].isnan().all() and x[1].isnan().all()     # (the post norm's mean)
        assert r[2, 5].isinf() and torch.equal(r[2, :5], clean[0][2, :5]) and not x[2].isfinite().any()
        assert r[3, 0].isnan() and torch.equal(r[3, 1:], clean[0][3, 1:]) and x[3].isnan().all()


def test_large_small_and_constant_rows(torch, qs):
    T, H = 6, 512
    a, e, ty = make(torch, qs, T, H, y="f32", r="f32", x="f32", kind="rms")
    for t in (a["y"], a["residual"]):
        t[0] *= 1e15
        t[1] *= 1e-15
        t[2] = 0.0
        t[3] = 1.0
    check(torch, a, e, ty, qs.moe_block_norm(**a, x_dtype=torch.float32), "rms")
    a, e, ty = make(torch, qs, T, H, y="f32", r="f32", x="f32", kind="layer", post=False)
    a["residual"][0] += 30.0                                 # a mean far from zero
    a["residual"][1], a["y"][1] = 0.0, 0.0
    check(torch, a, e, ty, qs.moe_block_norm(**a, x_dtype=torch.float32), "layer")
    # fp16 results past the type's range are infinities
    v = torch.full((1, 64), 60000.0, device="cuda", dtype=torch.float16)
    r, _ = qs.moe_block_norm(v, residual=v)
    assert r.isinf().all()


def test_offsets_past_32_bits(torch, qs):
    ld = ((1 << 31) // 3 + 8) // 8 * 8                       # (16-byte aligned rows)
    for off in (0, 1):
        H = 64
        buf = torch.empty(4 * ld + H + 1, dtype=torch.bfloat16, device="cuda")
        y = buf.as_strided((5, H), (ld, 1), off)
        a, e, ty = make(torch, qs, 5, H)
        y.copy_(a["y"])
        b = dict(a, y=y)
        check(torch, a, e, ty, qs.moe_block_norm(**b, r_out=y), off)


def test_streams_and_graphs(torch, qs):
    a, e, ty = make(torch, qs, 40, 2048, gate="token", act="sigmoid")
    want = qs.moe_block_norm(**a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qs.moe_block_norm(**a, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    r, x = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.moe_block_norm(**a, r_out=r, x_out=x)
    for seed in range(3):
        n, _, _ = make(torch, qs, 40, 2048, gate="token", act="sigmoid", seed=seed)
        for k in ("y", "residual", "gate"):
            a[k].copy_(n[k])
        g.replay()
        torch.cuda.synchronize()
        want = qs.moe_block_norm(**a)
        assert torch.equal(r, want[0]) and torch.equal(x, want[1])


def gates(torch, dtype):
    """Every finite bf16 value; for the wider types also values between them where a sigmoid's exponential
    leaves fp32's range on either side, and the type's largest."""
    g = (torch.arange(65536, dtype=torch.int32) << 16).view(torch.float32)
    g = g[g.isfinite() & (g.abs() <= torch.finfo(dtype).max)]
    if dtype != torch.bfloat16:
        d = torch.linspace(80.0, 210.0, 8192)
        g = torch.cat([g, d, -d, torch.tensor([-1.0, 1.0]) * torch.finfo(dtype).max])
    return g.to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gates_of_any_size(torch, qs, act, dtype):
    """The whole range of a gate: its activation is finite, and 0 where the exponential is infinite."""
    D = dtypes(torch)[dtype]
    g = gates(torch, D)
    H = 128
    g = torch.cat([g, g[:-len(g) % H]]).reshape(-1, H)
    for gate in (g, g[:, ::9].reshape(-1, 1)):
        y = torch.ones(gate.shape[0], H).to(D)
        y[:, ::3] = -0.75
        a = dict(y=y.cuda(), residual=None, gate=gate.cuda(), gate_act=act, scale=1.0, post=None, pre=None)
        r, _ = qs.moe_block_norm(**a, r_dtype=torch.float32)
        assert r.isfinite().all()
        check(torch, a, dict(post=None, pre=None), dict(r="f32", x="f32"), (r, None), (act, dtype, gate.shape))
        low = (gate.float() < -105.0).cuda().expand(-1, H)
        assert (r[low] == 0).all()
    # a row is normed beside such gates
    g = g[(g.float().abs() <= 1e4)]
    g = torch.cat([g, g[:-len(g) % H]]).reshape(-1, H)
    a = dict(y=torch.ones(g.shape[0], H).to(D).cuda(), residual=torch.randn(g.shape[0], H, device="cuda"), gate=g.cuda(),
             gate_act=act, scale=0.5, post=None, pre=qs.Norm(eps=1e-5))
    e = dict(post=None, pre=dict(kind="rms", eps=float(np.float32(1e-5)), offset=0.0, weight=None, bias=None))
    out = qs.moe_block_norm(**a, x_dtype=torch.float32)
    assert out[0].isfinite().all() and out[1].isfinite().all()
    check(torch, a, e, dict(r="f32", x="f32"), out, (act, dtype, "normed"))


def test_infinite_gates(torch, qs):
    inf = float("inf")
    for H in (8, 9):
        for gate in (torch.full((2, H), inf), torch.full((2, 1), inf)):
            gate[1] = -inf
            y = torch.full((2, H), 3.0, device="cuda")
            r, _ = qs.moe_block_norm(y, gate=gate.cuda(), gate_act="sigmoid")
            assert (r[0] == 3).all() and (r[1] == 0).all()
            r, _ = qs.moe_block_norm(y, gate=gate.cuda(), gate_act="silu")
            assert (r[0] == inf).all() and r[1].isnan().all()            # (-infinity times 0)
