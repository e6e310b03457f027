"""lora_gemm on the GPU against the plain 64-bit evaluation (lora_ref)."""
import numpy as np
import pytest

import lora_ref as ref

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


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def make(torch, T, K, N, R, n, seed=0, order="mixed", ragged=False, scales=True, dtype="bf16", base=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    ids = torch.randint(-1, n + 1, (T,), generator=g, dtype=torch.int32)
    if order == "packed":
        ids = ids.sort()[0]
    elif order == "one":
        ids = torch.full_like(ids, n - 1)
    elif order == "none":
        ids = torch.full_like(ids, -5)
    d = dict(a=(rnd(n, R, K) / K ** 0.5).bfloat16(), b=(rnd(n, N, R) / R ** 0.5).bfloat16(), ids=ids,
             x=rnd(T, K).bfloat16(), scales=rnd(n) + 1.5 if scales else None, ranks=None,
             base=rnd(T, N).to(torch.bfloat16 if dtype == "bf16" else torch.float32) if base else None)
    if ragged:
        d["ranks"] = torch.randint(0, R + 1, (n,), generator=g, dtype=torch.int32)
        d["ranks"][0] = R + 3                                # (counts as R)
        if n > 1:
            d["ranks"][1] = -2                               # (as 0)
        for i in range(n):                                   # past the rank: anything
            r = min(max(int(d["ranks"][i]), 0), R)
            d["a"][i, r:] = float("nan")
            d["b"][i, :, r:] = float("nan")
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def call(torch, qs, d, dtype, **kw):
    ad = qs.LoraAdapters(d["a"], d["b"], scales=d["scales"], ranks=d["ranks"])
    kw.setdefault("base", d["base"])
    return qs.lora_gemm(ad, d["ids"], d["x"], y_dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, **kw)


def check(d, got, dtype, what, rows=None):
    ids, x, base = d["ids"].cpu().numpy(), np64(d["x"]), np64(d["base"])
    got = np64(got)
    if rows is not None:
        ids, x, base, got = ids[rows], x[rows], None if base is None else base[rows], got[rows]
    y, b = ref.forward(np64(d["a"]), np64(d["b"]), ids, x, base, np64(d["scales"]),
                       None if d["ranks"] is None else d["ranks"].cpu().numpy(), dtype == "f32")
    ref.check(got, y, b, dtype == "bf16", what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order,ragged", [("mixed", False), ("mixed", True), ("packed", True), ("one", False), ("none", False)])
@pytest.mark.parametrize("T,K,N,R,n", [(1, 8, 1, 8, 1), (1, 2048, 256, 16, 3), (3, 72, 17, 24, 2), (16, 256, 64, 8, 40),
                                       (17, 264, 300, 64, 5), (48, 512, 1030, 32, 40), (130, 104, 257, 136, 4),
                                       (37, 1000, 65, 256, 6), (300, 64, 70, 40, 3)])
def test_shapes(torch, qs, T, K, N, R, n, order, ragged, dtype):
    d = make(torch, T, K, N, R, n, seed=T + K, order=order, ragged=ragged, dtype=dtype)
    y = call(torch, qs, d, dtype)
    check(d, y, dtype, (T, K, N, R, n, order, ragged))
    if order == "none":
        assert torch.equal(y, d["base"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_base_or_scales(torch, qs, dtype):
    for order in ("mixed", "none"):
        d = make(torch, 21, 128, 90, 16, 3, scales=False, base=False, dtype=dtype, order=order)
        check(d, call(torch, qs, d, dtype), dtype, order)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt(torch, qs, dtype):
    """Many tiles, runs of tokens of one adapter and borders between them."""
    T = 1500
    for order in ("packed", "mixed"):
        d = make(torch, T, 256, 520, 32, 6, order=order, ragged=True, dtype=dtype)
        rows = np.unique(np.r_[0:40, T - 40:T, np.random.default_rng(0).integers(0, T, 60)])
        check(d, call(torch, qs, d, dtype), dtype, order, rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_does_not_depend_on_the_others(torch, qs, dtype):
    d = make(torch, 70, 320, 200, 16, 5, dtype=dtype)
    y = call(torch, qs, d, dtype)
    p = torch.randperm(70, generator=torch.Generator().manual_seed(1)).cuda()
    e = dict(d, ids=d["ids"][p].contiguous(), x=d["x"][p].contiguous(), base=d["base"][p].contiguous())
    assert torch.equal(call(torch, qs, e, dtype), y[p])
    for t in (0, 69):
        e = dict(d, ids=d["ids"][t:t + 1], x=d["x"][t:t + 1], base=d["base"][t:t + 1])
        one = call(torch, qs, e, dtype)
        check(e, one, dtype, "one")
    # a NaN or an infinity in a token's x stays in its row
    e = dict(d, x=d["x"].clone())
    e["x"][7, 3], e["x"][8, 5] = float("nan"), float("inf")
    got = call(torch, qs, e, dtype)
    keep = [t for t in range(70) if t not in (7, 8)]
    assert torch.equal(got[keep], y[keep])
    n = d["a"].shape[0]
    for t in (7, 8):
        i = int(d["ids"][t])
        assert torch.equal(got[t], y[t]) if not 0 <= i < n else not got[t].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 136])
def test_the_same_bits_in_any_batch(torch, qs, R, dtype):
    """One token, 16 (one launch for small ranks), 70 and a prompt that fills the device: the sums of a token run
    in one order."""
    d = make(torch, 4500, 576, 80, R, 5, dtype=dtype, ragged=True)
    y = call(torch, qs, d, dtype)
    for lo, hi in ((3, 4), (0, 16), (16, 27), (100, 170)):
        e = dict(d, ids=d["ids"][lo:hi].contiguous(), x=d["x"][lo:hi], base=d["base"][lo:hi])
        assert torch.equal(call(torch, qs, e, dtype), y[lo:hi]), (lo, hi)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_in_place_and_rows_behind(torch, qs, dtype):
    T, K, N = 33, 96, 120
    d = make(torch, T, K, N, 24, 4, dtype=dtype, ragged=True)
    want = call(torch, qs, d, dtype)
    wide = torch.full((T + 3, N + 6), 5.0, dtype=want.dtype, device="cuda")
    wide[:T, 3:N + 3] = d["base"]
    xs = torch.zeros(T, 2 * K + 8, dtype=torch.bfloat16, device="cuda")
    xs[:, K:2 * K] = d["x"]
    v = wide[:T, 3:N + 3]
    ws = qs.lora_new_workspace(qs.LoraAdapters(d["a"], d["b"]), T + 50)      # (one for more tokens)
    out = call(torch, qs, dict(d, x=xs[:, K:2 * K]), dtype, base=v, y=v, workspace=ws)
    assert out.data_ptr() == v.data_ptr() and torch.equal(v, want)
    assert (wide[T:] == 5).all() and (wide[:, :3] == 5).all() and (wide[:, N + 3:] == 5).all()
    e = dict(d, ids=d["ids"][:0], x=d["x"][:0], base=d["base"][:0])
    assert call(torch, qs, e, dtype).shape == (0, N)
    with pytest.raises(qs.QsmoeError):
        call(torch, qs, d, dtype, base=v, y=wide[:T, 2:N + 2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, N, R", [(5, 64, 16), (5, 65, 32), (16, 576, 8), (16, 511, 16), (33, 64, 64), (33, 127, 16), (70, 640, 128),
                                     (70, 63, 40)])
def test_rows_at_any_alignment(torch, qs, T, N, R, dtype):
    """y and base as views whose rows begin anywhere and end beside other values, which stay."""
    d = make(torch, T, 96, N, R, 4, dtype=dtype, ragged=True)
    want = call(torch, qs, d, dtype)
    for left, right in ((1, 0), (3, 6), (8, 1)):
        views = []
        for fill in (5.0, -7.0):
            wide = torch.full((T + 2, left + N + right), fill, dtype=want.dtype, device="cuda")
            views.append(wide[1:T + 1, left:left + N])
            keep = torch.ones_like(wide, dtype=torch.bool)
            keep[1:T + 1, left:left + N] = False
            views.append((wide, keep, fill))
        base, _, y, (wide, keep, fill) = views
        base.copy_(d["base"])
        call(torch, qs, d, dtype, base=base, y=y)
        assert torch.equal(y, want) and (wide[keep] == fill).all(), (left, right)


def test_in_place_leaves_tokens_without_adapter(torch, qs):
    """A NaN with a payload of its own in such a row of a bf16 y stays bit for bit."""
    d = make(torch, 20, 64, 40, 8, 2)
    d["ids"][3] = -1
    bits = d["base"].view(torch.int16)
    bits[3] = 0x7FA5
    y = d["base"]
    call(torch, qs, d, "bf16", base=y, y=y)
    assert (y.view(torch.int16)[3] == 0x7FA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,R", [(5, 64, 16), (5, 71, 16), (40, 128, 64), (40, 130, 64), (200, 192, 16)])
def test_tokens_without_adapter_keep_the_sign_of_zero(torch, qs, T, N, R, dtype):
    """y[t] = base[t] bit for bit where a token has no adapter, zeros of either sign and subnormal values among
    them; without a base such rows are +0."""
    bits = torch.int16 if dtype == "bf16" else torch.int32
    d = make(torch, T, 64, N, R, 3, dtype=dtype)
    d["ids"][1::2] = -1
    d["base"][:, ::3] = -0.0
    d["base"][:, 1::3] *= 0.0
    d["base"][:, 5::9] = -1e-39
    y = call(torch, qs, d, dtype)
    assert torch.equal(y[1::2].view(bits), d["base"][1::2].view(bits))
    check(d, y, dtype, "others")
    assert (call(torch, qs, d, dtype, base=None)[1::2].view(bits) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", [(3, 64), (3, 70), (20, 128)])
def test_values_of_A_x_past_the_largest_bf16(torch, qs, T, N, dtype):
    """scale A x between the largest values of bf16 and fp32 (rounded to bf16 it would be infinite) is carried
    like any other."""
    K, R = 32, 8
    big = torch.finfo(torch.bfloat16).max
    d = dict(a=torch.zeros(2, R, K), b=torch.zeros(2, N, R), x=torch.zeros(T, K), ids=torch.arange(T).int() % 2,
             scales=torch.tensor([1 + 2.0 ** -8, -(1 + 2.0 ** -8 - 2.0 ** -20)]), ranks=None, base=torch.randn(T, N))
    d["a"][:, 0, 0] = 1.0
    d["x"][:, 0] = big
    d["b"][:, :, 0] = torch.linspace(-1, 1, N) * 2.0 ** -100
    D = torch.bfloat16 if dtype == "bf16" else torch.float32
    for k in ("a", "b", "x"):
        d[k] = d[k].bfloat16()
    d["base"] = d["base"].to(D)
    d = {k: None if v is None else v.cuda() for k, v in d.items()}
    y = call(torch, qs, d, dtype)
    assert y.isfinite().all()
    check(d, y, dtype, (T, N))


def test_offsets_past_32_bits(torch, qs):
    T, K, N, R = 4, 64, 48, 8
    d = make(torch, T, K, N, R, 3)
    d["ids"][:] = torch.tensor([0, 2, 1, 2], dtype=torch.int32)
    want = call(torch, qs, d, "bf16")
    ld = ((1 << 31) // 3 + 8) // 8 * 8                       # (16-byte aligned rows)
    buf = torch.empty(3 * ld + 64, dtype=torch.bfloat16, device="cuda")
    for what in ("x", "base", "y"):
        w = K if what == "x" else N
        v = buf.as_strided((T, w), (ld, 1))
        if what != "y":
            v.copy_(d[what])
        kw = {"y": v} if what == "y" else {}
        assert torch.equal(call(torch, qs, dict(d, **({} if what == "y" else {what: v})), "bf16", **kw), want), what
    # an adapter stack of more than 2^31 elements of B
    n, N = 130, 65536
    b = torch.zeros(n, N, 256, dtype=torch.bfloat16, device="cuda")
    a = torch.zeros(n, 256, 8, dtype=torch.bfloat16, device="cuda")
    a[n - 1, 255, :], b[n - 1, :, 255] = 1.0, 1.0
    y = qs.lora_gemm(qs.LoraAdapters(a, b), torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda"),
                     torch.ones(2, 8, dtype=torch.bfloat16, device="cuda"))
    assert (y[0] == 8).all() and (y[1] == 0).all()


def test_beside_a_quantized_projection(torch, qs):
    """mx4_gemm with adapters: the product, then the adapters in place."""
    T, K, N = 19, 256, 304
    d = make(torch, T, K, N, 16, 3, dtype="f32")
    c, s = qs.mx4_quantize(torch.randn(N, K, device="cuda"))
    ad = qs.LoraAdapters(d["a"], d["b"], scales=d["scales"])
    for yt in (torch.float32, torch.bfloat16):
        y0 = qs.mx4_gemm(c, s, N, K, d["x"], y_dtype=yt)
        want = qs.lora_gemm(ad, d["ids"], d["x"], base=y0)
        got = qs.mx4_gemm(c, s, N, K, d["x"], y_dtype=yt, adapters=ad, adapter_ids=d["ids"])
        assert torch.equal(got, want)
    # and q8_gemv's result for one token, in place
    y = torch.randn(1, N, device="cuda")
    e = dict(d, ids=d["ids"][:1], x=d["x"][:1], base=y.clone())
    qs.lora_gemm(ad, e["ids"], e["x"], base=y, y=y)
    check(e, y, "f32", "in place")


def test_streams_and_graphs(torch, qs):
    d = make(torch, 50, 256, 300, 16, 6)
    ad = qs.LoraAdapters(d["a"], d["b"], scales=d["scales"])
    want = qs.lora_gemm(ad, d["ids"], d["x"], base=d["base"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qs.lora_gemm(ad, d["ids"], d["x"], base=d["base"], stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    y, ws = torch.empty_like(want), qs.lora_new_workspace(ad, 50)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.lora_gemm(ad, d["ids"], d["x"], base=d["base"], y=y, workspace=ws)
    for seed in range(3):
        e = make(torch, 50, 256, 300, 16, 6, seed=seed)
        for k in ("ids", "x", "base"):
            d[k].copy_(e[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, qs.lora_gemm(ad, d["ids"], d["x"], base=d["base"]))


@pytest.mark.parametrize("n,T", [(1, 65), (3, 200), (40, 512), (40, 65), (9000, 700), (70, 3000), (2, 70000)])
def test_orders_of_requests(torch, qs, n, T):
    """Batches that are ordered by adapter first (more adapters than the order tells apart among them),
    runs that are not, and batches too long for it: each token's bits are those of its own call."""
    g = torch.Generator().manual_seed(n + T)
    K, R = 32, 8
    N = (4 << 20) // (T // 16 * R) + 8 if T <= 65536 else 24 # (as wide as it takes for a batch to be ordered)
    rnd = lambda *s: torch.randn(*s, device="cuda")
    torch.manual_seed(n + T)
    a, b, x, base = rnd(n, R, K).bfloat16(), rnd(n, N, R).bfloat16(), rnd(T, K).bfloat16(), rnd(T, N)
    ad = qs.LoraAdapters(a, b)
    mixed = torch.randint(-2, n + 2, (T,), generator=g, dtype=torch.int32)
    runs = (torch.arange(T) // 50 % n).int()
    for ids in (mixed, runs, torch.full((T,), n - 1, dtype=torch.int32), torch.full((T,), -1, dtype=torch.int32)):
        ids = ids.cuda()
        y = qs.lora_gemm(ad, ids, x, base=base)
        again = base.clone()
        qs.lora_gemm(ad, ids, x, base=again, y=again)
        assert torch.equal(y, again)
        part = torch.cat([qs.lora_gemm(ad, ids[i:i + 16], x[i:i + 16], base=base[i:i + 16]) for i in range(0, min(T, 800), 16)])
        assert torch.equal(y[:len(part)], part)
        rows = [0, T // 2, T - 1]
        w, bound = lora_of(a, b, ids, x, base, rows)
        ref.check(np64(y)[rows], w, bound, False)


def lora_of(a, b, ids, x, base, rows):
    """The reference for some rows, on their adapters only."""
    i = ids.cpu().numpy()[rows]
    ok = [int(v) if 0 <= v < a.shape[0] else -1 for v in i]
    use = [max(v, 0) for v in ok]
    return ref.forward(np64(a[use]), np64(b[use]), [j if v >= 0 else -1 for j, v in enumerate(ok)], np64(x)[rows],
                       np64(base)[rows], f32=True)
