"""MX4 on the GPU against the plain 64-bit implementation (mx4_ref): codes and scales bit
for bit, products within the error bound of their fp32 sums."""
import numpy as np
import pytest

import mx4_ref as ref

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
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype.is_floating_point else t.cpu().numpy()


def rand_x(rows, K, seed, special=True):
    """fp64 values with the cases a quantizer can go wrong at: ties, powers of two, zeros of
    both signs, a zero block, subnormals, the largest values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((rows, 1)))
    if special:
        b = x.reshape(-1, 32)
        grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
        b[0] = np.concatenate([grid, -grid]) * 2.0 ** -3          # every tie, largest 7 (saturates at 6)
        if len(b) > 1:
            b[1] = 0.0
            b[1, ::2] = -0.0
        if len(b) > 2:
            b[2] = np.ldexp(1.0, -rng.integers(0, 30, 32))
    return x


def to_dtype(x, dtype, torch):
    return torch.from_numpy(x).to(getattr(torch, dtype)).cuda()


def split_codes(buf, layout_rows, K):
    return buf.reshape(layout_rows, K // 2)


SHAPES = [(1, 32), (1, 64), (2, 96), (16, 128), (17, 544), (33, 2080), (5, 8192), (1, 2048), (130, 160)]


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_both_layouts(torch, qs, rows, K, dtype):
    x = to_dtype(rand_x(rows, K, seed=rows * K), dtype, torch)
    c, s = ref.quantize(np64(x))
    rc, rs = qs.mx4_quantize(x, layout=qs.MX4_ROWS)
    tc, ts = qs.mx4_quantize(x)
    torch.cuda.synchronize()
    assert np.array_equal(rc.cpu().numpy().reshape(rows, K // 2), ref.pack_rows(c))
    assert np.array_equal(rs.cpu().numpy().reshape(rows, K // 32), s)
    wc, ws = ref.to_tiles(c, s)
    assert np.array_equal(tc.cpu().numpy(), wc)
    assert np.array_equal(ts.cpu().numpy(), ws)
    pc, ps = qs.mx4_pack_rows16(rc, rs, rows, K)
    assert torch.equal(pc, tc) and torch.equal(ps, ts)
    want = ref.values(c, s)
    for layout, (cc, ss) in ((qs.MX4_ROWS, (rc, rs)), (qs.MX4_TILES, (tc, ts))):
        for yt in (torch.float32, torch.bfloat16):
            assert np.array_equal(np64(qs.mx4_dequantize(cc, ss, rows, K, y_dtype=yt, layout=layout)), want)


def test_quantize_every_bf16_pattern(torch, qs):
    """Each bf16 pattern next to largest values that put it at every position of the grid,
    infinities and NaN among them (their blocks become NaN blocks)."""
    bits = np.arange(65536, dtype=np.uint16)
    for anchor in (None, 0x3F80, 0x7F00, 0x0080, 0x4049):
        blk = np.zeros((65536, 32), np.uint16)
        blk[:, 5] = bits
        if anchor is not None:
            blk[:, 17] = anchor
        x = torch.from_numpy(blk.view(np.int16)).cuda()
        c, s = ref.quantize(ref.bf16_values(blk))
        rc, rs = qs.mx4_quantize(x, layout=qs.MX4_ROWS)
        assert np.array_equal(rc.cpu().numpy().reshape(-1, 16), ref.pack_rows(c)), anchor
        assert np.array_equal(rs.cpu().numpy().reshape(-1, 1), s), anchor


@pytest.mark.parametrize("dtype", ["float32", "float16"])
def test_quantize_extremes(torch, qs, dtype):
    info = np.finfo(dtype)
    tiny, big = float(info.smallest_subnormal), float(info.max)
    blk = np.zeros((8, 64))
    blk[0, :2] = big, -big
    blk[1, :4] = tiny, -tiny, 3 * tiny, 7 * tiny
    blk[2, 3] = np.inf
    blk[3, 40] = np.nan
    blk[4, 9] = -np.inf
    blk[5] = tiny
    blk[6] = float(info.tiny)
    x = torch.from_numpy(blk.astype(dtype)).cuda()
    c, s = ref.quantize(np64(x))
    tc, ts = qs.mx4_quantize(x)
    wc, ws = ref.to_tiles(c, s)
    assert np.array_equal(ts.cpu().numpy(), ws)
    assert np.array_equal(tc.cpu().numpy(), wc)


def test_more_tiles_than_workgroups(torch, qs):
    """More (panel, quad) pairs than the launch has workgroups: the two layouts, each made by its
    own kernel, agree over the whole matrix."""
    rows, K = 16 * (1 << 20) + 53, 32
    x = torch.randn(rows, K, device="cuda", dtype=torch.bfloat16)
    rc, rs = qs.mx4_quantize(x, layout=qs.MX4_ROWS)
    tc, ts = qs.mx4_quantize(x)
    pc, ps = qs.mx4_pack_rows16(rc, rs, rows, K)
    assert torch.equal(pc, tc) and torch.equal(ps, ts)
    assert torch.equal(qs.mx4_dequantize(tc, ts, rows, K, y_dtype=torch.bfloat16),
                       qs.mx4_dequantize(rc, rs, rows, K, y_dtype=torch.bfloat16, layout=qs.MX4_ROWS))
    c, s = ref.quantize(np64(x[-53:]))
    assert np.array_equal(rc[-53 * 16:].cpu().numpy().reshape(53, 16), ref.pack_rows(c))
    assert np.array_equal(rs[-53:].cpu().numpy().reshape(53, 1), s)


def test_quantize_strided_rows(torch, qs):
    x = to_dtype(rand_x(19, 512, seed=3), "bfloat16", torch)
    part = x[:, 64:64 + 288]                                     # row stride 512, offset 128 bytes
    for layout in (qs.MX4_ROWS, qs.MX4_TILES):
        a = qs.mx4_quantize(part, layout=layout)
        b = qs.mx4_quantize(part.contiguous(), layout=layout)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        y = torch.full((19, 320), 7.0, device="cuda")
        qs.mx4_dequantize(*a, 19, 288, y=y[:, 16:16 + 288], layout=layout)
        assert torch.equal(y[:, 16:304], qs.mx4_dequantize(*b, 19, 288, layout=layout))
        assert (y[:, :16] == 7).all() and (y[:, 304:] == 7).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_dequantize_every_code_and_scale(torch, qs, dtype):
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    want = ref.values(codes, scales)
    # in the output type: one rounding (fp32 and bf16 hold every finite value below their
    # overflow exactly; fp16 rounds)
    with np.errstate(over="ignore"):
        want = want.astype(np.float16 if dtype == "float16" else np.float32).astype(np.float64)
    for layout in (qs.MX4_ROWS, qs.MX4_TILES):
        c, s = (ref.pack_rows(codes), scales) if layout == qs.MX4_ROWS else ref.to_tiles(codes, scales)
        y = qs.mx4_dequantize(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), 256, 32,
                              y_dtype=getattr(torch, dtype), layout=layout)
        got = np64(y)
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


# --------------------------------------------------------------------------- products
def weights(N, K, seed, torch, qs):
    """An MX4 matrix: float64 values and device tiles (row scales spread, so scales differ)."""
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((N, K)) * np.exp(rng.standard_normal((N, 1))) / np.sqrt(K)
    c, s = ref.quantize(w)
    tc, ts = qs.mx4_pack_rows16(torch.from_numpy(ref.pack_rows(c)).cuda(), torch.from_numpy(s).cuda(), N, K)
    return ref.values(c, s), tc, ts


def activations(T, K, seed, torch):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K))
    x[:, rng.integers(0, K, max(1, K // 200))] *= 30.0
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


def check(y, want, bound, what):
    got = np64(y)
    extra = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) if str(y.dtype).endswith("bfloat16") else 0.0
    err = np.abs(got - want)
    bad = ~(err <= bound * (1 + 2.0 ** -7) + extra + 2.0 ** -140)
    assert not bad.any(), (what, int(bad.sum()), float((err - bound - extra).max()), np.argwhere(bad)[:4].tolist())


GEMM = [(4, 80, 65536), (16, 64, 4096), (18, 4100, 96), (520, 16400, 64), (1024, 16384, 160), (1, 16, 32), (1, 1, 64), (1, 2048, 2048), (2, 130, 96), (3, 2048, 8192), (5, 17, 160), (7, 64, 544),
        (8, 256, 512), (9, 33, 640), (16, 2048, 2048), (16, 48, 8192), (17, 100, 1056), (31, 64, 128),
        (33, 2080, 2080), (37, 2048, 8192), (64, 128, 2048), (65, 31, 288), (130, 250, 576), (257, 512, 1024),
        (300, 1000, 2080), (513, 2048, 512), (1000, 130, 4096)]


@pytest.mark.parametrize("T,N,K", GEMM)
def test_gemm(torch, qs, T, N, K):
    w, wc, ws = weights(N, K, T + N + K, torch, qs)
    x = activations(T, K, T * K + N, torch)
    xv = np64(x)
    want, bound = xv @ w.T, ref.product_bound(xv, w)
    check(qs.mx4_gemm(wc, ws, N, K, x), want, bound, "f32")
    check(qs.mx4_gemm(wc, ws, N, K, x, y_dtype=torch.bfloat16), want, bound, "bf16")
    # the same with x quantized
    c, s = ref.quantize(xv)
    xq = ref.values(c, s)
    xc, xs = qs.mx4_quantize(x)
    want, bound = xq @ w.T, ref.product_bound(xq, w)
    check(qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T), want, bound, "mx f32")
    check(qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T, y_dtype=torch.bfloat16), want, bound, "mx bf16")


@pytest.mark.parametrize("T,N,K", [(37, 2560, 8192), (20, 3000, 8192), (64, 2700, 2560), (17, 4200, 3584)])
def test_gemm_columns_that_the_shares_do_not_divide(torch, qs, T, N, K):
    """Split products whose quads of columns are no multiple of the shares."""
    test_gemm(torch, qs, T, N, K)


# large tiles (128 x 256): whole and partial quads of columns, first and last steps alone
@pytest.mark.parametrize("K", [32, 96, 128, 416, 512, 544, 640, 1024, 1184, 1664])
def test_gemm_large_tiles(torch, qs, K):
    T, N = 1000, 14500
    w, wc, ws = weights(N, K, K, torch, qs)
    x = activations(T, K, K + 1, torch)
    xv = np64(x)
    check(qs.mx4_gemm(wc, ws, N, K, x, y_dtype=torch.bfloat16), xv @ w.T, ref.product_bound(xv, w), "bf16")
    c, s = ref.quantize(xv)
    xq = ref.values(c, s)
    xc, xs = qs.mx4_quantize(x)
    check(qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T), xq @ w.T, ref.product_bound(xq, w), "mx f32")


@pytest.mark.parametrize("ldx", [2 ** 23, 2 ** 23 + 8])
def test_gemm_rows_far_apart(torch, qs, ldx):
    """Rows of x so far apart that their offsets pass 31 bits inside a tile."""
    T, N, K = 130, 58000, 96                     # two by 227 tiles of 128 x 256
    w, wc, ws = weights(N, K, 8, torch, qs)
    x = activations(T, K, 9, torch)
    xb = torch.empty(T * ldx, dtype=torch.bfloat16, device="cuda").view(T, ldx)
    xb[:, :K] = x
    xv = np64(x)
    check(qs.mx4_gemm(wc, ws, N, K, xb[:, :K]), xv @ w.T, ref.product_bound(xv, w), "f32")


@pytest.mark.parametrize("T", [9, 21])
def test_gemm_rows_at_the_limit_apart(torch, qs, T):
    N, K, ldx = 210, 160, 2 ** 27
    w, wc, ws = weights(N, K, 10, torch, qs)
    x = activations(T, K, 11, torch)
    xb = torch.empty(T * ldx, dtype=torch.bfloat16, device="cuda").view(T, ldx)
    xb[:, :K] = x
    xv = np64(x)
    check(qs.mx4_gemm(wc, ws, N, K, xb[:, :K]), xv @ w.T, ref.product_bound(xv, w), "f32")


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_gemm_strides_and_guards(torch, qs, T):
    """Rows of x and y inside wider buffers; what lies beside and behind y is left as it was."""
    N, K = 90, 416
    w, wc, ws = weights(N, K, 5, torch, qs)
    xb = activations(T, K + 32, 6, torch)
    x = xb[:, 16:16 + K]
    yb = torch.full((T + 3, N + 21), 7.0, device="cuda")
    y = yb[:T, 5:5 + N]
    qs.mx4_gemm(wc, ws, N, K, x, y=y)
    assert torch.equal(y, qs.mx4_gemm(wc, ws, N, K, x.contiguous()))
    assert (yb[T:] == 7).all() and (yb[:, :5] == 7).all() and (yb[:, 5 + N:] == 7).all()
    yb.fill_(7.0)
    xc, xs = qs.mx4_quantize(x)
    qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T, y=y)
    assert torch.equal(y, qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T))
    assert (yb[T:] == 7).all() and (yb[:, :5] == 7).all() and (yb[:, 5 + N:] == 7).all()


@pytest.mark.parametrize("T", [4, 40, 200])
@pytest.mark.parametrize("sigma", [1e-30, 1e-38, 1e30])
def test_gemm_range(torch, qs, T, sigma):
    """Activations far from 1, bf16 subnormals among them."""
    N, K = 48, 288
    w, wc, ws = weights(N, K, 8, torch, qs)
    x = (activations(T, K, 9, torch).float() * sigma).to(torch.bfloat16)
    xv = np64(x)
    # results below fp32's normal range may be flushed
    bound = ref.product_bound(xv, w) + 2.0 ** -126 * K
    check(qs.mx4_gemm(wc, ws, N, K, x), xv @ w.T, bound, "range")


@pytest.mark.parametrize("T", [3, 20, 150])
def test_gemm_not_finite(torch, qs, T):
    """A NaN or infinity in x reaches its token only, a NaN block of W its column only."""
    N, K = 40, 256
    w, wc, ws = weights(N, K, 10, torch, qs)
    x = activations(T, K, 11, torch)
    clean = qs.mx4_gemm(wc, ws, N, K, x)
    for val in (float("nan"), float("inf"), float("-inf")):
        xx = x.clone()
        xx[1, 200] = val
        y = qs.mx4_gemm(wc, ws, N, K, xx)
        # an infinity meets zero weights (NaN) and others (infinities): no finite value is left
        assert not torch.isfinite(y[1]).any()
        keep = torch.arange(T, device="cuda") != 1
        assert torch.equal(y[keep], clean[keep])
        xc, xs = qs.mx4_quantize(xx)
        y = qs.mx4_gemm_mx4x(wc, ws, N, K, xc, xs, T)
        assert torch.isnan(y[1]).all() and torch.isfinite(y[keep]).all()
    c, s = ref.quantize(np.where(np.isnan(w), 0, w))
    s[17, 3] = 255
    tc, ts = qs.mx4_pack_rows16(torch.from_numpy(ref.pack_rows(c)).cuda(), torch.from_numpy(s).cuda(), N, K)
    y = qs.mx4_gemm(tc, ts, N, K, x)
    keep = torch.arange(N, device="cuda") != 17
    assert torch.isnan(y[:, 17]).all() and torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("T", [2, 30, 300])
def test_gemm_of_the_smallest_and_largest_weights(torch, qs, T):
    """Scale bytes at both ends and subnormal activations against weights that bring them back: exact
    products; weights of 2^128 and more count as infinities beside bf16 activations, not beside MX4."""
    N, K = 96, 544
    rng = np.random.default_rng(T)
    for lo, hi, std in ((0, 3, 2.0 ** 100), (150, 160, 2.0 ** -130), (250, 252, 2.0 ** -20), (253, 254, 2.0 ** -20)):
        c = rng.integers(0, 16, (N, K)).astype(np.uint8)
        if hi > 252:
            c[::2] &= 9                                          # every other row below 2^127
        s = rng.integers(lo, hi + 1, (N, K // 32)).astype(np.uint8)
        wc, ws = qs.mx4_pack_rows16(torch.from_numpy(ref.pack_rows(c)).cuda(), torch.from_numpy(s).cuda(), N, K)
        w = ref.values(c, s)
        x = (torch.randn(T, K, generator=torch.Generator().manual_seed(T), dtype=torch.float64) * std).to(torch.bfloat16)
        xv = np64(x)
        y = qs.mx4_gemm(wc, ws, N, K, x.cuda())
        past = (np.abs(w) >= 2.0 ** 128).any(axis=1)
        assert past.any() == (hi > 252) and not past.all()
        assert not np.isfinite(np64(y)[:, past]).any()
        err, bound = np.abs(np64(y) - xv @ w.T), ref.product_bound(xv, w)
        assert (err[:, ~past] <= bound[:, ~past]).all(), (lo, hi)
        qc, qsc = ref.quantize(xv)
        xq = ref.values(qc, qsc)
        tc, ts = (torch.from_numpy(a).cuda() for a in ref.to_tiles(qc, qsc))
        y = np64(qs.mx4_gemm_mx4x(wc, ws, N, K, tc, ts, T))
        assert (np.abs(y - xq @ w.T) <= ref.product_bound(xq, w)).all(), (lo, hi)


@pytest.mark.parametrize("T", [1, 16, 100, 600])
def test_gemm_rows_are_independent(torch, qs, T):
    """A token's result does not depend on the other tokens, bit for bit."""
    N, K = 112, 1184
    _, wc, ws = weights(N, K, 12, torch, qs)
    x = activations(T, K, 13, torch)
    y = qs.mx4_gemm(wc, ws, N, K, x)
    other = torch.randn(T, K, device="cuda").to(torch.bfloat16) * 100
    other[T // 2] = x[T // 2]
    assert torch.equal(qs.mx4_gemm(wc, ws, N, K, other)[T // 2], y[T // 2])
    assert torch.equal(qs.mx4_gemm(wc, ws, N, K, x), y)


def test_empty_calls(torch, qs):
    _, wc, ws = weights(16, 64, 1, torch, qs)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert qs.mx4_gemm(wc, ws, 16, 64, x).shape == (0, 16)
    c, s = qs.mx4_quantize(x)
    assert c.numel() == 0 and s.numel() == 0
    assert qs.mx4_gemm_mx4x(wc, ws, 16, 64, c, s, 0).shape == (0, 16)
    assert qs.mx4_dequantize(c, s, 0, 64).shape == (0, 64)


def test_run_together_on_a_side_stream_and_in_a_graph(torch, qs):
    """Weights quantized and repacked on the device, then a quantized and an exact product,
    on a side stream and in a captured graph replayed with eager calls in between."""
    N, K, T = 80, 352, 70
    rng = np.random.default_rng(2)
    wt = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda()
    xs_ = [activations(T, K, s, torch) for s in (1, 2, 3)]

    def chain(x, ws):
        wc, wsc = qs.mx4_pack_rows16(*qs.mx4_quantize(wt, layout=qs.MX4_ROWS), N, K)
        a = qs.mx4_gemm(wc, wsc, N, K, x, workspace=ws)
        b = qs.mx4_gemm_mx4x(wc, wsc, N, K, *qs.mx4_quantize(x), T, y_dtype=torch.bfloat16, workspace=ws)
        return a, b

    ws = qs.mx4_new_workspace(T, N, K)
    eager = [chain(x, ws) for x in xs_]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain(xs_[0], qs.mx4_new_workspace(T, N, K))
    side.synchronize()
    assert torch.equal(got[0], eager[0][0]) and torch.equal(got[1], eager[0][1])
    buf = xs_[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(buf, ws)
    for i in (0, 1, 2, 1, 0):
        buf.copy_(xs_[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), i
        again = chain(xs_[i], ws)
        assert torch.equal(again[0], eager[i][0]) and torch.equal(again[1], eager[i][1]), i
