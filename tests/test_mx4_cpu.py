"""MX4 on the host: the refusals of the C ABI (every call below is refused, or has nothing to
do, before anything is enqueued, so no GPU is needed and the fake pointers are never read),
and pins of the plain reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import mx4_ref as ref
import quantized_sparse_moe_amd as q

FAKE = 0x7F0000000000          # 256-byte aligned, never dereferenced
FAR = FAKE + (1 << 40)
BAD = ctypes.c_size_t(-1).value
INV, UNS, WS = q.MOE_ERR_INVALID, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE


def quantize(x=FAKE, dt=q.MOE_BF16, rows=4, K=64, ldx=64, layout=q.MX4_TILES, c=FAR, s=FAR):
    return q.lib().mx4_quantize(x, dt, rows, K, ldx, layout, c, s, None)


def dequantize(c=FAR, s=FAR, rows=4, K=64, layout=q.MX4_TILES, y=FAKE, dt=q.MOE_F32, ldy=64):
    return q.lib().mx4_dequantize(c, s, rows, K, layout, y, dt, ldy, None)


def pack(c=FAKE, s=FAKE + (1 << 30), rows=32, K=64, tc=FAR, ts=FAR + (1 << 30)):
    return q.lib().mx4_pack_rows16(c, s, rows, K, tc, ts, None)


def gemm(wc=FAKE, wsc=FAKE, N=32, K=64, x=FAKE, T=4, ldx=64, y=FAKE, dt=q.MOE_F32, ldy=32, ws=FAKE, nb=1 << 40):
    return q.lib().mx4_gemm(wc, wsc, N, K, x, T, ldx, y, dt, ldy, ws, nb, None)


def gemm_mx4x(wc=FAKE, wsc=FAKE, N=32, K=64, xc=FAKE, xs=FAKE, T=4, y=FAKE, dt=q.MOE_F32, ldy=32, ws=FAKE,
              nb=1 << 40):
    return q.lib().mx4_gemm_mx4x(wc, wsc, N, K, xc, xs, T, y, dt, ldy, ws, nb, None)


@pytest.mark.parametrize("K", [0, 16, 31, 48, 65568])
def test_column_limits(K):
    assert quantize(K=K, ldx=1 << 17) == UNS and dequantize(K=K, ldy=1 << 17) == UNS and pack(K=K) == UNS
    assert gemm(K=K, ldx=1 << 17) == UNS and gemm_mx4x(K=K) == UNS
    for f in (q.lib().mx4_codes_size, q.lib().mx4_scales_size):
        assert f(4, K, q.MX4_ROWS) == BAD and f(4, K, q.MX4_TILES) == BAD
    assert q.lib().mx4_gemm_workspace_size(32, K, 4) == BAD


def test_row_limits_and_enums():
    big = (1 << 26) + 1
    assert quantize(rows=big) == UNS and dequantize(rows=big) == UNS and pack(rows=big) == UNS
    assert gemm(N=big, ldy=big) == UNS and gemm_mx4x(N=big, ldy=big) == UNS
    assert gemm(T=(1 << 20) + 1) == UNS and gemm_mx4x(T=(1 << 20) + 1) == UNS
    assert quantize(rows=-1) == INV and dequantize(rows=-1) == INV and pack(rows=-1) == INV
    assert gemm(T=-1) == INV and gemm(N=-1) == INV and gemm_mx4x(T=-1) == INV
    assert quantize(layout=2) == INV and dequantize(layout=-1) == INV
    assert quantize(dt=3) == INV and dequantize(dt=7) == INV
    assert gemm(dt=q.MOE_F16) == INV and gemm_mx4x(dt=q.MOE_F16) == INV
    assert q.lib().mx4_codes_size(4, 64, 2) == BAD and q.lib().mx4_scales_size(-1, 64, 0) == BAD
    assert q.lib().mx4_gemm_workspace_size(32, 64, (1 << 20) + 1) == BAD


def test_pointers_and_strides():
    for bad in (None, FAKE + 8):
        assert quantize(x=bad) == INV and quantize(c=bad) == INV
        assert dequantize(y=bad) == INV and dequantize(c=bad) == INV
        assert pack(c=bad) == INV and pack(tc=bad) == INV
        assert gemm(wc=bad) == INV and gemm(x=bad) == INV and gemm_mx4x(xc=bad) == INV and gemm_mx4x(wc=bad) == INV
    for bad in (None, FAKE + 2):
        assert quantize(s=bad) == INV and dequantize(s=bad) == INV and pack(s=bad) == INV and pack(ts=bad) == INV
        assert gemm(wsc=bad) == INV and gemm_mx4x(wsc=bad) == INV and gemm_mx4x(xs=bad) == INV
        assert gemm(y=bad) == INV and gemm_mx4x(y=bad) == INV
    assert gemm(y=FAKE + 1, dt=q.MOE_BF16) == INV
    assert quantize(ldx=32) == INV and quantize(ldx=68) == INV                  # short, misaligned rows
    assert quantize(dt=q.MOE_F32, ldx=66) == INV and dequantize(ldy=66) == INV
    assert dequantize(dt=q.MOE_F16, ldy=68) == INV
    assert gemm(ldx=60) == INV and gemm(ldx=68) == INV and gemm(ldy=31) == INV and gemm_mx4x(ldy=31) == INV


def test_rows_of_x_too_far_apart():
    assert gemm(ldx=(1 << 27) + 8) == UNS and gemm(ldx=(1 << 27) + 8, T=0) == q.MOE_OK


def test_overlapping_repack_is_refused():
    """Sources and destinations of the repack, and its two destinations, must be apart."""
    n = q.lib().mx4_codes_size(32, 64, q.MX4_ROWS)
    assert pack(tc=FAKE) == INV and pack(tc=FAKE + n - 16) == INV
    assert pack(ts=FAKE + 16) == INV and pack(tc=FAKE + (1 << 30)) == INV
    assert pack(ts=FAR + 16) == INV


def test_empty_calls_enqueue_nothing():
    assert quantize(rows=0, x=None, c=None, s=None) == q.MOE_OK
    assert dequantize(rows=0, y=None, c=None, s=None) == q.MOE_OK
    assert pack(rows=0, c=None, s=None, tc=None, ts=None) == q.MOE_OK
    assert gemm(T=0, x=None, y=None, ws=None) == q.MOE_OK and gemm(N=0, ldy=0, wc=None) == q.MOE_OK
    assert gemm_mx4x(T=0, xc=None, y=None) == q.MOE_OK
    assert q.lib().mx4_gemm_workspace_size(32, 64, 0) == 0


def test_workspace():
    """A product that needs a workspace refuses one that is missing, misaligned or short."""
    for N, K, T in ((2048, 2048, 1), (2048, 8192, 40), (512, 2048, 300), (16384, 2048, 4096), (130, 4096, 1000)):
        need = q.lib().mx4_gemm_workspace_size(N, K, T)
        assert need != BAD
        for f, kw in ((gemm, dict(ldx=K)), (gemm_mx4x, {})):
            if need:
                for w in (dict(ws=None), dict(ws=FAKE + 64), dict(nb=need - 1)):
                    assert f(N=N, K=K, T=T, ldy=N, **kw, **w) == WS
            assert f(N=N, K=K, T=T, ldy=N, ws=None, y=None, **kw) == INV


@pytest.mark.parametrize("N,K", [(1, 32), (100, 8192), (2048, 2048), (2048, 8192), (16384, 2048), (40000, 65536)])
def test_workspace_for_more_tokens_serves_fewer(N, K):
    """The size never falls as T grows (a smaller batch may be split into more shares)."""
    sizes = [q.lib().mx4_gemm_workspace_size(N, K, T) for T in [*range(1, 700), 1023, 1024, 1025, 4096, 1 << 20]]
    assert sizes == sorted(sizes) and sizes[-1] != BAD


@pytest.mark.parametrize("N,K", [(2560, 8192), (3000, 8192), (2048, 8192), (2700, 2560), (1, 65536), (4200, 3584)])
def test_every_share_of_the_columns_has_some(N, K):
    """The workspace of a split product holds the sums of its shares: no more of them than there are
    pieces of the columns, which are dealt out in whole quads of 512."""
    pitch, quads = -(-N // 4) * 4, -(-K // 512)
    for T in (17, 37, 64):                                       # (one row of tiles)
        size = q.lib().mx4_gemm_workspace_size(N, K, T)
        shares = size // (4 * T * pitch)
        assert size == shares * 4 * T * pitch and shares > 1
        per = -(-quads // shares)
        assert (shares - 1) * per < quads, (N, K, T, shares)


def mx4_desc(**kw):
    d = q.moe_layer_desc()
    d.hidden, d.inter, d.n_experts, d.top_k, d.bits, d.group = 2048, 512, 256, 8, 4, 32
    d.scale_dtype = q.MOE_E8M0
    d.router_w = FAKE
    d.gate, d.up = q.moe_qmat(FAKE, FAKE, None, 1024), q.moe_qmat(FAKE + 512 * 1024, FAKE, None, 1024)
    d.down = q.moe_qmat(FAKE, FAKE, None, 2048)
    d.has_shared = 1
    d.s_gate, d.s_up, d.s_down = d.gate, d.up, d.down
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def forward(d, T=4, x=FAKE, y=FAKE, dt=q.MOE_BF16, ws=FAKE, nb=1 << 40):
    return q.lib().moe_layer_forward(ctypes.byref(d), x, T, y, dt, None, None, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(group=64), UNS), (dict(bits=8), UNS), (dict(hidden=2080), UNS), (dict(inter=96), UNS),
    (dict(n_experts=257), UNS), (dict(top_k=17), UNS),
    (dict(gate=q.moe_qmat(FAKE, FAKE, None, 1000)), INV),              # matrices must start at a panel
    (dict(down=q.moe_qmat(FAKE, FAKE, None, 2032)), INV),              # stride < rows
    (dict(up=q.moe_qmat(FAKE + 8, FAKE, None, 1024)), INV), (dict(up=q.moe_qmat(FAKE, FAKE + 2, None, 1024)), INV),
    (dict(s_down=q.moe_qmat(None, FAKE, None, 2048)), INV), (dict(s_gate=q.moe_qmat(FAKE, None, None, 1024)), INV),
    (dict(router_w=None), INV), (dict(shared_gate_w=FAKE, has_shared=0), INV),
])
def test_layer_descriptor(kw, status):
    d = mx4_desc(**kw)
    for T in (4, 100, 400):
        assert forward(d, T=T) == status
    assert q.lib().moe_workspace_size(ctypes.byref(d), 4) == BAD


def test_layer_descriptor_accepted():
    """Biases are unused, and the affine layers' limit on (top_k + 1) * inter does not apply."""
    assert forward(mx4_desc(), T=0) == q.MOE_OK
    wide = mx4_desc(inter=2048, top_k=16, gate=q.moe_qmat(FAKE, FAKE, None, 4096), up=q.moe_qmat(FAKE, FAKE, None, 4096),
                    s_gate=q.moe_qmat(FAKE, FAKE, None, 4096), s_up=q.moe_qmat(FAKE, FAKE, None, 4096))
    assert q.lib().moe_workspace_size(ctypes.byref(wide), 64) != BAD
    affine = mx4_desc(scale_dtype=q.MOE_F16, group=64)
    assert forward(affine) == INV                                      # (needs biases)


def test_layer_tensors_are_checked():
    """from_mx4 refuses tensors of another size, type or layout before anything reads them."""
    import torch
    H, I, E = 128, 64, 3

    def mat(rows, cols):
        return (torch.zeros(q.lib().mx4_codes_size(rows, cols, q.MX4_TILES), dtype=torch.uint8),
                torch.zeros(q.lib().mx4_scales_size(rows, cols, q.MX4_TILES), dtype=torch.uint8))

    def make(**kw):
        a = dict(router_w=torch.zeros(E, H, dtype=torch.bfloat16), gate_up=mat(E * 2 * I, H), down=mat(E * H, I))
        a.update(kw)
        return q.LayerDesc.from_mx4(H, I, E, 2, **a)

    make()
    make(router_bias=torch.zeros(E), shared=(mat(2 * I, H), mat(H, I)), shared_gate_w=torch.zeros(H, dtype=torch.bfloat16))
    gu = mat(E * 2 * I, H)
    for bad in (dict(router_w=torch.zeros(E, H)), dict(router_w=torch.zeros(E, H - 32, dtype=torch.bfloat16)),
                dict(router_w=torch.zeros(H, E, dtype=torch.bfloat16).t()),
                dict(router_bias=torch.zeros(E, dtype=torch.float64)), dict(router_bias=torch.zeros(E + 1)),
                dict(shared_gate_w=torch.zeros(H)), dict(gate_up=(gu[0][:-16], gu[1])), dict(gate_up=(gu[0], gu[1][4:])),
                dict(down=(gu[0][::2], gu[1])), dict(shared=(mat(I, H), mat(H, I)))):
        with pytest.raises(q.QsmoeError):
            make(**bad)


@pytest.mark.parametrize("what,dtype", [("router_w", "float16"), ("shared_gate_w", "float16"), ("router_bias", "int32"),
                                        ("router_bias", "uint32"), ("router_w", "float32")])
def test_layer_tensors_of_another_type_of_the_same_width(what, dtype):
    """from_mx4 refuses 16- and 32-bit types it would read as something else; bits are taken."""
    import torch
    H, I, E = 128, 64, 3
    mat = lambda rows, cols: tuple(torch.zeros(f(rows, cols, q.MX4_TILES), dtype=torch.uint8)
                                   for f in (q.lib().mx4_codes_size, q.lib().mx4_scales_size))
    a = dict(router_w=torch.zeros(E, H, dtype=torch.int16), gate_up=mat(E * 2 * I, H), down=mat(E * H, I),
             router_bias=torch.zeros(E), shared=(mat(2 * I, H), mat(H, I)), shared_gate_w=torch.zeros(H, dtype=torch.uint16))
    q.LayerDesc.from_mx4(H, I, E, 2, **a)
    a[what] = torch.zeros(a[what].shape, dtype=getattr(torch, dtype))
    with pytest.raises(q.QsmoeError, match=what):
        q.LayerDesc.from_mx4(H, I, E, 2, **a)


def test_layer_workspace():
    d = mx4_desc()
    f = lambda T, c=0: q.lib().moe_workspace_size_chunked(ctypes.byref(d), T, c)
    sizes = [f(T) for T in [*range(1, 200), 1000, 4096]]
    assert sizes == sorted(sizes) and f(0) == 0 and f(16384) == f(4096)
    assert f(4096, 100) < f(4096, 1000) < f(4096, 4096)
    for T in (1, 64, 65, 129, 5000):
        least = f(T, 2)
        assert forward(d, T=T, nb=least - 1) == WS and forward(d, T=T, ws=None) == WS
        assert forward(d, T=T, ws=FAKE + 64) == WS
    assert forward(d, x=FAKE + 2) == INV and forward(d, dt=q.MOE_F16) == INV and forward(d, T=-1) == INV


def test_sizes_of_the_layouts():
    for rows, K in ((1, 32), (16, 128), (17, 160), (130, 2080)):
        c = np.zeros((rows, K), np.uint8)
        s = np.zeros((rows, K // 32), np.uint8)
        tc, ts = ref.to_tiles(c, s)
        f, g = q.lib().mx4_codes_size, q.lib().mx4_scales_size
        assert f(rows, K, q.MX4_TILES) == tc.size and g(rows, K, q.MX4_TILES) == ts.size
        assert f(rows, K, q.MX4_ROWS) == rows * K // 2 and g(rows, K, q.MX4_ROWS) == s.size


# ------------------------------------------------------------- pins of the reference
def test_reference_block_by_hand():
    """Largest value 7: floor(log2 7) = 2, so the scale is 2^0; ties go to even codes."""
    x = np.zeros((1, 32))
    x[0, :14] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.26, -0.74, -5.01, 0.24, 1.5, -6.0]
    c, s = ref.quantize(x)
    assert s[0, 0] == 127
    assert c[0, :14].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 9, 9, 15, 0, 3, 15]
    v = ref.values(c, s)[0]
    assert v[:14].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, -.5, -.5, -6, 0, 1.5, -6]


def test_reference_scale_limits():
    x = np.zeros((4, 32))
    x[1, 0] = 2.0 ** -126                                      # 2^-128 would be the scale: clamped to 2^-127
    x[2, 0] = 2.0 ** 127
    x[3, 0] = np.nan
    c, s = ref.quantize(x)
    assert s[:, 0].tolist() == [0, 0, 252, 255] and c[1, 0] == 4 and c[2, 0] == 6 and c[3].max() == 0
    v = ref.values(c, s)
    assert v[1, 0] == 2.0 ** -126 and v[2, 0] == 2.0 ** 127 and np.isnan(v[3]).all()


def test_reference_tiles_round_trip():
    """Every entry of the tile layout, found again from its stated position."""
    rng = np.random.default_rng(0)
    rows, K = 35, 672
    c = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = rng.integers(0, 255, (rows, K // 32)).astype(np.uint8)
    tc, ts = ref.to_tiles(c, s)
    S, Q = 6, 2
    for _ in range(500):
        r, k = int(rng.integers(rows)), int(rng.integers(K))
        lane = r % 16 + 16 * (k % 128 // 32)
        byte = tc[((r // 16 * S + k // 128) * 64 + lane) * 16 + k % 32 // 2]
        assert (byte >> (4 * (k % 2))) & 15 == c[r, k]
        st = k // 128
        assert ts[((r // 16 * Q + st // 4) * 64 + lane) * 4 + st % 4] == s[r, k // 32]


def test_reference_quantization_error():
    """Within the grid a value is off by at most half a step: |x - v| <= |x| / 4 for values of
    magnitude >= the scale, and half of the smallest step (a quarter of the scale) below."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((64, 256))
    c, s = ref.quantize(x)
    v, u = ref.values(c, s), np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    inside = np.abs(x) <= 6 * u
    assert (np.abs(x - v)[inside] <= np.maximum(np.abs(x) / 4, u / 4)[inside]).all()
    assert (np.abs(v)[~inside] == 6 * u[~inside]).all()
