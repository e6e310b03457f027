// mx4_gemm.hip -- y = x W^T with W in MX4 tiles and x in bf16 or MX4 (format, layouts and the
// matrix instructions each takes: mx4.h).
#include "mx4.h"

namespace qs {

namespace {

struct GemmArgs {
    const uint8_t *wc, *ws;    // weight tiles and scales
    const uint8_t *xc, *xs;    // MX4 activations: tiles and scales
    const uint16_t *x;         // bf16 activations
    void *y;
    int64_t ldx, ldy;
    int N, T, K, KS, KQ, P;    // KS, KQ: steps and quads of K; P: weight panels
    int y_dtype;
    int qs;                    // waves that share a panel: one quad each of a chunk of qs quads
    int ppw;                   // panels per workgroup
};

// Few tokens: bound by the weight stream.  A wave multiplies one 16-row weight panel by MT
// 16-token activation tiles over its share of the columns; every weight tile is read once, with
// contiguous 16-byte loads straight into registers, a chunk (one quad per wave, 4 KB of codes)
// ahead of its use.  bf16 activations are staged in LDS a chunk at a time, with coalesced
// reads (an MFMA operand read from global memory touches 64 separate 16-byte pieces, which
// costs the address unit four times the 16 cycles of a contiguous one); MX4 activations come
// as tiles and need no staging.  The qs waves of a panel meet in LDS, summed in wave order.
template <bool MX, int MT>
__global__ __launch_bounds__(512) void k_mx4_skinny(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nt = blockDim.x;
    const int n = lane & 15, g = lane >> 4;
    const int pw = wave / a.qs, wq = wave % a.qs;
    const int pp = blockIdx.x * a.ppw + pw;
    const int p = pp < a.P ? pp : a.P - 1;
    const int t0 = blockIdx.y * (16 * MT);
    const int rows = a.T - t0 < 16 * MT ? a.T - t0 : 16 * MT;    // tokens of this workgroup
    const int nm = (a.T + 15) / 16;                          // activation tiles in all

    u32x4 b[4];
    uint32_t sb = 0;
    auto load_w = [&](int q) __attribute__((always_inline)) {
        const uint8_t *c = a.wc + ((int64_t)p * a.KS + 4 * q) * MX_TILE + 16 * lane;
        sb = __builtin_nontemporal_load((const uint32_t *)(a.ws + ((int64_t)p * a.KQ + q) * MX_QS + 4 * lane));
#pragma unroll
        for (int i = 0; i < 4; ++i)                          // (steps past K: a valid tile, not used)
            b[i] = __builtin_nontemporal_load((const u32x4 *)(c + (4 * q + i < a.KS ? i : 0) * MX_TILE));
    };
    if (wq < a.KQ) load_w(wq);

    const int pitch = a.qs * 1024 + 16;                      // bytes of a staged row (padded: banks)
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int q0 = 0; q0 < a.KQ; q0 += a.qs) {
        if constexpr (!MX) {
            if (q0) __syncthreads();                         // the last chunk is consumed
            const int k0 = 512 * q0, nc = a.qs * 64;         // 16-byte pieces per row
            for (int i = tid; i < rows * nc; i += nt) {
                const int r = i / nc, c = i % nc, k = k0 + 8 * c;
                u32x4 v = {0u, 0u, 0u, 0u};
                if (k < a.K) v = *(const u32x4 *)(a.x + (t0 + r) * a.ldx + k);
                *(u32x4 *)(sm + r * pitch + 16 * c) = v;
            }
            __syncthreads();
        }
        const int q = q0 + wq;
        if (q < a.KQ) {
            u32x4 bb[4];
            const uint32_t sbb = sb;
#pragma unroll
            for (int i = 0; i < 4; ++i) bb[i] = b[i];
            if (q + a.qs < a.KQ) load_w(q + a.qs);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * q + i >= a.KS) break;
                if constexpr (MX) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int mt = t0 / 16 + m < nm ? t0 / 16 + m : nm - 1;   // past T: repeated, discarded
                        const uint32_t sa = *(const uint32_t *)(a.xs + ((int64_t)mt * a.KQ + q) * MX_QS + 4 * lane);
                        const u32x4 A = *(const u32x4 *)(a.xc + ((int64_t)mt * a.KS + 4 * q + i) * MX_TILE + 16 * lane);
                        acc[m] = mx_mfma(A, bb[i], acc[m], i, sa, sbb);
                    }
                } else {
                    const float sc = mx_scale(sbb, i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf16x8 B = mx_bf16(bb[i][j], sc);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int r = 16 * m + n < rows ? 16 * m + n : rows - 1;
                            const bf16x8 A = *(const bf16x8 *)(sm + r * pitch + wq * 1024 + 256 * i + 64 * g + 16 * j);
                            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, acc[m], 0, 0, 0);
                        }
                    }
                }
            }
        }
    }

    // join the panel's waves in wave order (through LDS, one activation tile at a time)
    f32x4 *red = (f32x4 *)sm;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (a.qs > 1) {
            __syncthreads();
            red[wave * 64 + lane] = acc[m];
            __syncthreads();
            if (wq == 0) {
                f32x4 s = red[wave * 64 + lane];
                for (int w = 1; w < a.qs; ++w) s += red[(wave + w) * 64 + lane];
                acc[m] = s;
            }
        }
        const int col = 16 * p + n;
        if (wq == 0 && pp < a.P && col < a.N) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = t0 + 16 * m + 4 * g + r;
                if (t < a.T) mx_store(a.y, t * a.ldy + col, acc[m][r], a.y_dtype);
            }
        }
    }
}

template <bool MX>
hipError_t launch_skinny(GemmArgs a, hipStream_t s) {
    const int nm = (a.T + 15) / 16;
    const int MT = nm >= 3 ? 4 : nm;
    const int rows = a.T < 16 * MT ? a.T : 16 * MT;
    a.qs = 1;
    // a chunk of activations takes rows * qs KB of LDS
    while (a.qs < 8 && 2 * a.qs <= a.KQ && (MX || rows * 2 * a.qs <= 60)) a.qs *= 2;
    a.ppw = 1;
    while (a.qs * a.ppw < 8 && a.P / (2 * a.ppw) >= 2 * n_compute_units()) a.ppw *= 2;
    const int waves = a.qs * a.ppw;
    const size_t red = a.qs > 1 ? (size_t)waves * 1024 : 16, stage = MX ? 0 : (size_t)rows * (a.qs * 1024 + 16);
    void (*k)(GemmArgs) = MT == 4 ? k_mx4_skinny<MX, 4> : MT == 2 ? k_mx4_skinny<MX, 2> : k_mx4_skinny<MX, 1>;
    hipLaunchKernelGGL(k, dim3((a.P + a.ppw - 1) / a.ppw, (nm + MT - 1) / MT), dim3(64 * waves),
                       red > stage ? red : stage, s, a);
    return hipGetLastError();
}

GemmArgs make_args(const uint8_t *wc, const uint8_t *ws, int64_t N, int64_t K, int64_t T, void *y, int y_dtype,
                   int64_t ldy) {
    GemmArgs a{};
    a.wc = wc;
    a.ws = ws;
    a.N = (int)N;
    a.K = (int)K;
    a.T = (int)T;
    a.KS = (int)mx4_steps(K);
    a.KQ = (int)mx4_quads(K);
    a.P = (int)((N + 15) / 16);
    a.y = y;
    a.y_dtype = y_dtype;
    a.ldy = ldy;
    return a;
}

}  // namespace

size_t mx4_gemm_ws(int64_t T, int64_t N, int64_t K) { return 0; }

hipError_t launch_mx4_gemm(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint16_t *x, int64_t T,
                           int64_t ldx, void *y, int y_dtype, int64_t ldy, uint8_t *ws, hipStream_t s) {
    GemmArgs a = make_args(wc, wsc, N, K, T, y, y_dtype, ldy);
    a.x = x;
    a.ldx = ldx;
    return launch_skinny<false>(a, s);
}

hipError_t launch_mx4_gemm_mx4x(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint8_t *xc,
                                const uint8_t *xs, int64_t T, void *y, int y_dtype, int64_t ldy, uint8_t *ws,
                                hipStream_t s) {
    GemmArgs a = make_args(wc, wsc, N, K, T, y, y_dtype, ldy);
    a.xc = xc;
    a.xs = xs;
    return launch_skinny<true>(a, s);
}

}  // namespace qs
