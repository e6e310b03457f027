// mx4.hip -- microscaled 4-bit (MX4) quantization, dequantization and the load-time repack
// into 16-row tiles (format and layouts: mx4.h).
//
// Quantization of a block of 32: the scale is the power of two 2^e with
// e = floor(log2 max|x|) - 2 (clamped to the byte's range, so a zero block has byte 0),
// elements x / 2^e round to the nearest code, ties to the even code, and saturate at 6.
// x / 2^e is exact, so a code is one rounding of x.  A block that holds a NaN or an infinity
// becomes a NaN block (byte 255, codes 0).
//
// All of these move bytes: a thread takes 8 consecutive values (16-byte reads), four
// neighbouring lanes a block, and the block's largest value goes round the four by DPP.  They
// are bound by memory: 4096 x 8192 bf16 to tiles 16.4 us (5.2 TB/s read and written; a large
// copy reaches 4.7, part of these 85 MB stay in the Infinity Cache) and back 13.6; 16390 x 2080
// fp32 to rows 29.0 (5.3 TB/s) and back 24.8; 268 MB of codes repacked 110 (5.2 TB/s).  One row
// of 2048 takes 2.5 and 2.3, a launch.
#include "mx4.h"

namespace qs {

namespace {

// 8 values of one thread: packed codes (4 bytes) and the block's scale byte (the same in
// the block's four lanes).  Every lane of the wave must call it.
struct Vals8 {
    u32x4 v[2];                              // 8 bf16 / f16 (v[0]) or 8 f32
};
template <int DT>
__device__ __forceinline__ Vals8 load8(const void *x, int64_t i, bool live) {
    Vals8 r;
    r.v[0] = r.v[1] = (u32x4){0u, 0u, 0u, 0u};
    if (live) {
        if constexpr (DT == MOE_F32) {
            r.v[0] = *(const u32x4 *)((const float *)x + i);
            r.v[1] = *(const u32x4 *)((const float *)x + i + 4);
        } else {
            r.v[0] = *(const u32x4 *)((const uint16_t *)x + i);
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ uint32_t quant8(const Vals8 &a, uint32_t &sb) {
    // the largest |x| as ordered bits
    uint32_t m;
    if constexpr (DT == MOE_F32) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(a.v[0][i] & 0x7fffffffu, a.v[1][i] & 0x7fffffffu));
    } else {
        m = absmax8_bf16(a.v[0]);            // (f16 orders by its bits as well)
    }
    m = max(m, dpp_u32<0xB1>(m));
    m = max(m, dpp_u32<0x4E>(m));
    bool bad;
    uint32_t ef;                             // fp32 exponent field of the block's largest value
    if constexpr (DT == MOE_F32) {
        bad = m >= 0x7f800000u;
        ef = m >> 23;
    } else if constexpr (DT == MOE_BF16) {
        bad = m >= 0x7f80u;
        ef = m >> 7;
    } else {
        bad = m >= 0x7c00u;
        ef = __float_as_uint(f16_to_f32((uint16_t)m)) >> 23;
    }
    sb = bad ? 255u : (ef > 2u ? ef - 2u : 0u);
    const float s = bad ? 1.0f : e8m0_to_f32(sb);
    uint32_t c = 0;
    if constexpr (DT == MOE_F32) {
#define QS_Q(I) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(a.v[(I) >> 1][2 * ((I) & 1)]), \
                                                            __uint_as_float(a.v[(I) >> 1][2 * ((I) & 1) + 1]), s, I);
        QS_Q(0) QS_Q(1) QS_Q(2) QS_Q(3)
#undef QS_Q
    } else if constexpr (DT == MOE_BF16) {
#define QS_Q(I) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)a.v[0][I]), s, I);
        QS_Q(0) QS_Q(1) QS_Q(2) QS_Q(3)
#undef QS_Q
    } else {
#define QS_Q(I) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)a.v[0][I]), s, I);
        QS_Q(0) QS_Q(1) QS_Q(2) QS_Q(3)
#undef QS_Q
    }
    return bad ? 0u : c;
}

// Tile layout: a workgroup writes one (panel, quad).  Thread t is lane n + 16 g of the tile
// and quarter j of its block: t = 64 g + 4 n + j, so its 4 bytes of codes land at byte 4 t
// and a step's tile is written in order; a wave reads 64 bytes of each of the 16 rows.
template <int DT>
__global__ __launch_bounds__(256) void k_mx4_quantize_tiles(const void *x, int64_t rows, int K, int64_t ldx,
                                                            uint8_t *codes, uint8_t *scales) {
    const int KS = (K + 127) >> 7, KQ = (KS + 3) >> 2;
    const int t = threadIdx.x, j = t & 3, n = (t >> 2) & 15, g = t >> 6;
    for (int64_t blk = blockIdx.x; blk < (rows + 15) / 16 * KQ; blk += gridDim.x) {
        const int64_t p = blk / KQ, row = 16 * p + n;
        const int q = (int)(blk - p * KQ);
        Vals8 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 512 * q + 128 * i + 32 * g + 8 * j;
            a[i] = load8<DT>(x, row * ldx + k, row < rows && k < K);
        }
        uint32_t sw = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t sb;
            const uint32_t c = quant8<DT>(a[i], sb);
            if (4 * q + i < KS) {
                *(uint32_t *)(codes + (p * KS + 4 * q + i) * MX_TILE + 4 * t) = c;
                sw |= sb << (8 * i);
            }
        }
        if (j == 0) *(uint32_t *)(scales + (p * KQ + q) * MX_QS + 4 * (n + 16 * g)) = sw;
    }
}

// Row layout: thread t takes values 8 t .. 8 t + 7 of the matrix in row-major order (K is a
// multiple of 32, so a block never leaves its row)
template <int DT>
__global__ __launch_bounds__(256) void k_mx4_quantize_rows(const void *x, int64_t rows, int K, int64_t ldx,
                                                           uint8_t *codes, uint8_t *scales) {
    const int64_t n8 = rows * (K / 8);
    for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < n8; i0 += (int64_t)gridDim.x * 256) {
        const int64_t i = i0 + threadIdx.x;
        const bool live = i < n8;
        int64_t src = 8 * i;
        if (ldx != K && live) src = i / (K / 8) * ldx + i % (K / 8) * 8;
        uint32_t sb;
        const uint32_t c = quant8<DT>(load8<DT>(x, src, live), sb);
        if (live) {
            *(uint32_t *)(codes + 4 * i) = c;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)sb;
        }
    }
}

// 8 codes -> 8 values
template <int DT>
__device__ __forceinline__ void dequant8(uint32_t c, uint32_t sb, void *y, int64_t i) {
    const float s = __uint_as_float(sb << 23);               // (the conversion reads its exponent byte)
    float f[8];
#define QS_D(I) { const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, I); f[2 * (I)] = p[0]; f[2 * (I) + 1] = p[1]; }
    QS_D(0) QS_D(1) QS_D(2) QS_D(3)
#undef QS_D
    if constexpr (DT == MOE_F32) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(f[k]);
            b[k] = __float_as_uint(f[k + 4]);
        }
        *(u32x4 *)((float *)y + i) = a;
        *(u32x4 *)((float *)y + i + 4) = b;
    } else {
        u32x4 a;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == MOE_BF16)    // exact: two significant bits
                a[k] = __builtin_amdgcn_perm(__float_as_uint(f[2 * k + 1]), __float_as_uint(f[2 * k]), 0x07060302u);
            else
                a[k] = pack_f16x2((_Float16)f[2 * k], (_Float16)f[2 * k + 1]);
        }
        *(u32x4 *)((uint16_t *)y + i) = a;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_mx4_dequantize_tiles(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                                              int K, void *y, int64_t ldy) {
    const int KS = (K + 127) >> 7, KQ = (KS + 3) >> 2;
    const int t = threadIdx.x, j = t & 3, n = (t >> 2) & 15, g = t >> 6;
    for (int64_t blk = blockIdx.x; blk < (rows + 15) / 16 * KQ; blk += gridDim.x) {
        const int64_t p = blk / KQ, row = 16 * p + n;
        const int q = (int)(blk - p * KQ);
        const uint32_t sw = *(const uint32_t *)(scales + (p * KQ + q) * MX_QS + 4 * (n + 16 * g));
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = 4 * q + i < KS ? *(const uint32_t *)(codes + (p * KS + 4 * q + i) * MX_TILE + 4 * t) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 512 * q + 128 * i + 32 * g + 8 * j;
            if (row < rows && k < K) dequant8<DT>(c[i], (sw >> (8 * i)) & 255u, y, row * ldy + k);
        }
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_mx4_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                                             int K, void *y, int64_t ldy) {
    const int64_t n8 = rows * (K / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        int64_t dst = 8 * i;
        if (ldy != K) dst = i / (K / 8) * ldy + i % (K / 8) * 8;
        dequant8<DT>(*(const uint32_t *)(codes + 4 * i), scales[i >> 2], y, dst);
    }
}

// Row-major codes and scales -> tiles: a workgroup writes one (panel, quad), a wave one step
__global__ __launch_bounds__(256) void k_mx4_pack(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K,
                                                  uint8_t *tc, uint8_t *ts) {
    const int KS = (K + 127) >> 7, KQ = (KS + 3) >> 2;
    const int lane = threadIdx.x & 63, i = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
    for (int64_t blk = blockIdx.x; blk < (rows + 15) / 16 * KQ; blk += gridDim.x) {
        const int64_t p = blk / KQ, row = 16 * p + n;
        const int q = (int)(blk - p * KQ);
        const int s = 4 * q + i, k = 128 * s + 32 * g;
        const bool live = row < rows && k < K;
        u32x4 c = {0u, 0u, 0u, 0u};
        uint8_t sb = 0;
        if (live) {
            c = *(const u32x4 *)(codes + (row * K + k) / 2);
            sb = scales[row * (K / 32) + k / 32];
        }
        if (s < KS) *(u32x4 *)(tc + (p * KS + s) * MX_TILE + 16 * lane) = c;
        ts[(p * KQ + q) * MX_QS + 4 * lane + i] = sb;
    }
}

}  // namespace

#define QS_BY_DTYPE(DT, CALL)                                  \
    do {                                                       \
        if ((DT) == MOE_BF16) { constexpr int D = MOE_BF16; CALL; } \
        else if ((DT) == MOE_F16) { constexpr int D = MOE_F16; CALL; } \
        else { constexpr int D = MOE_F32; CALL; }              \
    } while (0)

// rows * K / 8 threads, at most a few workgroups per compute unit
static unsigned row_grid(int64_t rows, int64_t K) {
    const int64_t b = (rows * (K / 8) + 255) / 256, cap = 64 * (int64_t)n_compute_units();
    return (unsigned)(b < cap ? b : cap);
}
// one workgroup per (panel, quad), up to the 2^20 after which they take several (a launch is
// limited to 2^32 threads)
static unsigned tile_grid(int64_t rows, int64_t K) {
    const int64_t b = (rows + 15) / 16 * mx4_quads(K);
    return (unsigned)(b < (1 << 20) ? b : 1 << 20);
}

hipError_t launch_mx4_quantize(const void *x, int dtype, int64_t rows, int64_t K, int64_t ldx, int layout,
                               uint8_t *codes, uint8_t *scales, hipStream_t s) {
    if (layout == MX4_TILES)
        QS_BY_DTYPE(dtype, hipLaunchKernelGGL(k_mx4_quantize_tiles<D>, dim3(tile_grid(rows, K)), dim3(256), 0, s, x,
                                              rows, (int)K, ldx, codes, scales));
    else
        QS_BY_DTYPE(dtype, hipLaunchKernelGGL(k_mx4_quantize_rows<D>, dim3(row_grid(rows, K)), dim3(256), 0, s, x, rows,
                                              (int)K, ldx, codes, scales));
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, int layout,
                                 void *y, int dtype, int64_t ldy, hipStream_t s) {
    if (layout == MX4_TILES)
        QS_BY_DTYPE(dtype, hipLaunchKernelGGL(k_mx4_dequantize_tiles<D>, dim3(tile_grid(rows, K)), dim3(256), 0, s,
                                              codes, scales, rows, (int)K, y, ldy));
    else
        QS_BY_DTYPE(dtype, hipLaunchKernelGGL(k_mx4_dequantize_rows<D>, dim3(row_grid(rows, K)), dim3(256), 0, s, codes,
                                              scales, rows, (int)K, y, ldy));
    return hipGetLastError();
}

hipError_t launch_mx4_pack(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, uint8_t *tc,
                           uint8_t *ts, hipStream_t s) {
    hipLaunchKernelGGL(k_mx4_pack, dim3(tile_grid(rows, K)), dim3(256), 0, s, codes, scales, rows, (int)K, tc, ts);
    return hipGetLastError();
}

}  // namespace qs
