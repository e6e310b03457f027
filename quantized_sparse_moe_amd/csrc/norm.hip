// norm.hip -- the norms around a block (moe_block_norm), one pass over a row:
//     z = act(gate) * post(y)      r' = r + scale * z      x = pre(r')
// with each part optional.  A norm is v -> (v / sqrt(mean v^2 + eps)) (offset + w) + b, or the same of
// v - mean v.
//
// Bound by memory: y, r and an elementwise gate read once, r' and x written once.  A row stays in the
// registers of the P threads that read it, 8 V values each, from its first load to its last
// store.  All loads of a row are under way before its first sum, a norm's weights before that norm's first (the
// second norm's too early cost registers: 131072 x 128 22.5 us instead of 19.7).  Sums, norms and the stream are
// fp32 (r' enters the second norm unrounded, whatever type it is stored in); only the two results are
// rounded.  The mean square is taken after the mean is subtracted, from registers.
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// 16 bytes wherever they lie (the hardware takes any alignment of a value's)
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;

// The V chunks of 8 neighbouring values of a row that a thread holds, P chunks apart.  Rows of odd width or
// offset (ODD): chunks begin where the row's memory is 16-byte aligned, `skew` values before its first, so
// that only the first and the last are not whole; these are read as the 8 values nearest to them, of which
// values lo .. hi - 1 count.  ODD 2: rows of fewer than 8 values.
template <int ODD, int P, int V>
struct Chunks {
    int H, col[V], lo[V], hi[V];                             // col: first column
    __device__ __forceinline__ Chunks(int t, int h, int skew) : H(h) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int s = (t + P * i) * 8 - skew;
            col[i] = ODD ? max(min(s, H - 8), 0) : s;        // (H < 8: 0)
            lo[i] = max(s - col[i], 0);
            hi[i] = min(min(s + 8 - col[i], 8), H);
        }
    }
    __device__ __forceinline__ bool whole(int i) const { return ODD ? (lo[i] == 0) & (hi[i] == 8) : col[i] < H; }
    __device__ __forceinline__ bool in(int i, int j) const { return ODD ? (j >= lo[i]) & (j < hi[i]) : col[i] < H; }
};

// loaded and not yet widened
template <int V>
struct Raw {
    u32x4 q[V][2];
};

template <int ODD, int P, int V>
__device__ __forceinline__ void load_row(Raw<V> &w, const void *p, int dt, int64_t off, const Chunks<ODD, P, V> &c) {
    if constexpr (ODD == 2) {                                // (one chunk: values past the row repeat its last)
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t o = off + min(j, c.H - 1);
            e[j] = dt == MOE_F32 ? ((const uint32_t *)p)[o] : ((const uint16_t *)p)[o];
        }
        const u32x4 a = {e[0], e[1], e[2], e[3]}, b = {e[4], e[5], e[6], e[7]};
        const u32x4 h = {e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        w.q[0][0] = dt == MOE_F32 ? a : h;
        w.q[0][1] = b;
    } else {
        // (the first 16 bytes without a branch on the type: with one, fp32 rows waited for the tensor before; us,
        // with one and so: 16384 x 8192 222 and 211, fp32 stream 302 and 305, 16384 x 5001 238 and 213)
        const int sh = dt == MOE_F32 ? 2 : 1;
        const char *s = (const char *)p + (off << sh);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (ODD || c.col[i] < c.H) w.q[i][0] = *(const u32x4_any *)(s + ((int64_t)c.col[i] << sh));
        if (dt == MOE_F32)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (ODD || c.col[i] < c.H) w.q[i][1] = *(const u32x4_any *)(s + ((int64_t)c.col[i] << 2) + 16);
    }
}

template <int V>
__device__ __forceinline__ float value(const Raw<V> &w, int dt, int i, int j) {
    if (dt == MOE_F32) return __uint_as_float(w.q[i][j >> 2][j & 3]);
    const uint32_t u = (j & 1) ? w.q[i][0][j >> 1] >> 16 : w.q[i][0][j >> 1] & 0xffffu;
    return dt == MOE_BF16 ? __uint_as_float(u << 16) : f16_to_f32((uint16_t)u);
}
template <int V>
__device__ __forceinline__ void widen(const Raw<V> &w, int dt, float (&f)[V][8]) {
    if (dt == MOE_F32) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = value(w, MOE_F32, i, j);
    } else if (dt == MOE_BF16) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = value(w, MOE_BF16, i, j);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = value(w, MOE_F16, i, j);
    }
}

template <int ODD, int P, int V>
__device__ __forceinline__ void store_row(void *p, int dt, int64_t off, const Chunks<ODD, P, V> &c, const float (&f)[V][8]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const f32x8 v = {f[i][0], f[i][1], f[i][2], f[i][3], f[i][4], f[i][5], f[i][6], f[i][7]};
        if (dt == MOE_F32) {
            float *d = (float *)p + off + c.col[i];
            if (c.whole(i)) {
                ((f32x4_any *)d)[0] = (f32x4){v[0], v[1], v[2], v[3]};
                ((f32x4_any *)d)[1] = (f32x4){v[4], v[5], v[6], v[7]};
            } else if (ODD) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c.in(i, j)) d[j] = v[j];
            }
            continue;
        }
        const u32x4 w = dt == MOE_BF16 ? __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8v))
                                       : __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8));
        uint16_t *d = (uint16_t *)p + off + c.col[i];
        if (c.whole(i)) {
            *(u32x4_any *)d = w;
        } else if (ODD) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.in(i, j)) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// sum over the P threads of a row, in all of them; slot: of the four sums a row may take, each
// its own words, so that one barrier a sum is enough
template <int P>
__device__ __forceinline__ float row_sum(float v, int slot) {
    if constexpr (P <= 64) return group_sum(v, P);
    __shared__ float part[4][P > 64 ? P / 64 : 1];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[slot][0];
#pragma unroll
    for (int w = 1; w < P / 64; ++w) s += part[slot][w];
    return s;
}

// values that are not of the row, or another chunk's, to 0
template <int ODD, int P, int V>
__device__ __forceinline__ void mask_row(float (&f)[V][8], const Chunks<ODD, P, V> &c) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = c.in(i, j) ? f[i][j] : 0.0f;
}

// f -> its norm (values past the row's end are 0 before and not used after)
template <int ODD, int P, int V>
__device__ __forceinline__ void norm_row(float (&f)[V][8], const NormArgs &n, const Chunks<ODD, P, V> &c, int slot) {
    Raw<V> w{}, b{};
    if (n.w) load_row<ODD, P, V>(w, n.w, n.dtype, 0, c);
    if (n.b) load_row<ODD, P, V>(b, n.b, n.dtype, 0, c);
    const float ih = 1.0f / (float)c.H;
    if (n.layer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += f[i][j];
        const float m = row_sum<P>(s, slot) * ih;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = c.in(i, j) ? f[i][j] - m : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) q = __builtin_fmaf(f[i][j], f[i][j], q);
    const float rs = 1.0f / __builtin_sqrtf(row_sum<P>(q, slot + 1) * ih + n.eps);
    float g[V][8];
    if (n.w) {
        widen(w, n.dtype, g);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * rs * (g[i][j] + n.offset);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] *= rs;
    }
    if (n.b) {
        widen(b, n.dtype, g);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] += g[i][j];
    }
}

__device__ __forceinline__ float activate(float g, int act) {
    if (act == MOE_ACT_NONE) return g;
    const float s = __builtin_amdgcn_rcpf(1.0f + exp_near(-g));                    // (the reciprocal is within a step)
    return act == MOE_ACT_SIGMOID ? s : g * s;
}

template <int ODD, int P, int V>
__global__ __launch_bounds__(P < 256 ? 256 : P) void k_block_norm(BlockNormArgs a) {
    constexpr int RPW = P < 256 ? 256 / P : 1;               // rows per workgroup
    const int64_t row = a.row0 + (int64_t)blockIdx.x * RPW + threadIdx.x / P;
    if (row >= a.T) return;                                  // (whole rows; P > 64: never)
    int skew = 0;
    if constexpr (ODD == 1) {
        // (of the tensor read first; the others lie the same way where their rows are as far apart)
        const uintptr_t p = a.y ? (uintptr_t)a.y + row * a.ldy * (a.dy == MOE_F32 ? 4 : 2)
                                : (uintptr_t)a.r + row * a.ldr * (a.dr == MOE_F32 ? 4 : 2);
        skew = (int)(p >> ((a.y ? a.dy : a.dr) == MOE_F32 ? 2 : 1)) & 7;
        if (a.H + 7 > 8 * P * V) skew = 0;                   // (no chunk to spare: as they lie)
    }
    const Chunks<ODD, P, V> c(threadIdx.x % P, a.H, skew);
    Raw<V> y{}, r{}, g{};
    if (a.y) load_row<ODD, P, V>(y, a.y, a.dy, row * a.ldy, c);
    if (a.r) load_row<ODD, P, V>(r, a.r, a.dr, row * a.ldr, c);
    if (a.gate && a.gate_cols > 1) load_row<ODD, P, V>(g, a.gate, a.dg, row * a.ldg, c);
    float gt = 1.0f;
    if (a.gate && a.gate_cols == 1) {
        const int64_t o = row * a.ldg;
        gt = a.dg == MOE_F32 ? ((const float *)a.gate)[o]
                             : a.dg == MOE_BF16 ? bf16_to_f32(((const uint16_t *)a.gate)[o])
                                                : f16_to_f32(((const uint16_t *)a.gate)[o]);
    }
    float z[V][8], f[V][8];
    if (a.y) {
        widen(y, a.dy, z);
        if (a.post.on) {
            if constexpr (ODD > 0) mask_row<ODD, P, V>(z, c);
            norm_row<ODD, P, V>(z, a.post, c, 0);
        }
        float s = a.scale;
        if (a.gate) {
            if (a.gate_cols == 1) {
                gt = activate(gt, a.act);
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[i][j] *= gt;
            } else {
                widen(g, a.dg, f);
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[i][j] *= activate(f[i][j], a.act);
            }
        }
        if (a.r) {
            widen(r, a.dr, f);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) z[i][j] = __builtin_fmaf(z[i][j], s, f[i][j]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) z[i][j] *= s;
        }
        if (a.ro) store_row<ODD, P, V>(a.ro, a.dro, row * a.ldro, c, z);
    } else {
        widen(r, a.dr, z);
    }
    if (a.pre.on) {
        mask_row<ODD, P, V>(z, c);
        norm_row<ODD, P, V>(z, a.pre, c, 2);
        store_row<ODD, P, V>(a.xo, a.dxo, row * a.ldxo, c, z);
    }
}

// Threads per row: 8 values each while a row has up to 512 or 1025 to 2048 of them, 16 up to 16384, in us for
// both norms of bf16 rows (TB/s):
//   16384 x 2048  256 threads 46.0 (5.83), 64 threads of 32 values 56.9      131072 x 1024  64 of 16: 183.4 (5.85)
//   16384 x 4096  256 of 16: 95.9 (5.60), 512 of 8: 96.0                     131072 x 512   64 of 8: 93.9 (5.72)
//   16384 x 8192  512 of 16: 210 (5.11), 256 of 32: 214, 1024 of 8: 266      8192 x 16384   1024 of 16: 224 (4.80)
//   (with a gate: 266 (5.05), 291, 370; a large copy moves 4.8)
// Odd widths (read and written value by value before): 32768 x 2047 117 (4.6; 156), 16384 x 8191 286 (3.8; 530),
// 16384 x 5001 213 (3.1; 430).
template <int ODD>
void launch_p(BlockNormArgs a, hipStream_t s) {
    // (a launch has fewer than 2^32 threads)
    auto go = [&](void (*k)(BlockNormArgs), int p) {
        const int64_t rpw = p < 256 ? 256 / p : 1, most = ((int64_t)1 << 31) / p;
        for (a.row0 = 0; a.row0 < a.T; a.row0 += most) {
            const int64_t rows = a.T - a.row0 < most ? a.T - a.row0 : most;
            hipLaunchKernelGGL(k, dim3((unsigned)((rows + rpw - 1) / rpw)), dim3((unsigned)(p < 256 ? 256 : p)), 0, s, a);
        }
    };
    const int w = a.H;
    if (ODD && w < 8) go(k_block_norm<2, 16, 1>, 16);
    else if (w <= 128) go(k_block_norm<ODD, 16, 1>, 16);
    else if (w <= 512) go(k_block_norm<ODD, 64, 1>, 64);
    else if (w <= 1024) go(k_block_norm<ODD, 64, 2>, 64);
    else if (w <= 2048) go(k_block_norm<ODD, 256, 1>, 256);
    else if (w <= 4096) go(k_block_norm<ODD, 256, 2>, 256);
    else if (w <= 8192) go(k_block_norm<ODD, 512, 2>, 512);
    else go(k_block_norm<ODD, 1024, 2>, 1024);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t s) {
    // rows whose chunks are all whole and aligned
    bool even = a.H % 8 == 0;
    auto check = [&](const void *p, int dt, int64_t ld) {
        if (p && ((uintptr_t)p % 16 || (a.T > 1 && ld * (dt == MOE_F32 ? 4 : 2) % 16))) even = false;
    };
    check(a.y, a.dy, a.ldy);
    check(a.r, a.dr, a.ldr);
    check(a.ro, a.dro, a.ldro);
    check(a.xo, a.dxo, a.ldxo);
    if (even) launch_p<0>(a, s);
    else launch_p<1>(a, s);
    return hipGetLastError();
}

}  // namespace qs
