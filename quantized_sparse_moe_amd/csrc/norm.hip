// norm.hip -- the norms around a block (moe_block_norm), one pass over a row:
//     z = act(gate) * post(y)      r' = r + scale * z      x = pre(r')
// with each part optional.  A norm is v -> (v / sqrt(mean v^2 + eps)) (offset + w) + b, or the same of
// v - mean v.
//
// Bound by memory: y, r and an elementwise gate read once, r' and x written once.  A row stays in the
// registers of the P threads that read it, 8 V values each, from its first load to its last
// store, and every load of a row (the weights' too) is under way before the first sum.  Sums, norms and the stream are
// fp32 (r' enters the second norm unrounded, whatever type it is stored in); only the two results are
// rounded.  The mean square is taken after the mean is subtracted, from registers.
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// 8 V values of a row as a thread holds them: V chunks of 8 neighbours, P chunks apart (VEC), or
// values P apart (rows that are not 16-byte aligned, or whose length is no multiple of 8).
template <bool VEC, int P, int V>
struct Row {
    static __device__ __forceinline__ int at(int t, int i, int j) { return VEC ? (t + P * i) * 8 + j : t + P * (8 * i + j); }
};

// loaded and not yet widened
template <bool VEC, int V>
struct Raw {
    u32x4 q[V][2];
};

template <bool VEC, int P, int V>
__device__ __forceinline__ void load_row(Raw<VEC, V> &w, const void *p, int dt, int64_t off, int t, int H) {
    if constexpr (VEC) {
        if (dt == MOE_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((t + P * i) * 8 < H) {
                    const u32x4 *s = (const u32x4 *)((const float *)p + off + (t + P * i) * 8);
                    w.q[i][0] = s[0];
                    w.q[i][1] = s[1];
                }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((t + P * i) * 8 < H) w.q[i][0] = *(const u32x4 *)((const uint16_t *)p + off + (t + P * i) * 8);
        }
    } else {
        // (past the row's end: its last value, not used)
        if (dt == MOE_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w.q[i][j >> 2][j & 3] = ((const uint32_t *)p)[off + min(Row<VEC, P, V>::at(t, i, j), H - 1)];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w.q[i][j >> 2][j & 3] = ((const uint16_t *)p)[off + min(Row<VEC, P, V>::at(t, i, j), H - 1)];
        }
    }
}

// the values (VEC: two 16-bit ones a word; else one a word)
template <bool VEC, int V>
__device__ __forceinline__ float value(const Raw<VEC, V> &w, int dt, int i, int j) {
    if (dt == MOE_F32) return __uint_as_float(w.q[i][j >> 2][j & 3]);
    uint32_t u;
    if constexpr (VEC) u = (j & 1) ? w.q[i][0][j >> 1] >> 16 : w.q[i][0][j >> 1] & 0xffffu;
    else u = w.q[i][j >> 2][j & 3];
    return dt == MOE_BF16 ? __uint_as_float(u << 16) : f16_to_f32((uint16_t)u);
}
template <bool VEC, int V>
__device__ __forceinline__ void widen(const Raw<VEC, V> &w, int dt, float (&f)[V][8]) {
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

template <bool VEC, int P, int V>
__device__ __forceinline__ void store_row(void *p, int dt, int64_t off, int t, int H, const float (&f)[V][8]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (VEC) {
            if ((t + P * i) * 8 >= H) continue;
            const int64_t o = off + (t + P * i) * 8;
            if (dt == MOE_F32) {
                f32x4 *d = (f32x4 *)((float *)p + o);
                d[0] = (f32x4){f[i][0], f[i][1], f[i][2], f[i][3]};
                d[1] = (f32x4){f[i][4], f[i][5], f[i][6], f[i][7]};
                continue;
            }
            const f32x8 v = {f[i][0], f[i][1], f[i][2], f[i][3], f[i][4], f[i][5], f[i][6], f[i][7]};
            *(u32x4 *)((uint16_t *)p + o) = dt == MOE_BF16 ? __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8v))
                                                           : __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = Row<VEC, P, V>::at(t, i, j);
                if (c >= H) continue;
                if (dt == MOE_F32) ((float *)p)[off + c] = f[i][j];
                else if (dt == MOE_BF16) ((uint16_t *)p)[off + c] = f32_to_bf16(f[i][j]);
                else ((_Float16 *)p)[off + c] = (_Float16)f[i][j];
            }
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

// values past the row's end to 0
template <bool VEC, int P, int V>
__device__ __forceinline__ void mask_row(float (&f)[V][8], int t, int H) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = Row<VEC, P, V>::at(t, i, j) < H ? f[i][j] : 0.0f;
}

// f -> its norm (values past the row's end are 0 before and not used after)
template <bool VEC, int P, int V>
__device__ __forceinline__ void norm_row(float (&f)[V][8], const NormArgs &n, int t, int H, int slot) {
    Raw<VEC, V> w{}, b{};
    if (n.w) load_row<VEC, P, V>(w, n.w, n.dtype, 0, t, H);
    if (n.b) load_row<VEC, P, V>(b, n.b, n.dtype, 0, t, H);
    const float ih = 1.0f / (float)H;
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
            for (int j = 0; j < 8; ++j) f[i][j] = Row<VEC, P, V>::at(t, i, j) < H ? f[i][j] - m : 0.0f;
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

template <bool VEC, int P, int V>
__global__ __launch_bounds__(P < 256 ? 256 : P) void k_block_norm(BlockNormArgs a) {
    constexpr int RPW = P < 256 ? 256 / P : 1;               // rows per workgroup
    const int t = threadIdx.x % P, H = a.H;
    const int64_t row = a.row0 + (int64_t)blockIdx.x * RPW + threadIdx.x / P;
    if (row >= a.T) return;                                  // (whole rows; P > 64: never)
    Raw<VEC, V> y{}, r{}, g{};
    if (a.y) load_row<VEC, P, V>(y, a.y, a.dy, row * a.ldy, t, H);
    if (a.r) load_row<VEC, P, V>(r, a.r, a.dr, row * a.ldr, t, H);
    if (a.gate && a.gate_cols > 1) load_row<VEC, P, V>(g, a.gate, a.dg, row * a.ldg, t, H);
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
            if constexpr (!VEC) mask_row<VEC, P, V>(z, t, H);
            norm_row<VEC, P, V>(z, a.post, t, H, 0);
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
        if (a.ro) store_row<VEC, P, V>(a.ro, a.dro, row * a.ldro, t, H, z);
    } else {
        widen(r, a.dr, z);
    }
    if (a.pre.on) {
        mask_row<VEC, P, V>(z, t, H);
        norm_row<VEC, P, V>(z, a.pre, t, H, 2);
        store_row<VEC, P, V>(a.xo, a.dxo, row * a.ldxo, t, H, z);
    }
}

// Threads per row: 8 values each while a row has up to 512 or 1025 to 2048 of them, 16 up to 16384, in us for
// both norms of bf16 rows (TB/s):
//   16384 x 2048  256 threads 46.0 (5.83), 64 threads of 32 values 56.9      131072 x 1024  64 of 16: 183.4 (5.85)
//   16384 x 4096  256 of 16: 95.9 (5.60), 512 of 8: 96.0                     131072 x 512   64 of 8: 93.9 (5.72)
//   16384 x 8192  512 of 16: 210 (5.11), 256 of 32: 214, 1024 of 8: 266      8192 x 16384   1024 of 16: 224 (4.80)
//   (with a gate: 266 (5.05), 291, 370; a large copy moves 4.8)
template <bool VEC>
void launch_p(BlockNormArgs a, hipStream_t s) {
    // (a launch has fewer than 2^32 threads)
    auto go = [&](void (*k)(BlockNormArgs), int p) {
        const int64_t rpw = p < 256 ? 256 / p : 1, most = ((int64_t)1 << 31) / p;
        for (a.row0 = 0; a.row0 < a.T; a.row0 += most) {
            const int64_t rows = a.T - a.row0 < most ? a.T - a.row0 : most;
            hipLaunchKernelGGL(k, dim3((unsigned)((rows + rpw - 1) / rpw)), dim3((unsigned)(p < 256 ? 256 : p)), 0, s, a);
        }
    };
    if (a.H <= 128) go(k_block_norm<VEC, 16, 1>, 16);
    else if (a.H <= 512) go(k_block_norm<VEC, 64, 1>, 64);
    else if (a.H <= 1024) go(k_block_norm<VEC, 64, 2>, 64);
    else if (a.H <= 2048) go(k_block_norm<VEC, 256, 1>, 256);
    else if (a.H <= 4096) go(k_block_norm<VEC, 256, 2>, 256);
    else if (a.H <= 8192) go(k_block_norm<VEC, 512, 2>, 512);
    else if (a.H <= 16384) go(k_block_norm<VEC, 1024, 2>, 1024);
    else go(k_block_norm<VEC, 1024, 4>, 1024);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t s) {
    // 16-byte accesses where every row of every tensor allows them
    bool vec = a.H % 8 == 0;
    auto check = [&](const void *p, int dt, int64_t ld) {
        if (p && ((uintptr_t)p % 16 || (a.T > 1 && ld * (dt == MOE_F32 ? 4 : 2) % 16))) vec = false;
    };
    check(a.y, a.dy, a.ldy);
    check(a.r, a.dr, a.ldr);
    if (a.gate_cols > 1) check(a.gate, a.dg, a.ldg);
    check(a.ro, a.dro, a.ldro);
    check(a.xo, a.dxo, a.ldxo);
    for (const NormArgs *n : {&a.post, &a.pre}) {
        check(n->w, n->dtype, 0);
        check(n->b, n->dtype, 0);
    }
    if (vec) launch_p<true>(a, s);
    else launch_p<false>(a, s);
    return hipGetLastError();
}

}  // namespace qs
