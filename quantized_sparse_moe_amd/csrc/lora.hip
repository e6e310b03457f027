// lora.hip -- low-rank adapters of many requests beside a shared projection (lora_gemm):
//     y[t] = base[t] + scale_a B_a (A_a x_t),  a = ids[t]     (y[t] = base[t] without an adapter)
// Two launches over tiles of 16 tokens on v_mfma_f32_16x16x32_bf16:
//
//   shrink  v = scale_a A_a x_t, summed in fp32 over the columns, which the waves of a workgroup share.  v is kept
//           as a sum of bf16 parts (two, or three where y is fp32: v to 2^-16 or 2^-24), one behind the
//           other, so that the second product runs on the same instruction.
//   expand  y = base + B_a v over those parts, each against the same rows of B.
//
// A tile's tokens need not share an adapter: its distinct ones are taken one after another, each against
// all 16 rows of the tile, and a token keeps the result of its own.  A token's result depends on its own
// row only, bit for bit.
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

// lane n < 16 of every 16 holds token n's adapter (-1: none); the distinct ones in token order
struct TileIds {
    int id;                                                  // of token lane % 16
    uint32_t first;                                          // bit n: token n is its adapter's first
    __device__ __forceinline__ void load(const int32_t *ids, int64_t t0, int64_t T, int n_adapters) {
        const int n = threadIdx.x & 15;
        id = t0 + n < T ? ids[t0 + n] : -1;
        if (id < 0 || id >= n_adapters) id = -1;
        bool dup = id < 0;
#pragma unroll
        for (int j = 0; j < 15; ++j) dup |= j < n && __builtin_amdgcn_readlane(id, j) == id;
        first = (uint32_t)__ballot(!dup) & 0xffffu;
    }
};

__device__ __forceinline__ int rank_of(const LoraArgs &a, int ad) {
    return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

// -------------------------------------------------------------------------- shrink
// One workgroup per (tile, 16 RB ranks, slot): the slot-th, slot + slots-th .. distinct adapters of the
// tile.
constexpr int SH_WAVES = 8;

template <int RB, int PARTS>
__global__ __launch_bounds__(64 * SH_WAVES) void k_lora_shrink(LoraArgs a) {
    __shared__ f32x4 red[SH_WAVES][RB][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    TileIds tile;
    tile.load(a.ids, t0, a.T, a.n);
    const int K = a.K, R = a.R, steps = (K + 31) / 32, r0 = blockIdx.y * 16 * RB;
    const uint16_t *xr = a.x + min(t0 + n, a.T - 1) * a.ldx;
    int k = 0;
    for (uint32_t m = tile.first; m; m &= m - 1, ++k) {
        if (k % (int)gridDim.z != (int)blockIdx.z) continue;
        const int ad = __builtin_amdgcn_readlane(tile.id, __builtin_ctz(m)), rank = rank_of(a, ad);
        f32x4 acc[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        const uint16_t *ar = a.a + (int64_t)ad * R * K;
        for (int s = wave; s < steps; s += SH_WAVES) {
            const int c = 32 * s + 8 * g;
            u32x4 A = {0u, 0u, 0u, 0u};
            if (c < K) A = *(const u32x4 *)(xr + c);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int r = r0 + 16 * i + n;
                u32x4 B = {0u, 0u, 0u, 0u};
                if (c < K && r < rank) B = *(const u32x4 *)(ar + (int64_t)r * K + c);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A), __builtin_bit_cast(bf16x8, B),
                                                                 acc[i], 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        // thread: a token and a rank
        for (int i = tid; i < 256 * RB; i += 64 * SH_WAVES) {
            const int rr = i & 15, tk = (i >> 4) & 15, b = i >> 8, l = rr + 16 * (tk >> 2), r = r0 + 16 * b + rr;
            const bool mine = __shfl(tile.id, tk, 64) == ad;
            if (!mine || r >= R) continue;
            float v = red[0][b][l][tk & 3];
#pragma unroll
            for (int w = 1; w < SH_WAVES; ++w) v += red[w][b][l][tk & 3];
            if (a.scales) v *= a.scales[ad];
            if (r >= rank) v = 0.0f;
            uint16_t *d = a.v + (t0 + tk) * PARTS * R + r;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const uint16_t h = f32_to_bf16(v);
                d[p * R] = h;
                v = __builtin_isfinite(v) ? v - bf16_to_f32(h) : 0.0f;
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------------- expand
// A wave takes 64 columns of y: lane n + 16 g holds the 16 columns 16 g .. + 15 of them for token n
// (operand row i of product m is column 16 (i / 4) + 4 m + i % 4 of B).
constexpr int EX_WAVES = 4;

template <int PARTS, bool F32>
__global__ __launch_bounds__(64 * EX_WAVES) void k_lora_expand(LoraArgs a) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    TileIds tile;
    tile.load(a.ids, t0, a.T, a.n);
    const int R = a.R, R8 = R / 8, steps = (PARTS * R8 + 3) / 4;
    const int64_t c0 = ((int64_t)blockIdx.y * EX_WAVES + wave) * 64, N = a.N, t = t0 + n;
    if (c0 >= N) return;
    float out[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = 0.0f;
    const int slot = blockIdx.z, slots = gridDim.z;
    bool have = slot == 0 && tile.id < 0;                    // (tokens without an adapter: the first slot's)
    int k = 0;
    for (uint32_t m = tile.first; m; m &= m - 1, ++k) {
        if (k % slots != slot) continue;
        const int ad = __builtin_amdgcn_readlane(tile.id, __builtin_ctz(m)), rank = rank_of(a, ad);
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        const bool mine = tile.id == ad;
        const uint16_t *vr = a.v + t * PARTS * R;
        for (int s = 0; s < steps; ++s) {
            const int q = 4 * s + g, r8 = 8 * (q % R8);      // 8 ranks of a part
            u32x4 V = {0u, 0u, 0u, 0u};
            if (mine && q < PARTS * R8) V = *(const u32x4 *)(vr + 8 * q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t c = c0 + 16 * (n >> 2) + 4 * i + (n & 3);
                u32x4 B = {0u, 0u, 0u, 0u};
                if (c < N && q < PARTS * R8 && r8 < rank) {
                    B = *(const u32x4 *)(a.b + ((int64_t)ad * N + c) * R + r8);
                    if (r8 + 8 > rank)                       // (past the rank: anything)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (r8 + 2 * j >= rank) B[j] = 0u;
                            else if (r8 + 2 * j + 1 >= rank) B[j] &= 0xffffu;
                        }
                }
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, B), __builtin_bit_cast(bf16x8, V),
                                                                 acc[i], 0, 0, 0);
            }
        }
        if (mine) {
            have = true;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[4 * i + r] = acc[i][r];
        }
    }
    if (!have || t >= a.T) return;
    if (tile.id < 0 && a.base == a.y) return;                // (in place: nothing to add)
    const int64_t c = c0 + 16 * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (c + i >= N) break;
        if constexpr (F32) {
            float v = out[i];
            if (a.base) v += ((const float *)a.base)[t * a.ldb + c + i];
            ((float *)a.y)[t * a.ldy + c + i] = v;
        } else {
            float v = out[i];
            if (a.base) v += bf16_to_f32(((const uint16_t *)a.base)[t * a.ldb + c + i]);
            ((uint16_t *)a.y)[t * a.ldy + c + i] = f32_to_bf16(v);
        }
    }
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, hipStream_t s) {
    const unsigned tiles = (unsigned)((a.T + 15) / 16);
    const dim3 sg(tiles, (unsigned)((a.R + 15) / 16), 1), eg(tiles, (unsigned)((a.N + 64 * EX_WAVES - 1) / (64 * EX_WAVES)), 1);
    if (a.f32) hipLaunchKernelGGL((k_lora_shrink<1, 3>), sg, dim3(64 * SH_WAVES), 0, s, a);
    else hipLaunchKernelGGL((k_lora_shrink<1, 2>), sg, dim3(64 * SH_WAVES), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.f32) hipLaunchKernelGGL((k_lora_expand<3, true>), eg, dim3(64 * EX_WAVES), 0, s, a);
    else hipLaunchKernelGGL((k_lora_expand<2, false>), eg, dim3(64 * EX_WAVES), 0, s, a);
    return hipGetLastError();
}

}  // namespace qs
