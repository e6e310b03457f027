// lora.hip -- low-rank adapters of many requests beside a shared projection (lora_gemm):
//     y[t] = base[t] + scale_a B_a (A_a x_t),  a = ids[t]     (y[t] = base[t] without an adapter)
// Two launches over tiles of 16 tokens on v_mfma_f32_16x16x32_bf16 (one for up to 16 tokens, where A is small; a
// batch of many requests is ordered by adapter first):
//
//   shrink  v = scale_a A_a x_t, summed in fp32 over the columns, which the waves of a workgroup share.  v is kept
//           as a sum of bf16 parts (two, or three where y is fp32: v to 2^-16 or 2^-24), one behind the
//           other, so that the second product runs on the same instruction.
//   expand  y = base + B_a v, each part of v against the same rows of B in registers.
//
// A tile's tokens need not share an adapter: its distinct ones are taken one after another, each against
// all 16 rows of the tile, and a token keeps the result of its own (few tokens: by workgroups of their
// own, "slots").  A token's result depends on its own row only, bit for bit.
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));
// rows of y and base may lie at any alignment of their values
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef bf16x8 __attribute__((aligned(2))) bf16x8_any;

// lane n < 16 of every 16 holds token n's adapter (-1: none) and its place among the tile's distinct
// ones, which are numbered in token order
struct TileIds {
    int id, ord;
    uint32_t first;                                          // bit n: token n is its adapter's first
    __device__ __forceinline__ void set(int of_token, int n_adapters) {
        const int n = threadIdx.x & 15;
        id = of_token < 0 || of_token >= n_adapters ? -1 : of_token;
        int lead = n;
        if (__ballot(id != __builtin_amdgcn_readfirstlane(id)) == 0) {
            lead = 0;                                        // (a request's tokens)
        } else {
#pragma unroll
            for (int j = 14; j >= 0; --j) lead = j < n && __builtin_amdgcn_readlane(id, j) == id ? j : lead;
        }
        first = (uint32_t)__ballot(id >= 0 && lead == n) & 0xffffu;
        ord = id < 0 ? 0 : __popc(first & ((1u << lead) - 1u));
    }
    __device__ __forceinline__ int adapter(uint32_t m) const { return __builtin_amdgcn_readlane(id, __builtin_ctz(m)); }
};

__device__ __forceinline__ int rank_of(const LoraArgs &a, int ad) {
    return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

// --------------------------------------------------------------------------- order
// The tokens of a batch of many requests, ordered by adapter (those without one last), so that tiles
// hold few distinct ones: perm[i] is the i-th token, sid[i] its adapter.  Tokens that come in runs already (at
// most one change in four tiles) stay as they are.  A counting sort by one workgroup; the order within an
// adapter is not fixed and changes no result.
// us of a call (K = 2048, N = 16384) with and without: 8 mixed adapters of rank 32, T = 4096 94 and 240, of rank 64
// 130 and 559; 40 of rank 64, T = 256 44 and 95; packed prompts, which need none, 90 and 84.  N = 2048, rank 16:
// T = 4096 30 and 61, T = 512 19 and 16, so the rule (lora_ordered) goes by the bytes of B a tile reads.
constexpr int OR_THREADS = 1024, OR_BINS = 8192;             // (more adapters share bins: any order will do)

__global__ __launch_bounds__(OR_THREADS) void k_lora_order(LoraArgs a) {
    __shared__ int bins[OR_BINS + 1];
    __shared__ int wsum[OR_THREADS / 64], changes;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, T = (int)a.T;
    const int nb = min(a.n, OR_BINS) + 1;
    auto bin = [&](int id) { return id < 0 || id >= a.n ? nb - 1 : a.n <= OR_BINS ? id : id % OR_BINS; };
    if (tid == 0) changes = 0;
    for (int i = tid; i < nb; i += OR_THREADS) bins[i] = 0;
    __syncthreads();
    // (whole waves go through the loops: every lane takes part in the ballots)
    int mine = 0;
    for (int t0 = wave * 64; t0 < T; t0 += OR_THREADS) {
        const int t = t0 + lane, id = a.ids[min(t, T - 1)], b = bin(id);
        const bool in = t < T;
        mine += __popcll(__ballot(in && t > 0 && a.ids[max(min(t, T - 1) - 1, 0)] != id));
        const int tokens = __popcll(__ballot(in));
        if (__ballot(in && b != __builtin_amdgcn_readfirstlane(b)) == 0) {
            if (lane == 0) atomicAdd(&bins[b], tokens);      // (one bin: one addition)
        } else if (in) {
            atomicAdd(&bins[b], 1);
        }
    }
    if (lane == 0) atomicAdd(&changes, mine);
    __syncthreads();
    if (changes * 64 <= T) {
        for (int t = tid; t < T; t += OR_THREADS) {
            a.perm[t] = t;
            a.sid[t] = a.ids[t];
        }
        return;
    }
    // first places of the bins
    const int per = (nb + OR_THREADS - 1) / OR_THREADS, b0 = min(tid * per, nb), b1 = min(b0 + per, nb);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += bins[b];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o, 64);
        if (lane >= o) incl += v;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < wave; ++w) at += wsum[w];
    for (int b = b0; b < b1; ++b) {
        const int n = bins[b];
        bins[b] = at;
        at += n;
    }
    __syncthreads();
    for (int t = tid; t < T; t += OR_THREADS) {
        const int id = a.ids[t], p = atomicAdd(&bins[bin(id)], 1);
        a.perm[p] = t;
        a.sid[p] = id;
    }
}

// -------------------------------------------------------------------------- shrink
// Ranks r0 .. r0 + 16 RB - 1 of v for the tokens of a tile that have adapter ad, by a whole workgroup: its
// waves share the columns, SU steps of 32 loaded at a time.  tok: the token of lane % 16 (past the last: any); v0:
// v of the tile's first, [16][PARTS][R].
// Ends with a barrier.
constexpr int SH_WAVES = 8;

template <int RB, int SU, int PARTS>
__device__ __forceinline__ void shrink(const LoraArgs &a, const TileIds &tile, int ad, int rank, int64_t tok, int r0,
                                       f32x4 (*red)[RB][64], uint16_t *v0) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int K = a.K, R = a.R, steps = (K + 31) / 32;
    const uint16_t *xr = a.x + tok * a.ldx, *ar = a.a + (int64_t)ad * R * K;
    f32x4 acc[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave; s0 < steps; s0 += SU * SH_WAVES) {
        u32x4 A[SU], B[SU][RB];
#pragma unroll
        for (int u = 0; u < SU; ++u) {
            const int c = 32 * (s0 + u * SH_WAVES) + 8 * g;
            A[u] = (u32x4){0u, 0u, 0u, 0u};
            if (c < K) A[u] = *(const u32x4 *)(xr + c);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int r = r0 + 16 * i + n;
                B[u][i] = (u32x4){0u, 0u, 0u, 0u};
                if (c < K && r < rank) B[u][i] = *(const u32x4 *)(ar + (int64_t)r * K + c);
            }
        }
#pragma unroll
        for (int u = 0; u < SU; ++u)
#pragma unroll
            for (int i = 0; i < RB; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[u]),
                                                                 __builtin_bit_cast(bf16x8, B[u][i]), acc[i], 0, 0, 0);
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
        uint16_t *d = v0 + tk * PARTS * R + r;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            uint16_t h = f32_to_bf16(v);
            // (past bf16's largest value, within fp32's: that value, and the rest in the next part)
            if (p == 0 && __builtin_isfinite(v) && (h & 0x7fff) == 0x7f80) --h;
            d[p * R] = h;
            v = __builtin_isfinite(v) ? v - bf16_to_f32(h) : 0.0f;
        }
    }
    __syncthreads();
}

// One workgroup per (tile, 16 RB ranks, slot): the slot-th, slot + slots-th .. distinct adapters of the
// tile.
template <int RB, int SU, int PARTS>
__global__ __launch_bounds__(64 * SH_WAVES) void k_lora_shrink(LoraArgs a) {
    __shared__ f32x4 red[SH_WAVES][RB][64];
    const int64_t t0 = (int64_t)blockIdx.x * 16, p = min(t0 + (threadIdx.x & 15), a.T - 1);
    const int64_t tok = a.perm ? a.perm[p] : p;
    TileIds tile;
    tile.set(t0 + (threadIdx.x & 15) < a.T ? (a.perm ? a.sid : a.ids)[p] : -1, a.n);
    for (uint32_t m = tile.first, k = 0; m; m &= m - 1, ++k) {
        if (k % gridDim.z != blockIdx.z) continue;
        const int ad = tile.adapter(m);
        shrink<RB, SU, PARTS>(a, tile, ad, rank_of(a, ad), tok, blockIdx.y * 16 * RB, red, a.v + t0 * PARTS * a.R);
    }
}

// -------------------------------------------------------------------------- expand
// A wave takes 64 columns of y for `tt` tiles of tokens, and keeps an adapter's rows of B (RS steps of 32
// ranks) in registers until a tile has another.  The weights are the first operand, so that a
// lane's registers are columns of one token (lane % 16): operand row n of product i is column
// 16 i + n of the 64 (fp32 y: 16 bytes a register quad), or 32 (i / 2) + 8 (n / 4) + 4 (i % 2) + n % 4 (bf16: two
// quads make 16 bytes), so that four lanes read and write 64 bytes in a row.
//
// Bound by memory: y read and written, each request's rows of B. T = 4096 x 16384, rank 32: 63 us, 268 MB of y at 4.2 TB/s
// (shrink 11); columns before tiles in the grid, so that neighbouring workgroups write neighbouring
// columns (the other way 80 us); the next tile's loads ahead of this one's products gain nothing
// (four waves a SIMD hide them, and spill fewer registers).
// Rows of any stride and alignment are read and written by 16 bytes as they lie.  TAIL: a width that is no
// multiple of 64, whose last columns go value by value (N = 16381 160 us, all of them so 287; fp32 y, N = 8191 126 and
// 268, three waves a SIMD, for four would spill: 136); the code for them costs the other widths 0.1 to
// 0.4 us of a call of few tokens, so they have kernels without it.
//
// FEW > 0: up to 16 tokens of up to 16 FEW ranks in one launch; every workgroup (of SH_WAVES) shrinks for
// itself, v stays in LDS.  us a call in a graph against two launches (K = 2048): T = 1, N = 2048, rank 16
// 6.8 and 9.1, rank 32 8.7 and 9.3, T = 16 with 8 adapters 8.7 and 11.3, T = 1, N = 16384, rank 16 7.0 and 9.2;
// ranks of 64 in turns of 32 9.8 and 9.2, so they take two launches, as do calls whose workgroups would read A
// too often (T = 16, N = 16384, 16 adapters: 15.0 and 14.6).
constexpr int EX_WAVES = 4;

template <int PARTS, bool F32, bool TAIL, int RS, int FEW = 0>
__global__ __launch_bounds__(64 * (FEW ? SH_WAVES : EX_WAVES))
    __attribute__((amdgpu_waves_per_eu(FEW ? 2 : RS == 1 && !(F32 && TAIL) ? 4 : RS <= 2 ? 3 : 2))) void k_lora_expand(LoraArgs a, int tt) {
    __shared__ f32x4 red[FEW ? SH_WAVES : 1][FEW ? FEW : 1][64];
    extern __shared__ __attribute__((aligned(16))) uint16_t few_v[];     // [16][PARTS][R]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int R = a.R, slot = blockIdx.z, slots = gridDim.z;
    const int64_t c0 = ((int64_t)blockIdx.x * (FEW ? SH_WAVES : EX_WAVES) + wave) * 64, N = a.N;
    if (!FEW && c0 >= N) return;
    const bool whole = c0 + (TAIL ? 64 : 1) <= N;            // (FEW: the last waves may have no columns)
    auto column = [&](int i, int row) { return c0 + (F32 ? 16 * i + row : 32 * (i >> 1) + 8 * (row >> 2) + 4 * (i & 1) + (row & 3)); };
    u32x4 B[RS][4];
    int held = -1, rank = 0;
    auto load_b = [&](int ad, int s0) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r8 = 32 * (s0 + s) + 8 * g;
                const int64_t c = column(i, n);
                B[s][i] = (u32x4){0u, 0u, 0u, 0u};
                if (c < N && r8 < rank) B[s][i] = *(const u32x4 *)(a.b + ((int64_t)ad * N + c) * R + r8);
            }
        if (rank & 7)                                        // (past the rank: anything)
#pragma unroll
            for (int s = 0; s < RS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 32 * (s0 + s) + 8 * g + 2 * j;
                        if (r >= rank) B[s][i][j] = 0u;
                        else if (r + 1 >= rank) B[s][i][j] &= 0xffffu;
                    }
    };
    const int64_t tiles = (a.T + 15) / 16, last = min((int64_t)(blockIdx.y + 1) * tt, tiles);
    // a tile's tokens and their adapters, read a tile ahead
    const int32_t *ids = a.perm ? a.sid : a.ids;
    int64_t p1 = min((int64_t)blockIdx.y * tt * 16 + n, a.T - 1);
    int t1 = a.perm ? a.perm[p1] : (int)p1, id1 = ids[p1];
    for (int64_t ti = (int64_t)blockIdx.y * tt; ti < last; ++ti) {
        const int64_t p = p1, t = t1;                        // place, token
        TileIds tile;
        tile.set(ti * 16 + n < a.T ? id1 : -1, a.n);
        if (ti + 1 < last) {
            p1 = min(p1 + 16, a.T - 1);
            t1 = a.perm ? a.perm[p1] : (int)p1;
            id1 = ids[p1];
        }
        // rows of this slot; in place, rows without an adapter stay
        const bool live = ti * 16 + n < a.T && tile.ord % slots == slot && (tile.id >= 0 || a.base != a.y);
        // (-0, which leaves every value of base as it is: rows without an adapter)
        f32x4 out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = (f32x4){-0.f, -0.f, -0.f, -0.f};
        // base, as its register quads
        u32x4 raw[F32 ? 4 : 2];
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) {
            raw[i] = (u32x4){0u, 0u, 0u, 0u};
            const int64_t c = column(F32 ? i : 2 * i, 4 * g);
            if (a.base && live && whole)
                raw[i] = F32 ? *(const u32x4_any *)((const float *)a.base + t * a.ldb + c)
                             : *(const u32x4_any *)((const uint16_t *)a.base + t * a.ldb + c);
        }
        for (uint32_t m = tile.first, k = 0; m; m &= m - 1, ++k) {
            if ((int)k % slots != slot) continue;
            const int ad = tile.adapter(m);
            const bool mine = tile.id == ad;
            if (ad != held) rank = rank_of(a, ad);
            f32x4 acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if constexpr (FEW > 0) {
                load_b(ad, 0);                               // (under the first product)
                shrink<FEW, 8 / FEW, PARTS>(a, tile, ad, rank, t, 0, red, few_v);
            }
            const uint16_t *vr = FEW ? few_v + n * PARTS * R : a.v + p * PARTS * R;
            for (int s0 = 0; 32 * s0 < rank; s0 += RS) {
                u32x4 V[RS][PARTS];
#pragma unroll
                for (int s = 0; s < RS; ++s)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const int r8 = 32 * (s0 + s) + 8 * g;
                        V[s][p] = (u32x4){0u, 0u, 0u, 0u};
                        if (mine && r8 < rank) V[s][p] = *(const u32x4 *)(vr + p * R + r8);
                    }
                if (!FEW && (ad != held || R > 32 * RS)) load_b(ad, s0);
#pragma unroll
                for (int s = 0; s < RS; ++s)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, B[s][i]),
                                                                             __builtin_bit_cast(bf16x8, V[s][p]), acc[i], 0, 0, 0);
            }
            held = ad;
            if constexpr (FEW > 0) __syncthreads();          // (v is read)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[i][r] = mine ? acc[i][r] : out[i][r];
        }
        if (!live) continue;
        if (whole) {
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t c = column(i, 4 * g);
                    *(f32x4_any *)((float *)a.y + t * a.ldy + c) = out[i] + __builtin_bit_cast(f32x4, raw[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t c = column(2 * i, 4 * g);
                    f32x8 w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[2 * j] = out[2 * i + (j >> 1)][2 * (j & 1)] + __uint_as_float(raw[i][j] << 16);
                        w[2 * j + 1] = out[2 * i + (j >> 1)][2 * (j & 1) + 1] + __uint_as_float(raw[i][j] & 0xffff0000u);
                    }
                    *(bf16x8_any *)((uint16_t *)a.y + t * a.ldy + c) = __builtin_convertvector(w, bf16x8);
                }
            }
        } else if constexpr (TAIL) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t c = column(i, 4 * g + r);
                    if (c >= N) continue;
                    float v = out[i][r];
                    if constexpr (F32) {
                        v += a.base ? ((const float *)a.base)[t * a.ldb + c] : 0.0f;
                        ((float *)a.y)[t * a.ldy + c] = v;
                    } else {
                        v += a.base ? bf16_to_f32(((const uint16_t *)a.base)[t * a.ldb + c]) : 0.0f;
                        ((uint16_t *)a.y)[t * a.ldy + c] = f32_to_bf16(v);
                    }
                }
        }
    }
}

// values of A: of one adapter, and of all workgroups together
constexpr int64_t FEW_A = 65536, FEW_ALL = 8 << 20;

template <int PARTS, bool F32, bool TAIL>
hipError_t launch_parts(const LoraArgs &a, hipStream_t s) {
    const int64_t tiles = (a.T + 15) / 16, rblk = (a.R + 15) / 16, cus = n_compute_units();
    // a tile's distinct adapters, at most; workgroups of their own until two a compute unit (T = 48 with 40
    // adapters of 16384 x 64: expand with 3 slots 21 us, with 6 23, with 11 25)
    const int64_t most = a.T < 16 ? (a.T < a.n ? a.T : a.n) : (a.n < 16 ? a.n : 16);
    auto slots = [&](int64_t groups) {
        int64_t k = (2 * cus + groups - 1) / groups;
        return (unsigned)(k < most ? k : most);
    };
    // Up to 16 tokens in one launch where the workgroups' reading of A, each for itself, is little
    const int64_t fblk = (a.N + 64 * SH_WAVES - 1) / (64 * SH_WAVES);
    if (tiles == 1 && a.R <= 32 && (int64_t)a.R * a.K <= FEW_A && fblk * most * a.R * a.K <= FEW_ALL) {
        const size_t lds = (size_t)16 * PARTS * a.R * 2;
        void (*k)(LoraArgs, int) = rblk == 1 ? k_lora_expand<PARTS, F32, TAIL, 1, 1> : k_lora_expand<PARTS, F32, TAIL, 1, 2>;
        hipLaunchKernelGGL(k, dim3((unsigned)fblk, 1, (unsigned)most), dim3(64 * SH_WAVES), lds, s, a, 1);
        return hipGetLastError();
    }
    if (a.perm) {
        hipLaunchKernelGGL(k_lora_order, dim3(1), dim3(OR_THREADS), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int rb = tiles >= cus && rblk >= 4 ? 4 : tiles >= cus && rblk >= 2 ? 2 : 1;
    const unsigned ry = (unsigned)((rblk + rb - 1) / rb);
    const dim3 sg((unsigned)tiles, ry, slots(tiles * ry));
    if (rb == 4) hipLaunchKernelGGL((k_lora_shrink<4, 2, PARTS>), sg, dim3(64 * SH_WAVES), 0, s, a);
    else if (rb == 2) hipLaunchKernelGGL((k_lora_shrink<2, 4, PARTS>), sg, dim3(64 * SH_WAVES), 0, s, a);
    else hipLaunchKernelGGL((k_lora_shrink<1, 8, PARTS>), sg, dim3(64 * SH_WAVES), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;

    const int64_t cblk = (a.N + 64 * EX_WAVES - 1) / (64 * EX_WAVES);
    int tt = 8;                                              // tiles a wave: while eight workgroups a compute unit remain
    while (tt > 1 && (tiles + tt - 1) / tt * cblk < 8 * cus) tt >>= 1;
    const unsigned tx = (unsigned)((tiles + tt - 1) / tt);
    const dim3 eg((unsigned)cblk, tx, slots((int64_t)tx * cblk));
    void (*k)(LoraArgs, int) = a.R <= 32   ? k_lora_expand<PARTS, F32, TAIL, 1>
                               : a.R <= 64 ? k_lora_expand<PARTS, F32, TAIL, 2>
                                           : k_lora_expand<PARTS, F32, TAIL, 4>;
    hipLaunchKernelGGL(k, eg, dim3(64 * EX_WAVES), 0, s, a, tt);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, hipStream_t s) {
    if (a.f32) return a.N % 64 ? launch_parts<3, true, true>(a, s) : launch_parts<3, true, false>(a, s);
    return a.N % 64 ? launch_parts<2, false, true>(a, s) : launch_parts<2, false, false>(a, s);
}

}  // namespace qs
