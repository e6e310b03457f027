// mx4_moe.hip -- the sparse MoE layer with MX4 experts for a few tokens (up to MX_TMAX a pass):
// three launches, two for up to four.
//
//   route    router logits on v_mfma_f32_16x16x32_bf16 (16 experts and 16 tokens per
//            workgroup, the columns split over its waves).  The workgroup that finishes a tile
//            of tokens last -- counted, so nothing ever waits -- takes their top-k, and the
//            last of those lists the experts any token chose (ascending) and each one's
//            tokens.
//   gate/up  one workgroup per (listed expert, 32 or 16 columns of h): gathers the expert's tokens
//            as the rows of the activation operand.  A list entry is up to 16 tokens of an
//            expert: an expert of more is loaded once for each of its entries, which run side by
//            side, so that the repeats come from the L2 (T = 128: 286 MB fetched past it for 281 MB of
//            weights), and an expert that one token chose costs one 16-row tile.  h = w silu(g) u carries the token's routing weight and leaves as the
//            bf16 pair hi + lo (h to 2^-17), two operand rows.
//   down     one workgroup per 32 rows of the output and share of the listed experts, gathering
//            each expert's rows of h; hi and lo of a token are neighbouring accumulator
//            registers and are added in the lane.  Shares are added in a fixed order by the
//            share that finishes last.
//
// One to four tokens take two: k_mx_token does route and gate/up.
//
// All are bound by the weight stream: (union of the chosen experts + shared), each once, x
// 3 H I x 17/32 bytes, and at few tokens by the chain of launches and round trips before and
// after it (2048 x 512, top 8 of 256 and a shared expert, times of the layer in a graph):
//   T = 1 15.9 us (15 MB: 2.4 at 6.3 TB/s)   T = 2 20.1   T = 4 26.4 (53 MB: 8)   T = 7 36.0 (89 MB: 14)
//   T = 20 61 (209 MB: 33)   T = 32 73 (272 MB: 43)   T = 64 92 (370 MB: 59)
//   T = 65 101   T = 128 123 (421 MB: 67)
//   under a skewed router T = 48 49 (52 experts), T = 128 82 (76 experts)
// From T = 7 on more experts cost 5.2 TB/s; about 20 us do not depend on them.  Of T = 7, route
// takes 9, gate/up 15, down 12.  Every sum is fp32 in a fixed order; there are no float atomics.
#include "decode_state.h"
#include "mx4.h"

namespace qs {

namespace {

constexpr int MT_THREADS = 512, MT_WAVES = 8;
constexpr int RT_THREADS = 1024, RT_WAVES = 16;
static_assert((TOPK_BASE + TOPK_COPIES * TOPK_STRIDE) * 4 <= (int)MX_CNT_OFF, "counters behind the decode state");
static_assert(MX_CNT_DOWN + 8192 / 16 <= 1024, "a counter per 16 output rows");

struct MxArgs {
    Layer L;
    MxBufs b;
    const uint16_t *x;
    int T;
    int gated;
    int route_only;
    int tagged;                       // route and gate/up ran as k_mx_token
    int32_t *out_idx;
    float *out_w;
    void *y;
    int y_dtype;
    int shares;                       // down: workgroups that share the items of the same output rows
};

__device__ __forceinline__ float ld_agent(const float *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// four times 16 bytes read at device scope, and waited for here (the compiler does not track
// loads issued from inline assembly)
__device__ __forceinline__ void ld_agent128x4(const float *p0, const float *p1, const float *p2, const float *p3,
                                              f32x4 &a, f32x4 &b, f32x4 &c, f32x4 &d) {
    asm volatile(
        "global_load_dwordx4 %0, %4, off sc1\n\t"
        "global_load_dwordx4 %1, %5, off sc1\n\t"
        "global_load_dwordx4 %2, %6, off sc1\n\t"
        "global_load_dwordx4 %3, %7, off sc1\n\t"
        "s_waitcnt vmcnt(0)"
        : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
        : "v"(p0), "v"(p1), "v"(p2), "v"(p3)
        : "memory");
}

// Whether this workgroup is the last of n to come here.  What it reads of the others' work they
// stored at device scope (written through), so the count only has to follow the stores'
// completion, and it reads at device scope.  The counter goes back to zero for the next call.
__device__ __forceinline__ bool last_of(uint32_t *cnt, uint32_t n, int *s_last) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // (every wave its own)
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        if (last) st_dev(cnt, 0u);
        *s_last = last;
    }
    __syncthreads();
    return *s_last != 0;
}

// An entry of the work list: up to 16 tokens of one expert, rows first .. first + count - 1 of
// its slot's list of tokens.
__device__ __forceinline__ int mx_item(int e, int slot, int tile, int count) {
    return e | slot << 8 | tile << 16 | count << 20;
}
struct MxItem {
    int e, list, count;                                      // expert, first entry of pos, tokens
};
// item i of a layer with nsh shared-expert items (16 tokens each) before the listed ones; act is
// the listed entry (not used for a shared item)
__device__ __forceinline__ MxItem mx_unpack(int i, int nsh, int act, int T) {
    if (i < nsh) return {0, -1, min(T - 16 * i, 16)};
    return {act & 255, (act >> 8 & 255) * MX_TMAX + 16 * (act >> 16 & 15), act >> 20};
}

// ---------------------------------------------------------------------------- route
// One workgroup per 16 experts (row E: the shared expert's gate) and 16 tokens, the columns
// split over its waves.  The workgroup that finishes a tile of 16 tokens last takes their
// top-k, a wave per token (one compute unit takes 4 us over 16 of them, so tiles do not wait
// for one another); the last of those lists the experts.
__global__ __launch_bounds__(RT_THREADS) void k_mx_route(MxArgs a) {
    __shared__ f32x4 red[RT_WAVES][64];
    __shared__ int s_last;
    __shared__ int s_slot[256], s_cnt[4], s_itm[4];
    constexpr int MW = MX_TMAX / 32;
    __shared__ uint32_t s_mask[256][MW];                     // tokens that chose the expert
    __shared__ int16_t s_sel[MX_TMAX * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, E = a.L.E, K = a.L.K, T = a.T, NE = E + a.gated;
    {
        const int e = blockIdx.x * 16 + n, ec = e < NE ? e : NE - 1, tr = blockIdx.y * 16 + n;
        const uint16_t *wr = ec < E ? a.L.router_w + (int64_t)ec * H : a.L.shared_gate_w;
        const uint16_t *xr = a.x + (int64_t)tr * H;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        const int steps = H / 32;
        for (int s0 = wave; s0 < steps; s0 += 4 * RT_WAVES) {
            u32x4 B[4], A[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = s0 + i * RT_WAVES, k = 32 * s + 8 * g;
                B[i] = A[i] = (u32x4){0u, 0u, 0u, 0u};
                if (s < steps) {
                    B[i] = *(const u32x4 *)(wr + k);
                    if (tr < T) A[i] = *(const u32x4 *)(xr + k);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[i]),
                                                              __builtin_bit_cast(bf16x8, B[i]), acc, 0, 0, 0);
        }
        red[wave][lane] = acc;
        __syncthreads();
        const int t = blockIdx.y * 16 + (tid >> 4), ee = blockIdx.x * 16 + (tid & 15);
        if (tid < 256 && t < T && ee < NE) {
            const int l = (tid & 15) + 16 * (tid >> 6), r = (tid >> 4) & 3;
            float v = red[0][l][r];
#pragma unroll
            for (int w = 1; w < RT_WAVES; ++w) v += red[w][l][r];
            if (a.L.router_bias && ee < E) v += a.L.router_bias[ee];
            st_dev((uint32_t *)a.b.logits + t * (E + 1) + ee, __float_as_uint(v));
        }
    }
    if (!last_of(a.b.cnt + blockIdx.y, gridDim.x, &s_last)) return;
    const int t = blockIdx.y * 16 + wave;
    if (t < T) {
        const float *lg = a.b.logits + t * (E + 1);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = lane + 64 * i;
            const float l = e < E ? ld_agent(lg + e) : 0.0f;
            v[i] = l != l ? -__builtin_inff() : l;
        }
        TopkOut tk = wave_topk_regs(v, E, K);
        tk.idx = min(max(tk.idx, 0), E - 1);
        if (lane < K) {
            s_sel[t * K + lane] = (int16_t)tk.idx;
            if (gridDim.y > 1) st_dev((uint32_t *)a.b.idx + t * K + lane, (uint32_t)tk.idx);
            a.b.w[t * K + lane] = tk.w;
            if (a.out_idx) a.out_idx[t * K + lane] = tk.idx;
            if (a.out_w) a.out_w[t * K + lane] = tk.w;
        }
    }
    if (a.route_only) return;
    const bool tiles = gridDim.y > 1;                        // (else the selections are all in LDS)
    if (tiles && !last_of(a.b.cnt + MX_TMAX / 16, gridDim.y, &s_last)) return;
    // ---- the chosen experts in ascending order, and under each its tokens in order
    if (tid < 256)
#pragma unroll
        for (int i = 0; i < MW; ++i) s_mask[tid][i] = 0u;
    __syncthreads();
    for (int i = tid; i < T * K; i += RT_THREADS) {
        if (tiles)
            s_sel[i] = (int16_t)__hip_atomic_load((const uint32_t *)a.b.idx + i, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT);
        const int tt = i / K;
        atomicOr(&s_mask[s_sel[i]][tt >> 5], 1u << (tt & 31));
    }
    __syncthreads();
    // an expert of more than 16 tokens is listed once per 16 of them (its items share the slot)
    int cnt = 0;
    if (tid < 256)
#pragma unroll
        for (int i = 0; i < MW; ++i) cnt += __popc(s_mask[tid][i]);
    const int own = (cnt + 15) >> 4;
    const uint64_t lt = (1ull << lane) - 1;
    int slot = 0, item = 0, slots = 0, items = 0;            // before this lane's, and of the wave
#pragma unroll
    for (int i = 0; i < MX_TMAX / 16; ++i) {
        const uint64_t b = __ballot(own > i);
        if (i == 0) {
            slot = __popcll(b & lt);
            slots = __popcll(b);
        }
        item += __popcll(b & lt);
        items += __popcll(b);
    }
    if (tid < 256 && lane == 0) {
        s_cnt[wave] = slots;
        s_itm[wave] = items;
    }
    __syncthreads();
    if (tid < 256) {
        for (int w = 0; w < wave; ++w) {
            slot += s_cnt[w];
            item += s_itm[w];
        }
        s_slot[tid] = slot;
        for (int i = 0; i < own; ++i) a.b.act[item + i] = mx_item(tid, slot, i, min(cnt - 16 * i, 16));
    }
    if (tid == 0) *a.b.nact = s_itm[0] + s_itm[1] + s_itm[2] + s_itm[3];
    __syncthreads();
    for (int i = tid; i < T * K; i += RT_THREADS) {
        const int e = s_sel[i], tt = i / K;
        int before = __popc(s_mask[e][tt >> 5] & ((1u << (tt & 31)) - 1));
#pragma unroll
        for (int q = 0; q < MW - 1; ++q)
            if (q < tt >> 5) before += __popc(s_mask[e][q]);
        a.b.pos[s_slot[e] * MX_TMAX + before] = (int16_t)i;
    }
}

// h of a token and expert, in the order down reads it as an MFMA operand: per step of 128 columns
// and MFMA j, the 8 columns 32 g + 8 j .. + 7 of the four blocks g, hi then lo each, so that a
// load's pieces of one row are 128 bytes together.
__host__ __device__ inline int64_t h_row(int I) { return (I + 127) / 128 * 256; }              // values of a row
__device__ __forceinline__ int h_place(int block) { return (block >> 2) * 256 + (block & 3) * 16; }   // of 32 columns

// -------------------------------------------------------------------------- gate/up
// The tokens' rows of x are staged in LDS, 2048 columns at a time: read as MFMA operands from
// global memory they are 64 separate 16-byte pieces a load, which costs the address unit four
// times a contiguous one.  PN panels of 16 columns of h a workgroup, four waves each: with one, more
// workgroups and their loads fit a compute unit, with two x is staged half as often (T = 7 35.9 and
// 37.2 us a layer, T = 12 48.8 and 48.7, T = 20 67.7 and 60.8; four panels 39.0, 51.8, 66.3).
// Workgroups that loop over items, loading ahead, gain nothing (T = 7 38, T = 20 61).
constexpr int GU_QUADS = MT_WAVES / 2;                       // quads of a chunk: one per wave of a panel
constexpr int GU_PITCH = GU_QUADS * 1024 + 16;               // bytes of a staged row (padded: banks)

// One item's block of 16 PN columns of h, by one workgroup: expert e (sh: the shared one), its cnt
// tokens, the row of h of token lane % 16 in pos (every wave) and its weight in w (wave 0).
struct GuShared {
    float w[16];
    int pos[16];
};
template <int PN>
__device__ __forceinline__ void gate_up_block(const MxArgs &a, uint8_t *sx, GuShared &s, int blk, bool sh, int e, int cnt,
                                              int pos, float w) {
    // [cnt][GU_PITCH] of x, then the waves' sums in its place
    f32x4(*red)[2][64] = (f32x4(*)[2][64])sx;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, I = a.L.I, K = a.L.K, T = a.T;
    // (field by field: a choice between two descriptors would put the arguments in memory)
    const uint8_t *gc = sh ? a.L.s_gate.codes : a.L.gate.codes, *uc = sh ? a.L.s_up.codes : a.L.up.codes;
    const uint8_t *gs = (const uint8_t *)(sh ? a.L.s_gate.scales : a.L.gate.scales);
    const uint8_t *us = (const uint8_t *)(sh ? a.L.s_up.scales : a.L.up.scales);
    const int64_t gst = sh ? a.L.s_gate.stride : a.L.gate.stride, ust = sh ? a.L.s_up.stride : a.L.up.stride;
    const int KS = (H + 127) >> 7, KQ = (KS + 3) >> 2;
    const int pw = wave % PN, kg = wave / PN;                // 16-column panel, quad of a chunk
    const int p = PN * blk + pw;
    const int64_t pg = (e * gst) / 16 + p, pu = (e * ust) / 16 + p;
    u32x4 bg[4], bu[4];
    uint32_t sg = 0, su = 0;
    auto load_w = [&](int q) __attribute__((always_inline)) {
        sg = *(const uint32_t *)(gs + (pg * KQ + q) * MX_QS + 4 * lane);
        su = *(const uint32_t *)(us + (pu * KQ + q) * MX_QS + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 4 * q + (4 * q + i < KS ? i : 0);
            bg[i] = __builtin_nontemporal_load((const u32x4 *)(gc + (pg * KS + s) * MX_TILE + 16 * lane));
            bu[i] = __builtin_nontemporal_load((const u32x4 *)(uc + (pu * KS + s) * MX_TILE + 16 * lane));
        }
    };
    if (kg < KQ) load_w(kg);
    if (wave == 0 && lane < cnt) {
        s.pos[lane] = pos;
        s.w[lane] = w;
    }
    {
        const int r = n < cnt ? n : cnt - 1;                 // (past the tokens: repeated, discarded)
        f32x4 ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
        for (int q0 = 0; q0 < KQ; q0 += GU_QUADS) {
            const int q = q0 + kg;
            if (q0 && q < KQ) load_w(q);                     // (the first is on its way)
            // a wave stages whole rows, 1 KB per load (columns past H meet zero weights: any value
            // of the row will do)
            for (int i = wave; i < cnt * GU_QUADS; i += GU_QUADS * PN) {
                const int row = i / GU_QUADS, c = i % GU_QUADS, ps = __builtin_amdgcn_readlane(pos, row);
                const int t = sh ? ps - T * K : ps / K, k = min((q0 + c) * 512 + 8 * lane, H - 8);
                *(u32x4 *)(sx + row * GU_PITCH + 1024 * c + 16 * lane) = *(const u32x4 *)(a.x + (int64_t)t * H + k);
            }
            __syncthreads();
            if (q < KQ) {
                const uint8_t *xr = sx + r * GU_PITCH + 1024 * kg + 64 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (4 * q + i >= KS) break;
                    const float cg = mx_scale(sg, i), cu = mx_scale(su, i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf16x8 A = *(const bf16x8 *)(xr + 256 * i + 16 * j);
                        ag = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, mx_bf16(bg[i][j], cg), ag, 0, 0, 0);
                        au = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, mx_bf16(bu[i][j], cu), au, 0, 0, 0);
                    }
                }
            }
            __syncthreads();                                 // the chunk is consumed
        }
        red[wave][0][lane] = ag;
        red[wave][1][lane] = au;
        __syncthreads();
        // thread: a token and a column
        const int tk = tid / (16 * PN), cb = tid % (16 * PN), col = 16 * PN * blk + cb, c = col & 31;
        if (tk < cnt) {
            const int l = (cb & 15) + 16 * (tk >> 2), rr = tk & 3, w0 = cb >> 4;
            float gv = 0.0f, uv = 0.0f;
#pragma unroll
            for (int k = 0; k < GU_QUADS; ++k) {
                gv += red[w0 + PN * k][0][l][rr];
                uv += red[w0 + PN * k][1][l][rr];
            }
            // h = w silu(g) u as the bf16 pair hi + lo
            const float h = silu(gv) * uv * s.w[tk];
            const uint16_t hi = f32_to_bf16(h);
            const uint16_t lo = f32_to_bf16(h - bf16_to_f32(hi));
            uint16_t *d = a.b.h + s.pos[tk] * h_row(I) + h_place(col >> 5) + 64 * (c >> 3) + (c & 7);
            d[0] = hi;
            d[8] = lo;
            // a last step of 64 columns: its other two blocks meet zero weights, and must be finite
            if ((I & 64) && col >= I - 32)
                for (int x = 1; x <= 2; ++x) {
                    uint16_t *z = a.b.h + s.pos[tk] * h_row(I) + h_place((col >> 5) + x) + 64 * (c >> 3) + (c & 7);
                    z[0] = z[8] = 0;
                }
        }
    }
}

template <int PN>
__global__ __launch_bounds__(64 * GU_QUADS * PN) __attribute__((amdgpu_waves_per_eu(4))) void k_mx_gate_up(MxArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t sx[];
    __shared__ GuShared s;
    const int lane = threadIdx.x & 63, n = lane & 15, K = a.L.K, T = a.T;
    const int nsh = a.L.has_shared ? (T + 15) >> 4 : 0, item = blockIdx.y;
    const bool sh = item < nsh;
    int nact = 0, act = 0;
    if (!sh) {
        nact = *a.b.nact;
        act = a.b.act[item - nsh];
        if (item - nsh >= nact) return;
    }
    const MxItem it = mx_unpack(item, nsh, act, T);
    const int pos = sh ? T * K + 16 * item + n : (int)a.b.pos[it.list + n];
    float w = 1.0f;
    if (threadIdx.x < it.count) {
        if (!sh) w = a.b.w[pos];
        else if (a.gated) w = sigmoid(a.b.logits[(16 * item + n) * (a.L.E + 1) + a.L.E]);
    }
    gate_up_block<PN>(a, sx, s, blockIdx.x, sh, it.e, it.count, pos, w);
}

// Up to this many tokens route and gate/up are one launch: us a layer against two launches (2048 x
// 512, 256 experts), T = 1 15.9 and 18.8, T = 2 20.1 and 23.4, T = 3 24.3 and 26.3, T = 4 26.6 and
// 28.8; T = 5 to 8 within 2 % (each workgroup takes every token's top-k, and they no longer all
// fit the device at once).
constexpr int TOKEN_MAX = 4;

// One to MT tokens: route and gate/up in one launch.  The first workgroups form the logits, 16 experts
// each, and write them to every copy of the decode state's logit words (shared out among the
// tokens) under the call's tag; the others wait, a wave per token, until it has all logits, and take
// the top-k themselves (decode_state.h: a wait is bounded, and only for workgroups of lower
// index).  The workgroup of (j, 32 columns of h) takes the j-th of the experts any token chose.
// Saves the last router workgroup's counting, selecting and listing and a launch.
template <int MT>
__global__ __launch_bounds__(MT_THREADS) __attribute__((amdgpu_waves_per_eu(4))) void k_mx_token(MxArgs a, int nR) {
    static_assert(MT <= MT_WAVES && MT * 16 <= LOGIT_COPIES * 16, "a wave and a logit copy per token");
    extern __shared__ __attribute__((aligned(16))) uint8_t sx[];
    __shared__ GuShared s;
    __shared__ float part[RT_WAVES][MT][16], lg[MT][16];
    __shared__ int s_idx[MT * 16];
    __shared__ float s_w[MT * 16], s_gate[MT];
    __shared__ uint32_t s_any[8];                            // experts that any token chose
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, E = a.L.E, K = a.L.K, NE = E + a.gated, T = MT == 1 ? 1 : a.T;
    int per = LOGIT_COPIES;                                  // copies of a token's logits
    if constexpr (MT > 1)
        while (per * T > LOGIT_COPIES) per >>= 1;
    uint32_t *ctl = a.b.ctl;
    const uint32_t tag = call_tag(ctl);
    if ((int)blockIdx.x < nR) {
        const int e = blockIdx.x * 16 + n, ec = e < NE ? e : NE - 1;
        const uint16_t *wr = ec < E ? a.L.router_w + (int64_t)ec * H : a.L.shared_gate_w;
        const uint16_t *xr = a.x + (int64_t)(n < T ? n : 0) * H;       // (rows past the tokens: the first, discarded)
        // (k_mx_route's sums in its order, so that the logits have the same bits: this wave takes the
        // shares of its waves `wave` and `wave` + 8)
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int steps = H / 32;
        for (int s0 = wave; s0 < steps; s0 += 4 * RT_WAVES) {
            u32x4 B[8], A[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int st = s0 + i * MT_WAVES, k = 32 * st + 8 * g;
                B[i] = A[i] = (u32x4){0u, 0u, 0u, 0u};
                if (st < steps) {
                    B[i] = *(const u32x4 *)(wr + k);
                    A[i] = *(const u32x4 *)(xr + k);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[i]),
                                                                     __builtin_bit_cast(bf16x8, B[i]), acc[i & 1], 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * g + r;
            if (t < MT) {
                part[wave][t][n] = acc[0][r];
                part[wave + MT_WAVES][t][n] = acc[1][r];
            }
        }
        __syncthreads();
        if (tid < 16 * T) {
            const int t = tid >> 4, ee = blockIdx.x * 16 + n;
            float v = part[0][t][n];
#pragma unroll
            for (int w = 1; w < RT_WAVES; ++w) v += part[w][t][n];
            if (a.L.router_bias && ee < E) v += a.L.router_bias[ee];
            lg[t][n] = v;
        }
        __syncthreads();
        // two words of a copy per thread, a copy's run of 128 bytes by 8 neighbouring ones
        const int t = (tid >> 3) / per;
        if (tid < LOGIT_COPIES * 8 && t < T) {
            const int q = tid & 7, e0 = blockIdx.x * 16 + 2 * q;
            uint32_t *dst = ctl + LOGIT_BASE + (tid >> 3) * LOGIT_STRIDE + 2 * e0;
            if (e0 + 1 < NE)
                st_dev128(dst, (u32x4){__float_as_uint(lg[t][2 * q]), tag, __float_as_uint(lg[t][2 * q + 1]), tag});
            else if (e0 < NE)
                st_dev64((uint64_t *)dst, __float_as_uint(lg[t][2 * q]) | ((uint64_t)tag << 32));
        }
        return;
    }
    const int b = blockIdx.x - nR, nblk = a.L.I / 32, item = b / nblk, blk = b % nblk;
    const int nsh = a.L.has_shared ? 1 : 0, j = item - nsh;  // j: place among the chosen experts
    const bool sh = j < 0;
    if constexpr (MT > 1) {
        if (tid < 8) s_any[tid] = 0u;
        __syncthreads();
    }
    if (wave < T && (!sh || a.gated)) {
        float gate;
        const TopkOut tk = select_topk_from(
            ctl, (const uint64_t *)(ctl + LOGIT_BASE + (wave * per + b % per) * LOGIT_STRIDE), tag, E, K, a.gated, &gate);
        if (lane < K) {
            s_idx[wave * K + lane] = tk.idx;
            s_w[wave * K + lane] = tk.w;
            if constexpr (MT > 1) atomicOr(&s_any[tk.idx >> 5], 1u << (tk.idx & 31));
        }
        if (lane == 0) s_gate[wave] = gate;
    }
    __syncthreads();
    int e = 0, cnt = T, pos = T * K + n;
    float w = 1.0f;
    if (sh) {
        if (a.gated && tid < T) w = s_gate[tid];
    } else {
        int total = K;
        if constexpr (MT == 1) {                             // (ascending already)
            e = __builtin_amdgcn_readfirstlane(s_idx[j]);
            pos = j;
        } else {
            // the j-th expert of the union, and which choices (token t's k-th: t K + k) are of it
            uint32_t word = 0;
            int k = 0, base = 0;
            total = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = __builtin_amdgcn_readfirstlane(s_any[i]);
                const int c = __popc(u);
                if (j >= total && j < total + c) {
                    word = u;
                    k = j - total;
                    base = 32 * i;
                }
                total += c;
            }
            if (j >= total) {
                // (after a wait that gave up, workgroups may hold different selections: the list has an
                // entry, here one of no tokens, in every place that the one of j = 0 may count)
                if (blk == 0 && tid == 0) a.b.act[j] = 0;
                return;
            }
            for (; k > 0; --k) word &= word - 1;
            e = base + __builtin_ctz(word);
            constexpr int Q = (MT * 16 + 63) / 64;
            cnt = 0;
            pos = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = 64 * q + lane;
                for (uint64_t m = __ballot(i < T * K && s_idx[i] == e); m; m &= m - 1) {
                    if (n == cnt) pos = 64 * q + __builtin_ctzll(m);
                    ++cnt;
                }
            }
        }
        if (tid < cnt) w = s_w[pos];
        if (blk == 0 && wave == 0) {                         // the lists that down reads
            if (lane < cnt) a.b.pos[j * MX_TMAX + lane] = (int16_t)pos;
            if (lane == 0) a.b.act[j] = mx_item(e, j, 0, cnt);
            if (lane == 0 && j == 0) *a.b.nact = total;
        }
        if (blk == 0 && j == 0 && tid < T * K) {
            if (a.out_idx) a.out_idx[tid] = s_idx[tid];
            if (a.out_w) a.out_w[tid] = s_w[tid];
        }
    }
    gate_up_block<2>(a, sx, s, blk, sh, e, cnt, pos, w);
}

// ----------------------------------------------------------------------------- down
// An item is a quad of the columns of a work-list entry (the shared expert's first) for 16 NP
// output rows; its tokens come eight at a time (16 operand rows, hi and lo of each).  Each wave adds its items'
// results into sums of its own in LDS, in item order (a register accumulator per token would
// have to run every item over all tokens); the waves' sums are added in wave order.
template <int NP, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(4))) void k_mx_down(MxArgs a) {
    constexpr int C = 16 * NP;                               // output rows
    extern __shared__ __attribute__((aligned(16))) float sums[];   // [W][T][C]
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, I = a.L.I, K = a.L.K, T = a.T;
    const int KS = (I + 127) >> 7, KQ = (KS + 3) >> 2;
    const int nsh = a.L.has_shared ? (T + 15) >> 4 : 0;
    const int z = blockIdx.y;
    const int p0 = NP * blockIdx.x;                          // H is a multiple of 64
    float *mine = sums + wave * T * C;
    // the next item's expert and tokens are fetched while this one is multiplied
    int act_nx = 0, pos_nx = 0;
    auto fetch = [&](int it) __attribute__((always_inline)) {
        const int i = it / KQ;
        act_nx = i >= nsh && i < nsh + MX_ITEMS ? a.b.act[i - nsh] : 0;
    };
    auto fetch_pos = [&](int it) __attribute__((always_inline)) {
        const int i = it / KQ;
        const MxItem w = mx_unpack(i, nsh, act_nx, T);
        pos_nx = w.list < 0 ? T * K + 16 * i + n : (int)a.b.pos[w.list + n];
    };
    int it = z * W + wave;
    fetch(it);
    // (the launch before is complete: the generation its logits were tagged with is used up)
    if (a.tagged && blockIdx.x == 0 && z == 0 && tid == 0) st_dev(a.b.ctl + CTL_GEN, call_tag(a.b.ctl));
    const int items = (*a.b.nact + nsh) * KQ;
    if (it < items) fetch_pos(it);
    for (int i = lane; i < T * C; i += 64) mine[i] = 0.0f;
    for (; it < items; it += a.shares * W) {
        const int q = it % KQ;
        const bool sh = it / KQ < nsh;
        const MxItem w = mx_unpack(it / KQ, nsh, __builtin_amdgcn_readfirstlane(act_nx), T);
        const int e = w.e, cnt = w.count;
        const int pos = pos_nx;
        const uint8_t *codes = sh ? a.L.s_down.codes : a.L.down.codes;
        const uint8_t *scales = (const uint8_t *)(sh ? a.L.s_down.scales : a.L.down.scales);
        const int64_t pe = (e * (sh ? a.L.s_down.stride : a.L.down.stride)) / 16 + p0;
        u32x4 b[NP][4];
        uint32_t sc[NP];
#pragma unroll
        for (int u = 0; u < NP; ++u) {
            sc[u] = *(const uint32_t *)(scales + ((pe + u) * KQ + q) * MX_QS + 4 * lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * q + (4 * q + i < KS ? i : 0);
                b[u][i] = __builtin_nontemporal_load((const u32x4 *)(codes + ((pe + u) * KS + s) * MX_TILE + 16 * lane));
            }
        }
        const int nx = it + a.shares * W;
        fetch(nx);
        for (int m0 = 0; m0 < cnt; m0 += 8) {
            const int r = m0 + (n >> 1), ps = __shfl(pos, r < cnt ? r : 0);
            const uint16_t *hr = a.b.h + ps * h_row(I) + 16 * g + 8 * (n & 1);
            f32x4 acc[NP];
#pragma unroll
            for (int u = 0; u < NP; ++u) acc[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * q + i >= KS) break;
                u32x4 A[4];                                  // (rows past the tokens repeat the first)
#pragma unroll
                for (int j = 0; j < 4; ++j) A[j] = *(const u32x4 *)(hr + 256 * (4 * q + i) + 64 * j);
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                    const float cs = mx_scale(sc[u], i);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, A[j]), mx_bf16(b[u][i][j], cs), acc[u], 0, 0, 0);
                }
            }
            if (m0 == 0 && nx < items) fetch_pos(nx);
            // hi and lo of a token are registers 0, 1 (or 2, 3) of one lane
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int rr = m0 + 2 * g + x, pt = __shfl(pos, rr < cnt ? rr : 0);
                if (rr < cnt) {
                    float *d = mine + (sh ? pt - T * K : pt / K) * C + n;
#pragma unroll
                    for (int u = 0; u < NP; ++u) d[16 * u] += acc[u][2 * x] + acc[u][2 * x + 1];
                }
            }
        }
        if (cnt == 0 && nx < items) fetch_pos(nx);           // (an entry of no tokens: k_mx_token)
    }
    __syncthreads();
    // thread: a token and four columns
    constexpr int PC = C / 4;
    const int tk = tid / PC, c4 = 4 * (tid % PC);
    const bool live = tk < T;
    const int64_t o = (int64_t)tk * H + C * blockIdx.x + c4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (live)
#pragma unroll
        for (int w = 0; w < W; ++w) v += *(const f32x4 *)(sums + (w * T + tk) * C + c4);
    if (a.shares > 1) {
        if (live) st_dev128(a.b.part + (int64_t)z * T * H + o, __builtin_bit_cast(u32x4, v));
        if (!last_of(a.b.cnt + MX_CNT_DOWN + blockIdx.x, a.shares, &s_last)) return;
        if (live) {
            v = (f32x4){0.f, 0.f, 0.f, 0.f};
            const float *pp = a.b.part + o;
            const int64_t st = (int64_t)T * H;
            for (int s = 0; s < a.shares; s += 4) {          // (past the last: repeated, not added)
                const int l = a.shares - 1;
                f32x4 q0, q1, q2, q3;
                ld_agent128x4(pp + s * st, pp + min(s + 1, l) * st, pp + min(s + 2, l) * st, pp + min(s + 3, l) * st, q0,
                              q1, q2, q3);
                v += q0;
                if (s + 1 <= l) v += q1;
                if (s + 2 <= l) v += q2;
                if (s + 3 <= l) v += q3;
            }
        }
    }
    if (live)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx_store(a.y, o + c, v[c], a.y_dtype);
}

// entries of the work list (at most), the shared expert's included
int64_t max_items(const Layer &L, int64_t T) {
    const int64_t experts = T * L.K < L.E ? T * L.K : L.E;
    return experts + T * L.K / 16 + (L.has_shared ? (T + 15) / 16 : 0);
}

// At most 32 items (one to three tokens of top-8): one panel per workgroup and 16 waves, so one
// or two rounds of loads and no shares (T = 1: 6.6 us against 7.9; T = 7, 57 items: 15.4
// against 12.3).  More: two panels and 8 waves, each row of h read for twice the weights, the
// items shared out until there are two workgroups per compute unit.  Over 64 tokens one panel,
// as the waves' sums of two would leave LDS for one workgroup per compute unit.
struct DownPlan {
    int np, waves, shares;
};
DownPlan down_plan(const Layer &L, int64_t T) {
    DownPlan d;
    const int64_t items = max_items(L, T) * ((L.I + 511) / 512);   // (at most)
    if (items <= 32 && T <= 64) {
        d.np = 1;
        d.waves = 16;
        d.shares = 1;
        return d;
    }
    d.np = T <= 64 ? 2 : 1;
    d.waves = 8;
    const int groups = L.H / (16 * d.np), want = (2 * n_compute_units() + groups - 1) / groups;
    const int64_t most = (items + d.waves - 1) / d.waves;
    int64_t s = want < MX_SHARES ? want : MX_SHARES;
    if (s > most) s = most;
    d.shares = (int)s;
    return d;
}

}  // namespace

hipError_t launch_mx_layer(const Layer &L, const uint16_t *x, int64_t T, const MxBufs &b, void *y, int y_dtype,
                           int32_t *out_idx, float *out_w, bool route_only, hipStream_t s) {
    MxArgs a{};
    a.L = L;
    a.b = b;
    a.x = x;
    a.T = (int)T;
    a.gated = L.shared_gate_w != nullptr && L.has_shared && !route_only;
    a.out_idx = out_idx;
    a.out_w = out_w;
    a.y = y;
    a.y_dtype = y_dtype;
    const DownPlan d = down_plan(L, T);
    a.shares = d.shares;
    a.route_only = route_only;
    a.tagged = T <= TOKEN_MAX && !route_only;
    const unsigned nR = (unsigned)((L.E + a.gated + 15) / 16);
    const size_t gu_x = (size_t)(T < 16 ? T : 16) * GU_PITCH, gu_red = MT_WAVES * 2048, gu_lds = gu_x > gu_red ? gu_x : gu_red;
    hipError_t e;
    if (a.tagged) {
        const dim3 grid(nR + (unsigned)(L.I / 32 * (T * L.K + (L.has_shared ? 1 : 0))));
        if (T == 1) hipLaunchKernelGGL(k_mx_token<1>, grid, dim3(MT_THREADS), gu_lds, s, a, (int)nR);
        else hipLaunchKernelGGL(k_mx_token<TOKEN_MAX>, grid, dim3(MT_THREADS), gu_lds, s, a, (int)nR);
    } else {
        hipLaunchKernelGGL(k_mx_route, dim3(nR, (unsigned)((T + 15) / 16)), dim3(RT_THREADS), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess || route_only) return e;
        const unsigned items = (unsigned)max_items(L, T);
        if (T <= 8)                                          // (figures at gate_up_block)
            hipLaunchKernelGGL(k_mx_gate_up<1>, dim3((unsigned)(L.I / 16), items), dim3(64 * GU_QUADS), gu_lds, s, a);
        else hipLaunchKernelGGL(k_mx_gate_up<2>, dim3((unsigned)(L.I / 32), items), dim3(128 * GU_QUADS), gu_lds, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 grid((unsigned)(L.H / (16 * d.np)), (unsigned)a.shares), thr((unsigned)(64 * d.waves));
    const size_t lds = (size_t)d.waves * T * 16 * d.np * 4;
    if (d.waves == 16) hipLaunchKernelGGL((k_mx_down<1, 16>), grid, thr, lds, s, a);
    else if (d.np == 1) hipLaunchKernelGGL((k_mx_down<1, 8>), grid, thr, lds, s, a);
    else hipLaunchKernelGGL((k_mx_down<2, 8>), grid, thr, lds, s, a);
    return hipGetLastError();
}

}  // namespace qs
