// mx4_moe.hip -- the sparse MoE layer with MX4 experts for a few tokens (up to MX_TMAX in one
// pass; more run in passes of MX_TMAX): three launches.
//
//   route    router logits on v_mfma_f32_16x16x32_bf16 (16 experts per workgroup, the columns
//            split over its waves).  The workgroup that finishes last -- counted, so nothing
//            ever waits -- takes every token's top-k, and lists the experts any token chose
//            (ascending), with each token's place among their rows of h.
//   gate/up  one workgroup per (listed expert, 32 columns of h): gathers the expert's tokens
//            as the rows of the activation operand, so each expert's weights are read once
//            however many tokens chose it, and an expert that one token chose costs one
//            16-row tile.  h = w silu(g) u carries the token's routing weight and leaves as
//            the bf16 pair hi + lo (h to 2^-17), two operand rows.
//   down     one workgroup per 32 rows of the output and share of the listed experts: the
//            experts' down matrices lie side by side along the reduction axis, so the sum over
//            experts is made by the accumulators; a token's rows of an expert it did not
//            choose are zero registers (masked loads).  hi and lo of a token are neighbouring
//            accumulator registers and are added in the lane.  Shares are added in a fixed
//            order by the share that finishes last.
//
// All three are bound by the weight stream: (union of the chosen experts + shared) x
// 3 H I x 17/32 bytes.  Every sum is fp32 in a fixed order; there are no float atomics.
#include "mx4.h"

namespace qs {

namespace {

constexpr int MT_THREADS = 512, MT_WAVES = 8;

struct MxArgs {
    Layer L;
    MxBufs b;
    const uint16_t *x;
    int T;
    int gated;
    int32_t *out_idx;
    float *out_w;
    void *y;
    int y_dtype;
    int shares;                       // down: workgroups per 32 output rows
};

__device__ __forceinline__ void st_agent(uint32_t *p, uint32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float ld_agent(const float *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the last of n to come here.  What it reads of the others' work they
// stored at device scope (written through), so the count only has to follow the stores'
// completion, and it reads at device scope.  The counter goes back to zero for the next call.
__device__ __forceinline__ bool last_of(uint32_t *cnt, uint32_t n, int *s_last) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // (every wave its own)
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        if (last) st_agent(cnt, 0u);
        *s_last = last;
    }
    __syncthreads();
    return *s_last != 0;
}

// ---------------------------------------------------------------------------- route
template <int MT>
__global__ __launch_bounds__(MT_THREADS) void k_mx_route(MxArgs a) {
    __shared__ f32x4 red[MT_WAVES][64];
    __shared__ int s_last;
    __shared__ int s_idx[MX_TMAX][16];
    __shared__ int s_slot[256], s_cnt[4];
    __shared__ uint8_t s_used[256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, E = a.L.E, K = a.L.K, T = a.T, NE = E + a.gated;
    // ---- logits of 16 experts (row E: the shared expert's gate), columns split over waves
    {
        const int e = blockIdx.x * 16 + n, ec = e < NE ? e : NE - 1;
        const uint16_t *wr = ec < E ? a.L.router_w + (int64_t)ec * H : a.L.shared_gate_w;
        f32x4 acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
        const int steps = H / 32;
        for (int s0 = wave; s0 < steps; s0 += 4 * MT_WAVES) {
            u32x4 B[4], A[MT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = s0 + i * MT_WAVES, k = 32 * s + 8 * g;
                const bool live = s < steps;
                B[i] = live ? *(const u32x4 *)(wr + k) : (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int t = 16 * m + n;
                    A[m][i] = live && t < T ? *(const u32x4 *)(a.x + (int64_t)t * H + k) : (u32x4){0u, 0u, 0u, 0u};
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[m][i]),
                                                                     __builtin_bit_cast(bf16x8, B[i]), acc[m], 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            red[wave][lane] = acc[m];
            __syncthreads();
            const int t = 16 * m + (tid >> 4), ee = blockIdx.x * 16 + (tid & 15);
            if (tid < 256 && t < T && ee < NE) {
                const int l = (tid & 15) + 16 * (tid >> 6), r = (tid >> 4) & 3;
                float v = red[0][l][r];
#pragma unroll
                for (int w = 1; w < MT_WAVES; ++w) v += red[w][l][r];
                if (a.L.router_bias && ee < E) v += a.L.router_bias[ee];
                st_agent((uint32_t *)a.b.logits + t * (E + 1) + ee, __float_as_uint(v));
            }
            __syncthreads();
        }
    }
    if (!last_of(a.b.cnt, gridDim.x, &s_last)) return;
    // ---- the last workgroup: one wave per token takes the top-k
    if (tid < 256) s_used[tid] = 0;
    __syncthreads();
    for (int t = wave; t < T; t += MT_WAVES) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float l = lane + 64 * i < E ? ld_agent(a.b.logits + t * (E + 1) + lane + 64 * i) : 0.0f;
            v[i] = l != l ? -__builtin_inff() : l;
        }
        TopkOut tk = wave_topk_regs(v, E, K);
        tk.idx = min(max(tk.idx, 0), E - 1);
        if (lane < K) {
            s_idx[t][lane] = tk.idx;
            s_used[tk.idx] = 1;
            a.b.idx[t * K + lane] = tk.idx;
            a.b.w[t * K + lane] = tk.w;
            if (a.out_idx) a.out_idx[t * K + lane] = tk.idx;
            if (a.out_w) a.out_w[t * K + lane] = tk.w;
        }
    }
    __syncthreads();
    // ---- the chosen experts in ascending order, and each token's row of h under them
    const bool used = tid < 256 && s_used[tid];
    const uint64_t bal = __ballot(used);
    if (tid < 256 && lane == 0) s_cnt[wave] = __popcll(bal);
    __syncthreads();
    const int nact = s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3];
    if (tid < 256) {
        int base = 0;
        for (int w = 0; w < wave; ++w) base += s_cnt[w];
        const int slot = base + __popcll(bal & ((1ull << lane) - 1));
        s_slot[tid] = slot;
        if (used) a.b.act[slot] = tid;
    }
    if (tid == 0) *a.b.nact = nact;
    for (int i = tid; i < nact * MX_TMAX; i += MT_THREADS) a.b.pos[i] = -1;
    __syncthreads();
    for (int i = tid; i < T * K; i += MT_THREADS) {
        const int t = i / K;
        a.b.pos[s_slot[s_idx[t][i % K]] * MX_TMAX + t] = (int16_t)i;
    }
}

// -------------------------------------------------------------------------- gate/up
__global__ __launch_bounds__(MT_THREADS) void k_mx_gate_up(MxArgs a) {
    __shared__ f32x4 red[MT_WAVES][2][64];
    __shared__ int s_tok[MX_TMAX], s_pos[MX_TMAX];
    __shared__ float s_w[MX_TMAX];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, I = a.L.I, K = a.L.K, T = a.T;
    const int slot = (int)blockIdx.y - (a.L.has_shared ? 1 : 0);
    const bool sh = slot < 0;
    if (!sh && slot >= *a.b.nact) return;
    const int64_t e = sh ? 0 : a.b.act[slot];
    const QMat mg = sh ? a.L.s_gate : a.L.gate, mu = sh ? a.L.s_up : a.L.up;
    const int KS = (H + 127) >> 7, KQ = (KS + 3) >> 2;
    const int pw = wave & 1, kg = wave >> 1;                 // 16-column panel, share of the columns
    const int p = 2 * blockIdx.x + pw;
    const int64_t pg = (e * mg.stride) / 16 + p, pu = (e * mu.stride) / 16 + p;

    // the expert's tokens, in order: the rows of the activation operand
    if (wave == 0) {
        int pos = -1;
        float w = 1.0f;
        if (lane < T) {
            pos = sh ? T * K + lane : a.b.pos[slot * MX_TMAX + lane];
            if (pos >= 0 && !sh) w = a.b.w[pos];
            if (sh && a.gated) w = sigmoid(a.b.logits[lane * (a.L.E + 1) + a.L.E]);
        }
        const uint64_t bal = __ballot(pos >= 0);
        if (pos >= 0) {
            const int r = __popcll(bal & ((1ull << lane) - 1));
            s_tok[r] = lane;
            s_pos[r] = pos;
            s_w[r] = w;
        }
        if (lane == 0) s_n = __popcll(bal);
    }
    __syncthreads();
    const int cnt = s_n;
    for (int m0 = 0; m0 < cnt; m0 += 16) {
        const bool live = m0 + n < cnt;
        const uint16_t *xr = a.x + (int64_t)(live ? s_tok[m0 + n] : 0) * H;
        f32x4 ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
        for (int q = kg; q < KQ; q += MT_WAVES / 2) {
            u32x4 bg[4], bu[4];
            const uint32_t sg = *(const uint32_t *)((const uint8_t *)mg.scales + (pg * KQ + q) * MX_QS + 4 * lane);
            const uint32_t su = *(const uint32_t *)((const uint8_t *)mu.scales + (pu * KQ + q) * MX_QS + 4 * lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * q + (4 * q + i < KS ? i : 0);
                bg[i] = __builtin_nontemporal_load((const u32x4 *)(mg.codes + (pg * KS + s) * MX_TILE + 16 * lane));
                bu[i] = __builtin_nontemporal_load((const u32x4 *)(mu.codes + (pu * KS + s) * MX_TILE + 16 * lane));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * q + i;
                if (s >= KS) break;
                u32x4 A[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 128 * s + 32 * g + 8 * j;
                    A[j] = live && k < H ? *(const u32x4 *)(xr + k) : (u32x4){0u, 0u, 0u, 0u};
                }
                const float cg = mx_scale(sg, i), cu = mx_scale(su, i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 Aj = __builtin_bit_cast(bf16x8, A[j]);
                    ag = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Aj, mx_bf16(bg[i][j], cg), ag, 0, 0, 0);
                    au = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Aj, mx_bf16(bu[i][j], cu), au, 0, 0, 0);
                }
            }
        }
        red[wave][0][lane] = ag;
        red[wave][1][lane] = au;
        __syncthreads();
        // thread: token m0 + tid / 32, column tid % 32 of the block
        const int tk = tid >> 5, c = tid & 31;
        if (m0 + tk < cnt) {
            const int l = (c & 15) + 16 * (tk >> 2), r = tk & 3, w0 = c >> 4;
            float gv = 0.0f, uv = 0.0f;
#pragma unroll
            for (int k = 0; k < MT_WAVES / 2; ++k) {
                gv += red[w0 + 2 * k][0][l][r];
                uv += red[w0 + 2 * k][1][l][r];
            }
            // h = w silu(g) u as the bf16 pair hi + lo
            const float h = silu(gv) * uv * s_w[m0 + tk];
            const uint16_t hi = f32_to_bf16(h);
            const uint16_t lo = f32_to_bf16(h - bf16_to_f32(hi));
            uint16_t *d = a.b.h + (int64_t)s_pos[m0 + tk] * 2 * I + 32 * blockIdx.x + c;
            d[0] = hi;
            d[I] = lo;
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------- down
// MT activation tiles of 8 tokens (16 rows: hi and lo of each)
template <int MT>
__global__ __launch_bounds__(MT_THREADS) void k_mx_down(MxArgs a) {
    __shared__ f32x2 red[MT_WAVES][2][64];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, g = lane >> 4;
    const int H = a.L.H, I = a.L.I, K = a.L.K, T = a.T;
    const int KS = (I + 127) >> 7, KQ = (KS + 3) >> 2;
    const int nsh = a.L.has_shared ? 1 : 0;
    const int items = (*a.b.nact + nsh) * KQ;
    const int z = blockIdx.y;
    const int p0 = 2 * blockIdx.x;                           // H is a multiple of 64
    f32x4 acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int it = z * MT_WAVES + wave; it < items; it += a.shares * MT_WAVES) {
        const int slot = it / KQ - nsh, q = it % KQ;         // the shared expert first
        const bool sh = slot < 0;
        const int64_t e = sh ? 0 : a.b.act[slot];
        const QMat md = sh ? a.L.s_down : a.L.down;
        u32x4 b[2][4];
        uint32_t sc[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t p = (e * md.stride) / 16 + p0 + u;
            sc[u] = *(const uint32_t *)((const uint8_t *)md.scales + (p * KQ + q) * MX_QS + 4 * lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * q + (4 * q + i < KS ? i : 0);
                b[u][i] = __builtin_nontemporal_load((const u32x4 *)(md.codes + (p * KS + s) * MX_TILE + 16 * lane));
            }
        }
        int pos[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = 8 * m + (n >> 1);
            pos[m] = t < T ? (sh ? T * K + t : (int)a.b.pos[slot * MX_TMAX + t]) : -1;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (__ballot(pos[m] >= 0) == 0ull) continue;     // none of these tokens chose it
            const uint16_t *hr = a.b.h + (int64_t)(pos[m] >= 0 ? 2 * pos[m] + (n & 1) : 0) * I;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = 4 * q + i;
                if (s >= KS) break;
                u32x4 A[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 128 * s + 32 * g + 8 * j;
                    A[j] = pos[m] >= 0 && k < I ? *(const u32x4 *)(hr + k) : (u32x4){0u, 0u, 0u, 0u};
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float cs = mx_scale(sc[u], i);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[m][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, A[j]), mx_bf16(b[u][i][j], cs), acc[m][u], 0, 0, 0);
                }
            }
        }
    }
    // join the waves in order, a tile of tokens at a time; rows 2 t and 2 t + 1 of a token
    // are registers 0, 1 (or 2, 3) of one lane
    float *part = a.b.part + (int64_t)z * T * H;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            red[wave][u][lane] = (f32x2){acc[m][u][0] + acc[m][u][1], acc[m][u][2] + acc[m][u][3]};
        __syncthreads();
        if (tid < 256) {
            const int u = tid >> 7, l = (tid >> 1) & 63, r = tid & 1;
            float v = red[0][u][l][r];
#pragma unroll
            for (int w = 1; w < MT_WAVES; ++w) v += red[w][u][l][r];
            const int t = 8 * m + 2 * (l >> 4) + r, col = 16 * (p0 + u) + (l & 15);
            if (t < T) {
                if (a.shares == 1) mx_store(a.y, (int64_t)t * H + col, v, a.y_dtype);
                else st_agent((uint32_t *)part + (int64_t)t * H + col, __float_as_uint(v));
            }
        }
        __syncthreads();
    }
    if (a.shares == 1 || !last_of(a.b.cnt + 1 + blockIdx.x, a.shares, &s_last)) return;
    for (int i = tid; i < T * 32; i += MT_THREADS) {
        const int64_t o = (int64_t)(i >> 5) * H + 32 * blockIdx.x + (i & 31);
        float v = ld_agent(a.b.part + o);
        for (int s = 1; s < a.shares; ++s) v += ld_agent(a.b.part + (int64_t)s * T * H + o);
        mx_store(a.y, o, v, a.y_dtype);
    }
}

// workgroups per 32 output rows: enough for two per compute unit, at most one per wave-item
int down_shares(const Layer &L, int64_t T) {
    const int groups = L.H / 32, want = (2 * n_compute_units() + groups - 1) / groups;
    int64_t slots = T * L.K < L.E ? T * L.K : L.E;           // (at most)
    slots = (slots + (L.has_shared ? 1 : 0)) * ((L.I + 511) / 512);
    const int64_t most = (slots + MT_WAVES - 1) / MT_WAVES;
    const int s = want < MX_SHARES ? want : MX_SHARES;
    return (int)(most < s ? most : s);
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
    a.shares = down_shares(L, T);
    const dim3 thr(MT_THREADS);
    const unsigned rg = (unsigned)((L.E + a.gated + 15) / 16);
    if (T <= 16) hipLaunchKernelGGL(k_mx_route<1>, dim3(rg), thr, 0, s, a);
    else if (T <= 32) hipLaunchKernelGGL(k_mx_route<2>, dim3(rg), thr, 0, s, a);
    else hipLaunchKernelGGL(k_mx_route<4>, dim3(rg), thr, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || route_only) return e;
    const int64_t routed = T * L.K < L.E ? T * L.K : L.E;
    hipLaunchKernelGGL(k_mx_gate_up, dim3((unsigned)(L.I / 32), (unsigned)(routed + (L.has_shared ? 1 : 0))), thr, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 grid((unsigned)(L.H / 32), (unsigned)a.shares);
    if (T <= 8) hipLaunchKernelGGL(k_mx_down<1>, grid, thr, 0, s, a);
    else if (T <= 16) hipLaunchKernelGGL(k_mx_down<2>, grid, thr, 0, s, a);
    else if (T <= 32) hipLaunchKernelGGL(k_mx_down<4>, grid, thr, 0, s, a);
    else hipLaunchKernelGGL(k_mx_down<8>, grid, thr, 0, s, a);
    return hipGetLastError();
}

}  // namespace qs
