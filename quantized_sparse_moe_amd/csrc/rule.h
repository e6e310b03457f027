// rule.h -- selection of experts under a routing rule (moe_router_rule), one wave per token.
//
// For the logits l of a token's E experts (live: above -infinity; a NaN is not):
//   s_e = 1 / (1 + exp(-l_e)), or exp(l_e - max l) / sum over the live ones (0 if not live)
//   c_e = s_e + bias_e; without a bias the order of s is the order of l, and c_e = l_e
//   groups of E / G consecutive experts, each worth its largest c or the sum of its two largest
//   s + bias: the best group_top_k stay (ties to the lower group)
//   the top_k largest c of those that stay (ties to the lower expert; ones that are not live
//   last, with weight 0), w_j = s_j, divided by their sum and scaled
//
// The selection is that of scores formed and compared in 64 bits: in a prompt of 16384 tokens some pair
// of scores at the edge of a selection lies closer than 32 bits resolve, and the choice would depend
// on how exp rounds there.  Such tokens are few, so scores are formed in fp32 first, to a known
// error: a token whose cuts (between the last expert taken and the first left, the same of groups)
// are wider than that is done, the others (one in 2400 at 256 sigmoid scores) are selected again in
// 64 bits.  Where c is the logit itself nothing is rounded, and ties are ties.  The weights are formed in
// 64 bits, by the lanes that hold them, and rounded once.  Every step is a chain of one wave: the
// number of its instructions is the time.
#pragma once
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

// What cuts must be wider than, times 2 + the largest |bias| of a live expert (one that is not live is not compared: with
// its infinite bias every token would be close, 16384 x 256 44 us instead of 20): the error of the difference of two sums of
// two scores in fp32, the bias's addition (2^-24 of 1 + |bias|) included.  A sigmoid s from exp_near (2^-22.3 of
// itself, times s (1 - s)) and a reciprocal with one step of Newton's (with 1 + e's rounding 2^-23 s) is off by less than
// 2^-22.4.  Softmax by __expf, off by (|x| + 2) 2^-23 of itself: less than 2^-20 (its sum of 256: |x| averages
// at most ln 256 there), and 2^-21 for the sums and the reciprocal.
constexpr float EDGE_SIGMOID = 1.0f / (1 << 20), EDGE_SOFTMAX = 1.0f / (1 << 17);

__device__ __forceinline__ float score_sigmoid(float x) {
    const float d = 1.0f + fminf(exp_near(-x), 1e30f), s = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, s, 1.0f), s, s);
}

__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);          // (-0 and 0 are equal)
    return (u >> 63) ? ~u : u | (1ull << 63);                            // monotone in v, above 1
}
// the same of fp32 (its keys are above 1 too), and its inverse
__device__ __forceinline__ uint32_t order_key32(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (uint64_t)dpp_u32<CTRL>((uint32_t)(v >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    return __longlong_as_double((long long)dpp_u64<CTRL>((uint64_t)__double_as_longlong(v)));
}
// largest over the wave, in every lane
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    v = max64(v, dpp_u64<0xB1>(v));
    v = max64(v, dpp_u64<0x4E>(v));
    v = max64(v, dpp_u64<0x141>(v));
    v = max64(v, dpp_u64<0x140>(v));
    return max64(max64(readlane64(v, 0), readlane64(v, 16)), max64(readlane64(v, 32), readlane64(v, 48)));
}
// sums over 16 lanes (a row) and over the wave, in every lane of it
__device__ __forceinline__ double row_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = row_sum_f64(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// whether this lane's bit of a mask is set (the mask as an execution mask: no instruction)
__device__ __forceinline__ bool lane_bit(uint64_t m) { return __builtin_amdgcn_inverse_ballot_w64(m); }

__device__ __forceinline__ int group_of(const RouteRule &r, int e) { return min((e * r.group_inv) >> 16, r.n_groups - 1); }

// a >= b: the two largest of a group's values so far, joined with another part of the group's
__device__ __forceinline__ void join_two(double &a, double &b, double a2, double b2) {
    b = fmax(fmax(b, b2), fmin(a, a2));
    a = fmax(a, a2);
}
__device__ __forceinline__ void join_two(uint32_t &a, uint32_t &b, uint32_t a2, uint32_t b2) {
    b = max(max(b, b2), min(a, a2));
    a = max(a, a2);
}

// The selection by 64-bit scores, as bit masks (sel[i] bit l: expert l + 64 i).  on: the logit is live; live: the
// bias too.
__device__ __forceinline__ void select64(const RouteRule &r, const float (&v)[4], const bool (&on)[4], const bool (&live)[4],
                                         float top, int E, int K, double *scratch, uint64_t (&sel)[4]) {
    const int lane = threadIdx.x & 63;
    double s[4], z = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (softmax, an infinite largest logit: 1 for those, 0 for the others)
        if (r.sigmoid) s[i] = on[i] ? 1.0 / (1.0 + exp(-(double)v[i])) : 0.0;
        else s[i] = !on[i] ? 0.0 : v[i] == top ? 1.0 : exp((double)v[i] - (double)top);
        z += s[i];
    }
    if (!r.sigmoid) {
        z = wave_sum_f64(z);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
    }
    uint64_t key[4];                                         // 1: not live, 0: no candidate
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        double c = (double)v[i], g = s[i];
        if (r.bias && e < E) c = g = s[i] + (double)r.bias[e];
        key[i] = e >= E ? 0ull : live[i] ? order_key64(c) : 1ull;
        if (r.n_groups > 1 && e < E) scratch[e] = !live[i] ? -__builtin_inf() : r.group_top2 ? g : c;
    }
    if (r.n_groups > 1) {
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int q = 1 << r.group_shift, g = lane >> r.group_shift;
        double a = -__builtin_inf(), b = a;
        if (g < r.n_groups)
            for (int j = lane & (q - 1); j < r.group_size; j += q) join_two(a, b, scratch[g * r.group_size + j], -__builtin_inf());
        for (int o = 1; o < q; o <<= 1) join_two(a, b, __shfl_xor(a, o, 64), __shfl_xor(b, o, 64));
        const uint64_t gk = order_key64(r.group_top2 && b > -__builtin_inf() ? a + b : a);
        int rank = 0;
        for (int j = 0; j < r.n_groups; ++j) {
            const uint64_t o = readlane64(gk, j << r.group_shift);
            rank += o > gk || (o == gk && j < g);
        }
        const uint64_t kept = __ballot(g < r.n_groups && rank < r.group_k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!((kept >> (group_of(r, lane + 64 * i) << r.group_shift)) & 1)) key[i] = 0ull;
    }
    // top_k rounds, each taking the largest key, the lowest expert among equal ones
#pragma unroll
    for (int i = 0; i < 4; ++i) sel[i] = 0;
    for (int n = 0; n < K; ++n) {
        const uint64_t m = wave_max_u64(max64(max64(key[0], key[1]), max64(key[2], key[3])));
        bool done = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t at = done ? 0ull : __ballot(key[i] == m);
            const uint64_t one = at & (0ull - at);
            sel[i] |= one;
            if (lane_bit(one)) key[i] = 0ull;
            done = done || at != 0;
        }
    }
}

// What a token's selection leaves to its weights.
struct Chosen {
    int idx;                                                 // lanes j < K: the j-th expert in ascending id
    float x;                                                 // and its logit (-infinity: weight 0)
    float top;                                               // the largest live logit (softmax)
    double z;                                                // sum of exp(l - top) (softmax without renorm; else 0)
};

// The bias of experts lane + 64 i (not used without one): loaded before the logits are waited for.
__device__ __forceinline__ void load_bias(const RouteRule &r, int E, float (&bias)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = r.bias ? r.bias[min((int)(threadIdx.x & 63) + 64 * i, E - 1)] : 0.0f;
}

// v[i]: the logit of expert lane + 64 i (ignored for ids >= E), bias from load_bias.  W: waves of the workgroup that may be
// in here at once (wave w uses slot w % W); scratch: E doubles of LDS for this wave, needed (with
// groups) until the selection is done.
template <int W>
__device__ __forceinline__ Chosen wave_choose(const RouteRule &r, const float (&v)[4], const float (&bias)[4], int E, int K,
                                              double *scratch) {
    __shared__ int rs_idx[W][16];
    __shared__ float rs_v[W][16];
    const int lane = threadIdx.x & 63, wv = (threadIdx.x >> 6) % W;
    const uint64_t lt = (1ull << lane) - 1;
    const float NONE = -__builtin_inff();
    bool on[4], live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) live[i] = on[i] = lane + 64 * i < E && v[i] > NONE;
    const float unit = r.sigmoid ? EDGE_SIGMOID : EDGE_SOFTMAX;
    float c[4], g[4], edge = 2.0f * unit, top = 0.0f;        // c: for the selection, g: for the groups
    if (!r.sigmoid) {
        uint32_t mk = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) mk = max(mk, on[i] ? order_key32(v[i]) : 0u);
        top = key_value(wave_max_bcast(mk));
    }
    // fp32 scores where they are compared (rather than logits)
    const bool scored = r.bias || (r.n_groups > 1 && r.group_top2);
    if (scored) {
        if (r.sigmoid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = score_sigmoid(v[i]);
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = !on[i] ? 0.0f : v[i] == top ? 1.0f : __expf(v[i] - top);
                z += g[i];
            }
            z = __builtin_amdgcn_rcpf(wave_sum(z));
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] *= z;
        }
        if (r.bias) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                live[i] = live[i] & (bias[i] > NONE);
                m = max(m, __float_as_uint(live[i] ? bias[i] : 0.0f) & 0x7fffffffu);
                c[i] = g[i] = g[i] + bias[i];
            }
            edge = unit * (2.0f + __uint_as_float(wave_max_bcast(m)));   // (infinity: no cut is wide enough)
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = g[i] = v[i];
    }
    uint32_t key[4];                                         // 1: not live, 0: no candidate
#pragma unroll
    for (int i = 0; i < 4; ++i) key[i] = lane + 64 * i >= E ? 0u : live[i] ? order_key32(c[i]) : 1u;
    bool close = false;                                      // a cut is not wide enough to be sure
    if (r.n_groups > 1) {
        // (as keys: 1 for experts that are not live; the experts' own where a group's values are theirs)
        uint32_t *sc = (uint32_t *)scratch;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 64 * i < E) sc[lane + 64 * i] = r.bias || !r.group_top2 ? key[i] : live[i] ? order_key32(g[i]) : 1u;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // 2^group_shift lanes per group look through its experts for the two largest
        const int q = 1 << r.group_shift, gr = lane >> r.group_shift;
        uint32_t a = 1u, b = 1u;
        if (gr < r.n_groups)
            for (int j = lane & (q - 1); j < r.group_size; j += q) join_two(a, b, sc[gr * r.group_size + j], 1u);
        if (q > 1) join_two(a, b, dpp_u32<0xB1>(a), dpp_u32<0xB1>(b));
        if (q > 2) join_two(a, b, dpp_u32<0x4E>(a), dpp_u32<0x4E>(b));
        if (q > 4) join_two(a, b, dpp_u32<0x141>(a), dpp_u32<0x141>(b));
        if (q > 8) join_two(a, b, dpp_u32<0x140>(a), dpp_u32<0x140>(b));
        if (q > 16) join_two(a, b, (uint32_t)__shfl_xor((int)a, 16, 64), (uint32_t)__shfl_xor((int)b, 16, 64));
        const uint32_t gk = r.group_top2 && b > 1u ? order_key32(key_value(a) + key_value(b)) : a;
        int rank = 0;
        for (int j = 0; j < r.n_groups; ++j) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, j << r.group_shift);
            rank += o > gk || (o == gk && j < gr);
        }
        const bool stays = gr < r.n_groups && rank < r.group_k;
        const uint64_t kept = __ballot(stays);
        if (scored) {
            const uint32_t worst = ~wave_max_bcast(stays ? ~gk : 0u), next = wave_max_bcast(gr < r.n_groups && !stays ? gk : 1u);
            close = next > 1u && !(key_value(worst) - key_value(next) > edge);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!((kept >> (group_of(r, lane + 64 * i) << r.group_shift)) & 1)) key[i] = 0u;
        // (the scratch is read before select64 writes it: one wave, in order)
    }
    // the top_k-th largest key T, counting repeats: each lane's four in order, rounds that take every
    // head equal to the largest
    uint32_t q0 = max(key[0], key[1]), q1 = min(key[0], key[1]), q2 = max(key[2], key[3]), q3 = min(key[2], key[3]);
    {
        const uint32_t h0 = max(q0, q2), l0 = min(q0, q2), h1 = max(q1, q3), l1 = min(q1, q3);
        q0 = h0;
        q1 = max(l0, h1);
        q2 = min(l0, h1);
        q3 = l1;
    }
    uint32_t T;
    for (int left = K;;) {
        T = wave_max_bcast(q0);
        const bool pop = q0 == T;
        left -= __popcll(__ballot(pop));
        q0 = pop ? q1 : q0;
        q1 = pop ? q2 : q1;
        q2 = pop ? q3 : q2;
        q3 = pop ? 0u : q3;
        if (left <= 0) break;
    }
    uint64_t gt[4], eq[4], sel[4];
    int need = K, ties = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        gt[i] = __ballot(key[i] > T);
        eq[i] = __ballot(key[i] == T);
        need -= __popcll(gt[i]);
        ties += __popcll(eq[i]);
    }
    if (r.bias && __builtin_amdgcn_readfirstlane((int)T) != 1) {         // (without one c is exact)
        const uint32_t N = wave_max_bcast(q0);               // the next one
        close |= ties > need || (N > 1u && !(key_value(T) - key_value(N) > edge));
    }
    if (__builtin_amdgcn_readfirstlane((int)close)) {
        select64(r, v, on, live, top, E, K, scratch, sel);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // of the ties the lowest `need`
            const int n = __popcll(eq[i]);
            sel[i] = gt[i] | (n <= need ? eq[i] : __ballot(lane_bit(eq[i]) && __popcll(eq[i] & lt) < need));
            need = max(need - n, 0);
        }
    }
    int base = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (lane_bit(sel[i])) {
            const int p = base + __popcll(sel[i] & lt);
            rs_idx[wv][p] = lane + 64 * i;
            rs_v[wv][p] = live[i] ? v[i] : NONE;
        }
        base += __popcll(sel[i]);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    Chosen out;
    out.idx = lane < K ? rs_idx[wv][lane] : 0;
    out.x = lane < K ? rs_v[wv][lane] : NONE;
    out.top = top;
    out.z = 0.0;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (!r.renorm && !r.sigmoid) {                           // softmax over every live expert
#pragma unroll
        for (int i = 0; i < 4; ++i) out.z += !on[i] ? 0.0 : v[i] == top ? 1.0 : exp((double)v[i] - (double)top);
        out.z = wave_sum_f64(out.z);
    }
    return out;
}

// The weight of a lane's logit x, over the 16 lanes of a token (every lane of them comes here).
__device__ __forceinline__ float row_weight(const RouteRule &r, float x, float top, double z) {
    const double d = r.sigmoid ? -(double)x : (double)x - (double)top;
    double w = exp(d), sum = 1.0;
    if (r.sigmoid) w = 1.0 / (1.0 + w);
    else if (x == top) w = 1.0;                              // (an infinite one too)
    if (!(x > -__builtin_inff())) w = 0.0;
    if (r.renorm) sum = row_sum_f64(w);
    else if (!r.sigmoid) sum = z;
    // (divided first: scale / sum overflows where the selected scores are all below 2^-1024 or so)
    return sum > 0.0 ? (float)(w / sum * (double)r.scale) : 0.0f;
}

// Both: lanes j < K return the j-th selected expert in ascending id and its weight.
template <int W>
__device__ __forceinline__ TopkOut wave_select(const RouteRule &r, const float (&v)[4], const float (&bias)[4], int E, int K,
                                               double *scratch) {
    const Chosen c = wave_choose<W>(r, v, bias, E, K, scratch);
    TopkOut out;
    out.idx = c.idx;
    out.w = 0.0f;
    if ((threadIdx.x & 63) < 16) out.w = row_weight(r, c.x, c.top, c.z);
    return out;
}

}  // namespace

}  // namespace qs
