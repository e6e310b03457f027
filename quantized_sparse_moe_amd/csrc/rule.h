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
// Scores are formed and compared in 64 bits: in a prompt of 16384 tokens some pair of scores at
// the edge of a selection lies closer than 32 bits resolve, and the selection would depend on
// how exp rounds there.  Every step is a chain of one wave, so its length is its time.
#pragma once
#include "common.h"
#include "internal.h"

namespace qs {

namespace {

__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);          // (-0 and 0 are equal)
    return (u >> 63) ? ~u : u | (1ull << 63);                            // monotone in v, above 1
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (uint64_t)dpp_u32<CTRL>((uint32_t)(v >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)v);
}
// largest over the wave, in every lane
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    v = max64(v, dpp_u64<0xB1>(v));
    v = max64(v, dpp_u64<0x4E>(v));
    v = max64(v, dpp_u64<0x141>(v));
    v = max64(v, dpp_u64<0x140>(v));
    return max64(max64(readlane64(v, 0), readlane64(v, 16)), max64(readlane64(v, 32), readlane64(v, 48)));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// v[i]: the logit of expert lane + 64 i (ignored for ids >= E).  On return lanes j < K hold the
// j-th selected expert in ascending id and its weight.  W: waves of the workgroup that may be
// in here at once (wave w uses slot w % W); scratch: E doubles of LDS for this wave, needed (with
// groups) until the selection is done.
template <int W>
__device__ __forceinline__ TopkOut wave_select(const RouteRule &r, const float (&v)[4], int E, int K, double *scratch) {
    __shared__ int rs_idx[W][16];
    __shared__ float rs_w[W][16];
    const int lane = threadIdx.x & 63, wv = (threadIdx.x >> 6) % W;
    const uint64_t lt = (1ull << lane) - 1;
    bool live[4];
    double s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) live[i] = lane + 64 * i < E && v[i] > -__builtin_inff();
    if (r.sigmoid) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = live[i] ? 1.0 / (1.0 + exp(-(double)v[i])) : 0.0;
    } else {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, live[i] ? order_key(v[i]) : 0u);
        m = wave_max_bcast(m);
        const float top = __uint_as_float((m & 0x80000000u) ? (m & 0x7fffffffu) : ~m);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (an infinite largest logit: 1 for those, 0 for the others)
            s[i] = !live[i] ? 0.0 : v[i] == top ? 1.0 : exp((double)v[i] - (double)top);
            z += s[i];
        }
        z = wave_sum_f64(z);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
    }
    // selection values, and their keys: 1 for experts that are not live, 0 for none at all
    double c[4];
    uint64_t key[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        c[i] = (double)v[i];
        double g = s[i];
        if (r.bias && e < E) {
            c[i] = g = s[i] + (double)r.bias[e];
            live[i] = live[i] && g > -__builtin_inf();
        }
        key[i] = e >= E ? 0ull : live[i] ? order_key64(c[i]) : 1ull;
        if (r.n_groups > 1 && e < E) scratch[e] = !live[i] ? -__builtin_inf() : r.group_top2 ? g : c[i];
    }
    if (r.n_groups > 1) {
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // 2^group_shift lanes per group look through its experts for the two largest
        const int q = 1 << r.group_shift, g = lane >> r.group_shift;
        double a = -__builtin_inf(), b = a;
        if (g < r.n_groups)
            for (int j = lane & (q - 1); j < r.group_size; j += q) {
                const double t = scratch[g * r.group_size + j];
                b = fmax(b, fmin(a, t));
                a = fmax(a, t);
            }
        for (int o = 1; o < q; o <<= 1) {
            const double a2 = __shfl_xor(a, o, 64), b2 = __shfl_xor(b, o, 64);
            b = fmax(fmax(b, b2), fmin(a, a2));
            a = fmax(a, a2);
        }
        const uint64_t gk = order_key64(r.group_top2 && b > -__builtin_inf() ? a + b : a);
        int rank = 0;
        for (int j = 0; j < r.n_groups; ++j) {
            const uint64_t o = readlane64(gk, j << r.group_shift);
            rank += o > gk || (o == gk && j < g);
        }
        const uint64_t kept = __ballot(g < r.n_groups && rank < r.group_k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ge = min((int)(((lane + 64 * i) * r.group_inv) >> 16), r.n_groups - 1);
            if (!((kept >> (ge << r.group_shift)) & 1)) key[i] = 0ull;
        }
    }
    // top_k rounds, each taking the largest key, the lowest expert among equal ones
    uint64_t sel[4] = {0, 0, 0, 0};
    for (int n = 0; n < K; ++n) {
        const uint64_t m = wave_max_u64(max64(max64(key[0], key[1]), max64(key[2], key[3])));
        bool done = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t at = done ? 0ull : __ballot(key[i] == m);
            const uint64_t one = at & (0ull - at);
            sel[i] |= one;
            if ((one >> lane) & 1) key[i] = 0ull;
            done = done || at != 0;
        }
    }
    double sum = 1.0;
    if (r.renorm) {
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) part += ((sel[i] >> lane) & 1) && live[i] ? s[i] : 0.0;
        sum = wave_sum_f64(part);
    }
    const double f = sum > 0.0 ? (double)r.scale / sum : 0.0;
    int base = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((sel[i] >> lane) & 1) {
            const int p = base + __popcll(sel[i] & lt);
            rs_idx[wv][p] = lane + 64 * i;
            rs_w[wv][p] = live[i] ? (float)(s[i] * f) : 0.0f;
        }
        base += __popcll(sel[i]);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    TopkOut out;
    out.idx = lane < K ? rs_idx[wv][lane] : 0;
    out.w = lane < K ? rs_w[wv][lane] : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return out;
}

}  // namespace

}  // namespace qs
