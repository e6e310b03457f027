// select.hip -- experts and weights of tokens whose router logits are given (moe_select): one
// wave per token over rule.h's selection, logits read once, 16-byte results of a token together.
#include "rule.h"

namespace qs {

namespace {

constexpr int SW = 4;                       // waves (tokens) per workgroup

struct SelectArgs {
    RouteRule rule;
    const void *logits;
    int64_t T, ld;
    int E, K;
    int32_t *idx;
    float *w;
};

template <int DT>
__global__ __launch_bounds__(64 * SW) void k_select(SelectArgs a) {
    __shared__ double scratch[SW][256];
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * SW + (threadIdx.x >> 6);
    if (t >= a.T) return;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        v[i] = 0.0f;
        if (e < a.E) {
            if constexpr (DT == MOE_F32) v[i] = ((const float *)a.logits)[t * a.ld + e];
            else if constexpr (DT == MOE_F16) v[i] = f16_to_f32(((const uint16_t *)a.logits)[t * a.ld + e]);
            else v[i] = bf16_to_f32(((const uint16_t *)a.logits)[t * a.ld + e]);
        }
    }
    const TopkOut tk = wave_select<SW>(a.rule, v, a.E, a.K, scratch[threadIdx.x >> 6]);
    if (lane < a.K) {
        a.idx[t * a.K + lane] = tk.idx;
        a.w[t * a.K + lane] = tk.w;
    }
}

}  // namespace

hipError_t launch_select(const RouteRule &rule, const void *logits, int dtype, int64_t T, int E, int64_t ld, int K,
                         int32_t *idx, float *w, hipStream_t s) {
    SelectArgs a;
    a.rule = rule;
    a.logits = logits;
    a.T = T;
    a.ld = ld;
    a.E = E;
    a.K = K;
    a.idx = idx;
    a.w = w;
    const dim3 grid((unsigned)((T + SW - 1) / SW));
    if (dtype == MOE_F32) hipLaunchKernelGGL(k_select<MOE_F32>, grid, dim3(64 * SW), 0, s, a);
    else if (dtype == MOE_F16) hipLaunchKernelGGL(k_select<MOE_F16>, grid, dim3(64 * SW), 0, s, a);
    else hipLaunchKernelGGL(k_select<MOE_BF16>, grid, dim3(64 * SW), 0, s, a);
    return hipGetLastError();
}

}  // namespace qs
