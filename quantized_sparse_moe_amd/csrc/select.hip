// select.hip -- experts and weights of tokens whose router logits are given (moe_select): one
// wave per token over rule.h's selection, then the weights of a workgroup's tokens in one wave.
//
// Bound by the selection's own instructions, some 590 vector ones a token at 256 experts in 8 biased groups
// (top-8: 18 a round; 44 to rank the groups; 30 cycles' worth of exponentials): 16384 tokens take 20 us,
// where their 18 MB would pass in 3.7; 60 experts of softmax 11, one token 4.1 (a launch and a chain).
// Two tokens a wave, 32 lanes each, take 29: what each lane does for twice as many experts outweighs the
// shorter reductions.
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
    __shared__ double scratch[SW][256], s_z[SW];
    __shared__ float s_x[SW][16], s_top[SW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * SW, t = t0 + wave;
    if (t < a.T) {
        float v[4], bias[4];
        load_bias(a.rule, a.E, bias);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = min(lane + 64 * i, a.E - 1);
            if constexpr (DT == MOE_F32) v[i] = ((const float *)a.logits + t * a.ld)[o];
            else if constexpr (DT == MOE_F16) v[i] = f16_to_f32(((const uint16_t *)a.logits + t * a.ld)[o]);
            else v[i] = bf16_to_f32(((const uint16_t *)a.logits + t * a.ld)[o]);
        }
        const Chosen c = wave_choose<SW>(a.rule, v, bias, a.E, a.K, scratch[wave]);
        if (lane < a.K) a.idx[t * a.K + lane] = c.idx;
        if (lane < 16) s_x[wave][lane] = c.x;
        if (lane == 0) {
            s_top[wave] = c.top;
            s_z[wave] = c.z;
        }
    }
    // the weights of all four tokens in one wave, 16 lanes each
    __syncthreads();
    const int row = lane >> 4, j = lane & 15;
    if (wave == 0 && t0 + row < a.T) {
        const float w = row_weight(a.rule, s_x[row][j], s_top[row], s_z[row]);
        if (j < a.K) a.w[(t0 + row) * a.K + j] = w;
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
