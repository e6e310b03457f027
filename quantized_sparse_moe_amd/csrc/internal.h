// internal.h -- argument blocks passed from the host entry points (api.cpp) to the
// kernel launchers of libqsmoe.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qsmoe.h"

namespace qs {

struct QMat {                      // one stack of affine-quantized matrices
    const uint8_t *codes;
    const uint16_t *scales;        // fp16 bits
    const uint16_t *biases;        // fp16 bits
    int64_t stride;                // rows between matrices
};

// A routing rule (moe_router_rule; selection in rule.h), as the kernels read it
struct RouteRule {
    const float *bias;             // [E] added to the scores for the selection, or null
    float scale;                   // of the weights
    int sigmoid, renorm;
    int n_groups, group_k, group_top2, group_size;
    int group_shift;               // 2^group_shift lanes look through a group: the most with n_groups of them in a wave
    int group_inv;                 // 65536 / group_size, rounded up: e * group_inv >> 16 is e / group_size for e < 256
};

struct Layer {
    int H, I, E, K, bits;          // hidden, inter, experts, top_k, code bits
    const uint16_t *router_w;      // bf16 [E][H]
    const float *router_bias;      // [E] or null
    QMat gate, up, down;
    int has_shared;
    QMat s_gate, s_up, s_down;
    int sb_bf16;                   // scales and biases are bf16 (else fp16)
    const uint16_t *shared_gate_w; // bf16 [H]: shared output scaled by sigmoid(g . x); or null
    int mx4;                       // MX4 tiles instead of affine codes (scales: E8M0 tiles, no biases)
    int ruled;                     // experts are selected by `rule` (else: the largest logits, softmax over them)
    RouteRule rule;
};

// -------------------------------------------------------------------- decode T = 1
// Decode state at the start of every workspace: zero before the first call, then kept
// by the library between calls (call generation, completion counters, and the tagged
// logit and h words the workgroups of one call hand to each other).
constexpr size_t WS_CTL_BYTES = 2 * 1024 * 1024;

struct DecodeBufs {
    uint32_t *ctl;                 // WS_CTL_BYTES of decode state
};

// the workspace's error word (word 0 of the state) copied to *out, then optionally cleared
hipError_t launch_ws_status(uint32_t *ctl, uint32_t *out, bool clear, hipStream_t s);

hipError_t launch_decode_layer(const Layer &L, const uint16_t *x, const DecodeBufs &b, void *y,
                               int y_dtype, int32_t *out_idx, float *out_w, hipStream_t s);
// T = 2 .. 4 tokens in one launch, the routed experts read once for all of them
constexpr int SMALL_TMAX = 4;   // tokens of one small-batch decode launch
bool decode_small_eligible(const Layer &L, int64_t T);
hipError_t launch_decode_small_layer(const Layer &L, const uint16_t *x, int64_t T, const DecodeBufs &b, void *y,
                                     int y_dtype, int32_t *out_idx, float *out_w, hipStream_t s);
hipError_t launch_decode_small_route(const Layer &L, const uint16_t *x, int64_t T, const DecodeBufs &b,
                                     int32_t *out_idx, float *out_w, hipStream_t s);
hipError_t launch_decode_route(const Layer &L, const uint16_t *x, const DecodeBufs &b,
                               int32_t *out_idx, float *out_w, hipStream_t s);

// ------------------------------------------------------------------- prefill T >= 2
constexpr int ROUTER_TOKENS = 16;  // tokens per router workgroup (= one binning block)
constexpr int GEMM_MT = 10;        // 16-row MFMA subtiles per GEMM tile (even)
constexpr int GEMM_BM = 16 * GEMM_MT;

struct Tile {                      // one row block of one expert bin
    int32_t expert;                // 0..E-1, or E for the shared expert
    int32_t row0;                  // first row in the h / perm position space
    int32_t nrows;                 // 1..GEMM_BM
    int32_t pad;
};

// fp16 operands of the grouped path carry power-of-two range scales: x 2^a per token
// (a in xexp), h 2^e per (row, 128-column block) (e in hexp, block-major: the exponents
// of one block for all T*K + T rows together), slot rows 2^e per (row, 64-column block)
// (sexp, block-major as well, rows padded to a multiple of 16)
constexpr int HEXP_STRIDE = 16;    // inter <= 2048: at most 16 blocks of 128 columns
// a state word read by the grouped GEMM: nonzero gives every h block the scale that puts
// its largest value in [2^14, 2^15) instead of the shared one (0 for ordinary blocks), so
// that nearly every down tile must rescale (set only by tests of that rescale)
constexpr int CTL_HBLOCK_EXACT = 33;

struct PrefillBufs {
    uint16_t *x16;                 // [T][H] fp16 x 2^a, columns permuted per 8-group (code order)
    uint32_t *xmax;                // [T][8] largest |x| per token and logits expert block
    int32_t *xexp;                 // [T] the a of each token's x16 row
    float *logits;                 // [T][E] router logits
    int32_t *idx;                  // [T][K]
    float *w;                      // [T][K]
    int32_t *blkcnt;               // [nblk][E]  assignments per (16-token block, expert)
    int32_t *blkoff;               // [nblk][E]  first position of that block's rows in the expert bin
    int32_t *expert_off;           // [E+1]
    int32_t *perm;                 // [T*K]      position -> t*K + j
    Tile *tiles;                   // [max_tiles] routed full, routed partial, then shared tiles
    int32_t *ntiles;               // [3] routed tiles, routed + shared tiles, and a flag the
                                   // down pass sets when some slot block has a nonzero scale
    int32_t *tile_done;            // [max_tiles] gate/up column blocks finished per tile
    uint32_t *ctl;                 // the workspace's state region (word 0: bounded-wait error flag)
    uint16_t *h;                   // [(T*K + T)][I] fp16, columns permuted per 8-group
    int8_t *hexp;                  // [HEXP_STRIDE][T*K + T]
    uint16_t *slot;                // [T*K + T][H] fp16: w_j * o_j per (token, slot), then shared o
    int8_t *sexp;                  // [H / 64][sexp_rows(T, K)]
    float *sgate;                  // [T] shared-expert gate sigmoid(g . x_t) (gated layers)
};

__host__ __device__ inline int64_t sexp_rows(int64_t T, int K) { return (T * K + T + 15) / 16 * 16; }
int64_t prefill_max_routed_tiles(int64_t T, int K, int E);
int64_t prefill_max_tiles(int64_t T, int K, int E);

hipError_t launch_prefill_router(const Layer &L, const uint16_t *x, int64_t T,
                                 const PrefillBufs &b, bool write_x16, int32_t *out_idx,
                                 float *out_w, hipStream_t s);
hipError_t launch_prefill_binning(const Layer &L, int64_t T, const PrefillBufs &b, hipStream_t s);
hipError_t launch_prefill_gemms(const Layer &L, int64_t T, const PrefillBufs &b, void *y,
                                int y_dtype, hipStream_t s);

// y from the slot rows (both kinds of experts)
hipError_t launch_prefill_combine(const Layer &L, int64_t T, const PrefillBufs &b, void *y, int y_dtype, hipStream_t s);

// --------------------------------------------------------------------------- Q8_0
int n_compute_units();   // of the current device, queried once
hipError_t launch_q8_gemv(const uint8_t *tiles, int64_t N, int64_t K, const uint16_t *x,
                          void *y, int y_dtype, hipStream_t s);
hipError_t launch_q8_quantize_x(const uint16_t *x, int64_t K, int8_t *xq, uint16_t *xd, hipStream_t s);
hipError_t launch_q8_gemv_q8x(const uint8_t *tiles, int64_t N, int64_t K, const int8_t *xq, const uint16_t *xd,
                              const uint16_t *x, void *y, int y_dtype, hipStream_t s);
hipError_t launch_q8_pack(const uint8_t *rows, int64_t N, int64_t K, uint8_t *tiles,
                          hipStream_t s);

// ---------------------------------------------------------------------------- MX4
// column steps of 128 and groups of four steps of a row of K values (layouts: mx4.h)
__host__ __device__ inline int64_t mx4_steps(int64_t K) { return (K + 127) / 128; }
__host__ __device__ inline int64_t mx4_quads(int64_t K) { return (K + 511) / 512; }
hipError_t launch_mx4_quantize(const void *x, int dtype, int64_t rows, int64_t K, int64_t ldx, int layout,
                               uint8_t *codes, uint8_t *scales, hipStream_t s);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, int layout,
                                 void *y, int dtype, int64_t ldy, hipStream_t s);
hipError_t launch_mx4_pack(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, uint8_t *tc,
                           uint8_t *ts, hipStream_t s);
size_t mx4_gemm_ws(int64_t T, int64_t N, int64_t K);      // bytes of workspace of launch_mx4_gemm
hipError_t launch_mx4_gemm(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint16_t *x, int64_t T,
                           int64_t ldx, void *y, int y_dtype, int64_t ldy, uint8_t *ws, hipStream_t s);
hipError_t launch_mx4_gemm_mx4x(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint8_t *xc,
                                const uint8_t *xs, int64_t T, void *y, int y_dtype, int64_t ldy, uint8_t *ws,
                                hipStream_t s);

// The MoE layer with MX4 experts (mx4_moe.hip), MX_TMAX tokens a pass.  Its counters lie in
// the workspace's state region behind the affine kernels' words: zero before the first call,
// and put back to zero by every call.
constexpr int MX_TMAX = 128, MX_SHARES = 8;
constexpr int MX_ITEMS = 256 + MX_TMAX * 16 / 16;         // of the work list: experts, and one per 16 tokens
constexpr size_t MX_CNT_OFF = WS_CTL_BYTES - 4096;        // bytes
constexpr int MX_CNT_DOWN = 16;                           // counters before: route's
struct MxBufs {
    uint32_t *ctl;                 // the workspace's state region
    uint32_t *cnt;                 // completion counters: [i] token tile i of route, [MX_TMAX / 16]
                                   // its tiles, [MX_CNT_DOWN + i] the i-th output rows of down
    float *logits;                 // [T][E + 1] (column E: the shared expert's gate)
    int32_t *idx;                  // [T][K]
    float *w;                      // [T][K]
    int32_t *act;                  // [MX_ITEMS] the work list: up to 16 tokens of a chosen expert each
    int32_t *nact;                 // [1] its length
    int16_t *pos;                  // [E][MX_TMAX] per chosen expert its tokens' rows of h (t K + j), in order
    uint16_t *h;                   // [T*K + T][2 x I up to 128] bf16: w silu(g) u as hi and lo
    float *part;                   // [MX_SHARES][T][H] the down shares' sums
};
hipError_t launch_mx_layer(const Layer &L, const uint16_t *x, int64_t T, const MxBufs &b, void *y, int y_dtype,
                           int32_t *out_idx, float *out_w, bool route_only, hipStream_t s);

// The expert products of a prompt (mx4_group.hip), between the binning and the combine:
// b.h holds bf16 pairs there, [T*K + T][hi, lo][I].
hipError_t launch_mx_group(const Layer &L, const uint16_t *x, int64_t T, const PrefillBufs &b, hipStream_t s);

// ---------------------------------------------------------- around the layer's blocks
hipError_t launch_select(const RouteRule &rule, const void *logits, int dtype, int64_t T, int E, int64_t ld, int K,
                         int32_t *idx, float *w, hipStream_t s);

struct NormArgs {
    int on, layer, dtype;          // dtype: of w and b
    float eps, offset;
    const void *w, *b;             // [H] or null
};
struct BlockNormArgs {
    const void *y, *r, *gate;      // null: absent
    void *ro, *xo;
    int dy, dr, dg, dro, dxo;      // types
    int64_t ldy, ldr, ldg, ldro, ldxo;
    NormArgs post, pre;
    int gate_cols, act;            // 1: a value per row; else elementwise
    float scale;
    int64_t T, row0;               // rows row0 .. of T (set by the launcher)
    int H;
};
hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t s);

struct LoraArgs {
    const uint16_t *a, *b;         // [n][R][K], [n][N][R] bf16
    const float *scales;           // [n] or null
    const int32_t *ranks;          // [n] or null
    const int32_t *ids;            // [T]
    const uint16_t *x;             // [T] rows, ldx apart
    const void *base;              // [T] rows of y's type, or null
    void *y;
    int32_t *perm, *sid;           // workspace: tokens ordered by adapter, and their adapters; or null
    uint16_t *v;                   // workspace: [T][parts][R] bf16, in that order
    int64_t T, ldx, ldb, ldy, N;
    int n, R, K, f32;
};
constexpr int LORA_PARTS = 3;      // bf16 parts of a value of v, at most
// whether tokens are ordered first: where reading an adapter's B once more for every tile that holds one of
// its tokens costs more than the launch (lora.hip).  Not past 65536 tokens: batches that long are prompts, whose tokens
// come in runs, and one workgroup's pass over the ids would cost these more than it gives (us of 131072 tokens not
// ordered and ordered: N = 2048, rank 16 in runs 392 and 500, mixed 1503 and 582; N = 16384, rank 32 in runs 2103 and 2217,
// mixed 6629 and 2536)
inline bool lora_ordered(int64_t T, int64_t n_adapters, int64_t N, int64_t R) {
    return n_adapters > 1 && T > 64 && T <= 65536 && (T / 16) * N * R >= 4 << 20;
}
hipError_t launch_lora(const LoraArgs &a, hipStream_t s);

// ---------------------------------------------------------------- measured ceilings
hipError_t launch_calib_read(const void *buf, int64_t bytes, uint32_t *out, hipStream_t s);
hipError_t launch_calib_mfma(int iters, int blocks, float *out, hipStream_t s);

}  // namespace qs
