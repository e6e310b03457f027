/*
 * qsmoe.h -- C ABI of the MI355X (gfx950) quantized sparse mixture-of-experts FFN
 * layer and the dense Q8_0 decode GEMV.
 *
 * Sources, cited by page title and section:
 *   [LILY]  "Optimizing on-device inference for Apple Silicon" (Perplexity blog):
 *           "Qwen creates three distinct workload shapes" (router scores 256 experts,
 *           picks eight; a shared expert processes every token), "Dequantize weights
 *           during matrix multiplication" (4-bit integer codes, one scale and bias per
 *           group of 64 weights; fp32 accumulation), "Keep expert routing on the GPU"
 *           (histogram -> prefix scan -> scatter -> block map, no CPU round trip),
 *           "Match tile size to expert load", "Optimize the single-row weight path",
 *           "Reduce intermediate and state traffic" (fused expert input projections
 *           with the gated activation; fused output projection with the routing score
 *           and the shared-expert result).
 *   [OMLX]  "oMLX MoE gate/up fusion: qwen35_moe_gate_up implementation analysis"
 *           (pwwt.cn): "Fusion principle" ([gate; up] concatenated along the output
 *           axis is bit-identical to separate gate and up), "_can_fuse" (eligibility:
 *           equal group size, bits, shapes and dtypes).
 *   [EMBER] "Ember packed Q8 decode" (voidwest.dev): Q8_0 blocks ([fp16 scale][32 x
 *           int8]) and the packed 16-row tile (eight 64-byte groups + 16 fp16 scales,
 *           544 bytes); a reusable decode workspace instead of per-layer temporaries.
 *
 * General conventions
 *   - Every tensor pointer is a DEVICE pointer (HBM) unless stated otherwise; every
 *     call only enqueues work on `stream` (a hipStream_t; NULL = the null stream) and
 *     never synchronizes with the host.
 *   - The caller owns and frees every buffer.  The library allocates no device memory
 *     and keeps no state between calls.  Descriptors are read during the call only.
 *   - All validation runs on the host before the first enqueue; on any error nothing
 *     is enqueued and the outputs are untouched.  No exception or abort crosses the ABI.
 *   - Results are bit-deterministic for equal inputs, device and build: there are no
 *     floating-point atomics and every reduction has a fixed order.
 *   - Calls on different streams with distinct workspaces and outputs may run
 *     concurrently.
 */
#ifndef QSMOE_H
#define QSMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 3

typedef int32_t moe_status;
#define MOE_OK               0
#define MOE_ERR_INVALID     -1   /* NULL / misaligned pointer, negative size, bad enum   */
#define MOE_ERR_UNSUPPORTED -2   /* shape or format outside the supported limits         */
#define MOE_ERR_WORKSPACE   -3   /* workspace NULL, misaligned or too small              */
#define MOE_ERR_DEVICE      -4   /* a HIP launch failed (hipGetLastError)                */

/* Bits of the workspace error word (read with moe_workspace_status).  Every wait of one
 * workgroup for another inside a launch is bounded; a wait that gives up sets its bit and
 * lets the kernel finish, so the grid always drains, and that call's outputs are not to be
 * trusted.  A correct call on a device that runs the whole grid sets no bit. */
#define MOE_WS_ERR_DECODE_WAIT 1u   /* a one-launch decode kernel (T <= 8), or the first launch of an
                                       MX4 layer of up to 4 tokens, gave up a wait        */
#define MOE_WS_ERR_GEMM_WAIT   2u   /* a grouped-GEMM down tile gave up waiting for its h  */

/* element types */
#define MOE_BF16 0
#define MOE_F16  1
#define MOE_F32  2
#define MOE_E8M0 3   /* scale_dtype only: an MX4 layer */

/*
 * A stack of affine-quantized matrices, each [rows][cols], quantized in groups of
 * 64 consecutive columns of one row ([LILY] "Dequantize weights during matrix
 * multiplication"):  W[r][c] = scale[r][c/64] * q[r][c] + bias[r][c/64]
 * with an unsigned integer code q in [0, 2^bits).
 *   codes   uint8; matrix e, row r starts at byte (e*mat_stride + r) * cols*bits/8.
 *           4-bit codes: column 2i in the low nibble of byte i, 2i+1 in the high.
 *   scales  fp16, [..][cols/64]; matrix e, row r at element (e*mat_stride + r)*cols/64
 *   biases  fp16, same shape and indexing as scales
 *   mat_stride  rows between consecutive matrices: `rows` for a plain stack, or
 *           2*inter when gate and up are the two halves of one fused [gate; up]
 *           stack ([OMLX] "Fusion principle"; then up.codes = gate.codes +
 *           inter*cols*bits/8 and up.scales/biases = gate.* + inter*cols/64).
 * codes must be 16-byte aligned (every row then starts 16-byte aligned, given the
 * shape limits below); scales and biases 2-byte aligned.
 */
typedef struct {
    const void *codes;
    const void *scales;
    const void *biases;
    int64_t     mat_stride;
} moe_qmat;

/*
 * One MoE FFN layer ([LILY] "Qwen creates three distinct workload shapes").
 *   router_w     [n_experts][hidden] bf16
 *   router_bias  [n_experts] fp32 added to the logits before selection, or NULL
 *   gate, up     [n_experts][inter][hidden] stacks;  down [n_experts][hidden][inter]
 *   has_shared   1: the shared expert (s_gate, s_up [inter][hidden], s_down
 *                [hidden][inter], one matrix each) processes every token with weight 1
 *                (or, with shared_gate_w, with weight sigmoid(shared_gate_w . x))
 *   scale_dtype  MOE_F16 or MOE_BF16: the format of every qmat's scales and biases
 *                (bf16 is the checkpoint format the pages print)
 *   shared_gate_w  [hidden] bf16 (16-byte aligned) or NULL; needs has_shared
 * Limits (else MOE_ERR_UNSUPPORTED): group == 64; bits in {4, 8};
 *   1 <= n_experts <= 256; 1 <= top_k <= min(n_experts, 16);
 *   hidden % 64 == 0, 64 <= hidden <= 8192; inter % 64 == 0, 64 <= inter <= 2048;
 *   (top_k + 1) * inter <= 24576 (the batch-1 kernel hands every h value of a call
 *   between workgroups through a fixed region of the workspace).
 * Every qmat needs mat_stride >= its rows (MOE_ERR_INVALID otherwise).
 *
 * MX4 layers: scale_dtype MOE_E8M0 with bits == 4 and group == 32 makes every qmat a stack
 *   of microscaled 4-bit matrices in MX4_TILES (see the mx4_ functions below; a stack is
 *   repacked as one matrix of all its rows): codes 16-byte aligned, scales 4-byte aligned,
 *   biases unused, mat_stride a multiple of 16 (for the up half of a fused [gate; up] stack
 *   codes and scales start inter/16 panels behind gate's).  The other limits hold, except
 *   the one on (top_k + 1) * inter.
 */
typedef struct {
    int32_t hidden, inter, n_experts, top_k, bits, group;
    int32_t scale_dtype;
    const void  *router_w;
    const float *router_bias;
    moe_qmat gate, up, down;
    int32_t    has_shared;
    moe_qmat s_gate, s_up, s_down;
    const void *shared_gate_w;
} moe_layer_desc;

int          moe_abi_version(void);                 /* MOE_ABI_VERSION of the library */
const char  *moe_status_string(moe_status s);   /* static string, never NULL */

/*
 * Bytes of device workspace moe_route / moe_layer_forward need for T tokens
 * (0 when T <= 0; SIZE_MAX when the descriptor is invalid).  The workspace must be
 * 256-byte aligned.  Its first 2 MiB are the state of the one-launch decode kernels
 * (T <= 8): a call counter, completion counters, tagged words the workgroups of one call
 * hand to each other, and the error word.  It must be zero before the first call that
 * uses the workspace (allocate it zero-filled) and then belongs to the library: every
 * call leaves it ready for the next one, so no clearing launch is needed per call
 * ([EMBER] "packed Q8 decode": one reusable decode workspace instead of per-layer
 * temporaries).  A caller that writes it must zero it again before the next call.  The
 * rest is scratch whose contents are undefined between calls.  Calls that share one
 * workspace must not overlap in time (issue them on one stream).  T >= 2 is processed in
 * chunks inside one call ([LILY] "Reduce intermediate and state traffic": bounded
 * intermediate buffers): this size is for chunks of MOE_PREFILL_CHUNK tokens, so it stops
 * growing there (~200 MiB for any T >= 4096 at hidden 2048, inter 512, top-8).
 */
size_t moe_workspace_size(const moe_layer_desc *d, int64_t T);

/* Default tokens per prefill chunk (T >= 2). */
#define MOE_PREFILL_CHUNK 4096

/*
 * Bytes of workspace for T tokens run in chunks of `chunk` tokens (0: the default
 * MOE_PREFILL_CHUNK; chunk >= T: unchunked; 1 counts as 2).  moe_route /
 * moe_layer_forward accept any workspace at least as large as the chunk-2 size and take
 * the largest chunk whose buffers fit in the ws_bytes they are given, so a caller that can
 * spare the memory avoids re-reading the expert weights once per chunk, and one short of
 * memory can bound it.  Chunking changes no result: every token is computed by the same
 * kernels whatever chunk it falls in, bit for bit.  SIZE_MAX for an invalid descriptor,
 * T > 2^20 or chunk < 0.
 */
size_t moe_workspace_size_chunked(const moe_layer_desc *d, int64_t T, int64_t chunk);

/*
 * Enqueues on `stream` a copy of the workspace's error word (MOE_WS_ERR_* bits, 0 when
 * every call so far completed every wait) into *status_out, a device uint32, and, when
 * `clear` is nonzero, resets the word to 0 afterwards.  ws must be a workspace of
 * ws_bytes >= 2 MiB used by moe_route / moe_layer_forward (or freshly zeroed); the call
 * is ordered with the layer calls on the same stream.
 */
moe_status moe_workspace_status(void *ws, size_t ws_bytes, uint32_t *status_out, int32_t clear,
                                void *stream);

/*
 * Router only ([LILY] "Qwen creates three distinct workload shapes"): fp32 logits
 * l[t][e] = sum_c x[t][c] * router_w[e][c] (+ router_bias[e]), the top_k largest per
 * token (exact ties to the lower expert id), and weights renormalised over the
 * selection, w_j = exp(l_j - l_max) / sum_{i in selection} exp(l_i - l_max).
 *   x        [T][hidden] bf16
 *   topk_idx [T][top_k] int32, ascending expert id within a token (written)
 *   topk_w   [T][top_k] fp32, aligned with topk_idx (written)
 *   ws       device workspace of ws_bytes >= moe_workspace_size(d, T)
 * T == 0 returns MOE_OK and enqueues nothing; T > 2^20 is MOE_ERR_UNSUPPORTED.
 */
moe_status moe_route(const moe_layer_desc *d, const void *x, int64_t T,
                       int32_t *topk_idx, float *topk_w,
                       void *ws, size_t ws_bytes, void *stream);

/*
 * The whole layer: router, top-k, (T >= 2) expert binning, fused [gate; up]
 * projection + SwiGLU h = silu(g) * u with silu(z) = z / (1 + e^-z), down
 * projection, and the combine
 *     y[t] = sum over the selected experts in ascending id of w_j * o_j  +  o_shared,
 * accumulated in fp32 in that fixed order ([LILY] "Reduce intermediate and state
 * traffic"; [OMLX] "Fusion principle").
 *   x        [T][hidden] bf16, any finite values: every fp16 operand of the kernels
 *            (x, the dequantized weights, h, the routed outputs) carries an exact
 *            power-of-two range scale, so results stay within the parity bound of
 *            an fp64 evaluation for activations, scales and biases anywhere in
 *            bf16's range, as long as the intermediate values fit in fp32
 *   y        [T][hidden], y_dtype MOE_BF16 (round-to-nearest-even) or MOE_F32
 *   topk_idx, topk_w  optional outputs as in moe_route (NULL to skip)
 * Path: T == 1 runs the batch-1 decode kernel (register dequantization on the vector
 * ALUs, fp32 intermediates); T = 2 .. 4 the same kernel design over all tokens at once,
 * each expert any token selected read once (when T * (top_k + 1) * inter <= 98496);
 * T = 5 .. 8 two such launches of ceil(T/2) and floor(T/2) tokens (when both fit);
 * larger T runs the grouped-GEMM path (MFMA on fp16 operands dequantized in registers,
 * fp32 accumulation, fp16 intermediates, each under its range scale).
 * For a given T the result does not depend on whether gate/up are fused or separate,
 * nor on the other tokens of the call (tokens are independent), bit for bit.
 * MX4 layers: up to 128 tokens run in three launches (up to 4 in two) that load a chosen
 * expert once for every 16 tokens that chose it (MFMA on bf16 operands: x as it is, the weights
 * exact, h as a bf16 pair, to 2^-17, so that an fp32 y is off by about 2e-6 of its norm); more run
 * the grouped path (the same products in tiles, weighted expert outputs in fp16 under range
 * scales before the combine, as in an affine layer: 2e-4 of y's norm, an eighth of what rounding
 * y to bf16 costs).  There a token's result does not depend on the others, bit for bit; up to
 * 128 tokens it may in its last fp32 bits (the order in which its experts are summed depends on
 * the pass's experts).  What they keep in the workspace's state follows the same rules (zero
 * before the first call, then the library's).
 */
moe_status moe_layer_forward(const moe_layer_desc *d, const void *x, int64_t T,
                               void *y, int32_t y_dtype,
                               int32_t *topk_idx, float *topk_w,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * Routing rules: other ways to choose a token's experts and weights than moe_route's.  For the
 * logits l of a token (live: above -infinity; a NaN is not):
 *   score     MOE_SCORE_SIGMOID  s_e = 1 / (1 + exp(-l_e))
 *             MOE_SCORE_SOFTMAX  s_e = exp(l_e) / sum of exp over all live experts
 *   select_bias  [n_experts] fp32 (or NULL): c_e = s_e + select_bias[e] is what experts are chosen
 *             by (their weights stay s_e); without it, the scores themselves, in the order of the logits also
 *             where 64 bits hold them equal (sigmoid above 37, softmax 745 below the largest)
 *   n_groups  groups of n_experts / n_groups consecutive experts, of which the group_top_k best stay:
 *             by the largest c of the group (MOE_GROUP_MAX) or by the sum of its two largest
 *             (MOE_GROUP_TOP2); ties go to the lower group.  1: no groups
 *   the top_k largest c of the groups that stay, ties to the lower expert id
 *   renorm    1: w_j = s_j / sum over the selected s (0 where that sum is 0 in 64 bits);  0: w_j = s_j
 *   scale     a factor on every weight (finite)
 * An expert that is not live, or whose bias is NaN or -infinity, is chosen only when nothing else
 * is left, and has weight 0; a row without a live expert has weights 0.  Scores are formed and
 * compared in 64 bits.  Limits (else MOE_ERR_UNSUPPORTED): n_groups <= 64 divides n_experts,
 * group_top_k groups hold at least top_k experts.  The rule is read during the call,
 * select_bias by the kernels.
 */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX  0
#define MOE_GROUP_TOP2 1
typedef struct {
    int32_t score, renorm;
    int32_t n_groups, group_top_k, group_score;
    float   scale;
    const float *select_bias;
} moe_router_rule;

/*
 * A rule applied to logits that are there already.
 *   logits   [T][n_experts], row stride ld (elements, >= n_experts), MOE_BF16, MOE_F16 or MOE_F32
 *   topk_idx [T][top_k] int32 ascending, topk_w [T][top_k] fp32 (written)
 * The outputs must not overlap the logits, select_bias or each other (MOE_ERR_INVALID).
 * Limits: T <= 2^20, n_experts <= 256, top_k <= min(n_experts, 16).  T == 0 enqueues nothing.
 */
moe_status moe_select(const moe_router_rule *rule, const void *logits, int32_t dtype, int64_t T, int64_t n_experts,
                      int64_t ld, int32_t top_k, int32_t *topk_idx, float *topk_w, void *stream);

/*
 * moe_route and moe_layer_forward under a rule instead of their own (rule NULL:
 * MOE_ERR_INVALID); arguments, limits, paths, workspaces and results otherwise as theirs
 * (router_bias is part of the logits).  The logits are fp32 sums whose order differs between paths, so
 * a token whose scores lie within their rounding may be routed otherwise in a batch of another size.
 */
moe_status moe_route_rule(const moe_layer_desc *d, const moe_router_rule *rule, const void *x, int64_t T,
                          int32_t *topk_idx, float *topk_w, void *ws, size_t ws_bytes, void *stream);
moe_status moe_layer_forward_rule(const moe_layer_desc *d, const moe_router_rule *rule, const void *x, int64_t T,
                                  void *y, int32_t y_dtype, int32_t *topk_idx, float *topk_w,
                                  void *ws, size_t ws_bytes, void *stream);

/*
 * moe_layer_forward for callers that cannot allocate device memory or pass a workspace
 * (code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same kernels and the same results, bit for bit, with the workspace replaced by a
 * 64 MiB array the library holds on each GPU from load until the process ends.  This
 * call allocates nothing.  The caller still passes x, y and the optional topk outputs
 * (as for moe_layer_forward).  The array is shared by every call of this entry point on
 * one GPU and keeps the last call's contents: calls that overlap in time on one GPU race
 * (issue them on one stream).  Prompts longer than the array holds run in chunks that
 * fit it (no result changes, only more passes over the expert weights); a layer whose
 * 2-token chunk does not fit returns MOE_ERR_WORKSPACE (none within the limits above
 * does).  Errors and limits otherwise as for moe_layer_forward; MOE_ERR_DEVICE when the
 * array's address cannot be obtained on the current device.
 */
moe_status moe_layer_forward_static(const moe_layer_desc *d, const void *x, int64_t T,
                                    void *y, int32_t y_dtype,
                                    int32_t *topk_idx, float *topk_w, void *stream);

/*
 * The norms around a block, joined with its gate, residual scale and the residual stream, row by
 * row:
 *     z  = post(y) * act(gate)            (post, gate: where given)
 *     r' = r + scale * z                  (r NULL: scale * z;  y NULL: r' = r)
 *     x  = pre(r')
 * A norm (moe_norm) is  v -> u / sqrt(mean(u^2) + eps) * (offset + weight) + bias  with u = v
 * (MOE_NORM_RMS) or u = v - mean(v) (MOE_NORM_LAYER); weight NULL: no gain (nor offset), bias NULL: none.
 *   y, r, r_out, x  [T][H], row strides ldy, ldr, ldro, ldx in elements (>= H), each MOE_BF16, MOE_F16
 *               or MOE_F32; r_out receives r', x the second norm.  Either may be NULL, x exactly
 *               when pre is
 *   gate        [T][H] (gate_cols == H) or a value per row (gate_cols == 1), row stride ldg;
 *               gate_act MOE_ACT_NONE, MOE_ACT_SIGMOID 1 / (1 + exp(-g)), MOE_ACT_SILU g / (1 + exp(-g))
 *   weight, bias  [H] of the norm's dtype
 * Sums, norms and r' are fp32 until they are stored (pre reads r' before its rounding), so the mean
 * square must fit in fp32: |v| up to 2^63 or so.  A gate's sigmoid below fp32's normal range counts as 0.  NaN
 * and infinities stay in their row.
 * r_out or x may be y, r or gate itself (same pointer, type and stride: in place), or other columns of the
 * same matrix; any other overlap with an input, and any of the outputs with each other, is
 * MOE_ERR_INVALID, as are a post, gate or r_out without y.
 * Limits (else MOE_ERR_UNSUPPORTED): 1 <= H <= 16384, T <= 2^26.  T == 0 enqueues nothing.
 */
#define MOE_NORM_RMS   0
#define MOE_NORM_LAYER 1
#define MOE_ACT_NONE    0
#define MOE_ACT_SIGMOID 1
#define MOE_ACT_SILU    2
typedef struct {
    int32_t kind, dtype;
    float   eps, offset;
    const void *weight, *bias;
} moe_norm;
moe_status moe_block_norm(const void *y, int32_t y_dtype, int64_t ldy, const void *r, int32_t r_dtype, int64_t ldr,
                          const moe_norm *post, const void *gate, int32_t gate_dtype, int64_t ldg, int64_t gate_cols,
                          int32_t gate_act, float scale, const moe_norm *pre, void *r_out, int32_t r_out_dtype, int64_t ldro,
                          void *x, int32_t x_dtype, int64_t ldx, int64_t T, int64_t H, void *stream);

/*
 * Dense Q8_0 decode GEMV over 16-row packed tiles ([EMBER] packed 16-row tile):
 *     y[n] = sum_b d[n][b] * sum_{c<32} q[n][32b + c] * x[32b + c]
 * with fp32 accumulation.
 *   w_tiles  (N/16)*(K/32) tiles of 544 bytes, panel-major (tile p*(K/32) + b holds
 *            rows 16p..16p+15, columns 32b..32b+31): eight 64-byte groups, group j =
 *            rows 0..15 x codes 4j..4j+3 (4 bytes per row, rows in order), then the
 *            16 fp16 scales in row order.  16-byte aligned.
 *   x        [K] bf16;  y  [N], y_dtype MOE_BF16 or MOE_F32
 * Limits: N % 16 == 0, K % 32 == 0, N >= 16, 32 <= K <= 8192 (else MOE_ERR_UNSUPPORTED).
 */
moe_status q8_gemv(const void *w_tiles, int64_t N, int64_t K, const void *x,
                     void *y, int32_t y_dtype, void *stream);

/*
 * Activation quantization for the Q8_0 GEMV ([EMBER]: the activation is quantized once
 * and the quantized copy is shared by the projections that read it, Q/K/V and gate/up).
 * Each block of 32 values of x becomes a Q8_0 block, stored split:
 *     d[b]  = max_c |x[32b + c]| / 127, computed in binary32, stored as fp16 (nearest even)
 *     q[i]  = x[i] / d[b] in binary32 (the unrounded d), rounded half away from zero,
 *             clamped to [-127, 127]; an all-zero block has d = 0 and q = 0
 *   x   [K] bf16 (2-byte aligned);  xq [K] int8 (4-byte aligned);  xd [K/32] fp16
 *       (2-byte aligned); all device memory, xq / xd written, owned by the caller.
 * Limits: K % 32 == 0, K <= 8192 (else MOE_ERR_UNSUPPORTED); K = 0 enqueues nothing.
 */
moe_status q8_quantize_x(const void *x, int64_t K, void *xq, void *xd, void *stream);

/*
 * Dense Q8_0 GEMV with a quantized activation (from q8_quantize_x):
 *     y[n] = sum_b d[n][b] * xd[b] * sum_{c<32} q[n][32b + c] * xq[32b + c]
 * the inner sums exact in int32 (v_dot4_i32_i8), the scaling and the sum over b in fp32.
 *   w_tiles  as for q8_gemv;  xq [K] int8 (4-byte aligned), xd [K/32] fp16;
 *   y [N], y_dtype MOE_BF16 or MOE_F32.  Limits as for q8_gemv.
 */
moe_status q8_gemv_q8x(const void *w_tiles, int64_t N, int64_t K, const void *xq, const void *xd,
                         void *y, int32_t y_dtype, void *stream);

/*
 * The same GEMV taking x [K] bf16 (8-byte aligned) and quantizing it inside the kernel
 * with q8_quantize_x's rule (identical codes and scales, so identical y) while staging
 * it: no separate launch and no codes in memory.  Limits as for q8_gemv.
 */
moe_status q8_gemv_qx(const void *w_tiles, int64_t N, int64_t K, const void *x, void *y,
                        int32_t y_dtype, void *stream);

/*
 * Load-time repacking ([EMBER] packed 16-row tile): row-contiguous Q8_0 blocks
 * w_rows [N][K/32] x 34 bytes ([fp16 d][32 x int8]) -> w_tiles (layout of q8_gemv).
 * Pure byte moves, idempotent; w_rows and w_tiles must not overlap.
 * Limits: N % 16 == 0, K % 32 == 0.
 */
moe_status q8_pack_rows16(const void *w_rows, int64_t N, int64_t K, void *w_tiles,
                            void *stream);

/*
 * Microscaled 4-bit matrices (MX4): FP4 E2M1 elements (sign in bit 3, magnitudes 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6) in blocks of 32 consecutive columns of one row, one E8M0 scale byte
 * per block:  W[r][c] = 2^(scale[r][c/32] - 127) * e2m1(code[r][c]);  scale 255 makes the
 * block NaN.  Two layouts hold the same codes and scales:
 *   MX4_ROWS   codes [rows][K/2], column 2i in the low nibble of byte i, 2i+1 in the high;
 *              scales [rows][K/32].  The interchange layout.
 *   MX4_TILES  what the products read, rows in panels of 16 and columns in steps of 128
 *              (S = ceil(K/128) steps, P = ceil(rows/16) panels):  codes [P][S][64][16],
 *              entry n + 16 g of tile (p, s) = row 16p + n, columns 128s + 32g .. +31 in
 *              the byte order of MX4_ROWS;  scales [P][ceil(S/4)][64][4], byte i of entry
 *              n + 16 g of (p, q) = row 16p + n, block 4 (4q + i) + g.  Rows and columns
 *              past the matrix hold zeros.
 * mx4_codes_size / mx4_scales_size: bytes of the two buffers (SIZE_MAX when a size or the
 * layout is outside the limits).
 * Limits of every mx4_ call (else MOE_ERR_UNSUPPORTED): K % 32 == 0, 32 <= K <= 65536,
 * rows, N <= 2^26, T <= 2^20.  Zero rows (T == 0, N == 0) enqueue nothing.  codes buffers
 * are 16-byte aligned, scales buffers 4-byte; matrices of values have 16-byte aligned rows
 * (base pointer and row stride; strides ldx, ldy are in elements, >= the row's length),
 * except y of the products, which only needs its element's alignment.
 */
#define MX4_ROWS  0
#define MX4_TILES 1
size_t mx4_codes_size(int64_t rows, int64_t K, int32_t layout);
size_t mx4_scales_size(int64_t rows, int64_t K, int32_t layout);

/*
 * Quantization.  Per block, e = floor(log2(max|x|)) - 2, scale = clamp(e, -127, 127) + 127
 * (a zero block: 0); each code is x / 2^e rounded to the nearest, ties to the even code,
 * saturating at 6, the sign kept (of zeros too).  A block that holds a NaN or an infinity
 * becomes a NaN block (scale 255, codes 0).
 *   x       [rows][K], x_dtype MOE_BF16, MOE_F16 or MOE_F32, row stride ldx
 *   codes, scales   in `layout`, written whole (padding of MX4_TILES included)
 */
moe_status mx4_quantize(const void *x, int32_t x_dtype, int64_t rows, int64_t K, int64_t ldx, int32_t layout,
                        void *codes, void *scales, void *stream);

/*
 * The values of an MX4 matrix: y [rows][K], row stride ldy, y_dtype MOE_BF16 or MOE_F32
 * (exact wherever the value exists in the type) or MOE_F16 (one rounding to nearest even;
 * infinity past its range).
 */
moe_status mx4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t K, int32_t layout,
                          void *y, int32_t y_dtype, int64_t ldy, void *stream);

/*
 * Load-time repacking MX4_ROWS -> MX4_TILES (byte moves; source and destination must not
 * overlap).  A stack of matrices whose row count is a multiple of 16 is repacked as one
 * matrix of all its rows.
 */
moe_status mx4_pack_rows16(const void *codes, const void *scales, int64_t rows, int64_t K,
                           void *t_codes, void *t_scales, void *stream);

/*
 * Products with an MX4 weight matrix in MX4_TILES (N rows, K columns), fp32 accumulation:
 *     mx4_gemm        y[t][n] = sum_c x[t][c] W[n][c],  x [T][K] bf16, row stride ldx (at most
 *                     2^27, else MOE_ERR_UNSUPPORTED)
 *     mx4_gemm_mx4x   the same with x quantized: x_codes, x_scales hold T rows in MX4_TILES
 *   y   [T][N], row stride ldy, y_dtype MOE_BF16 (rounded to nearest even) or MOE_F32
 *   ws  device workspace of ws_bytes >= mx4_gemm_workspace_size(N, K, T) (NULL when that is
 *       0; one for T tokens also serves fewer), 256-byte aligned, contents undefined before
 *       and after; calls that share it must not overlap in time.
 * Every product is exact; only the fp32 sums round (and y, where it is bf16).  mx4_gemm (and the
 * layer) multiply the weights as bf16: one of 2^128 or more, which takes a scale byte of 253 or
 * 254 (mx4_quantize makes none), counts as an infinity there; mx4_gemm_mx4x takes them as they
 * are.  A NaN or infinity in x leaves no finite value in its token's row of y (mx4x: NaN, as
 * the block is) and does not reach the others; a NaN block of W makes its column of y NaN, an
 * infinity in W leaves no finite value there.
 * A token's result may depend on T (the order of its sums), not on the other tokens.
 */
size_t mx4_gemm_workspace_size(int64_t N, int64_t K, int64_t T);
moe_status mx4_gemm(const void *w_codes, const void *w_scales, int64_t N, int64_t K, const void *x, int64_t T,
                    int64_t ldx, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream);
moe_status mx4_gemm_mx4x(const void *w_codes, const void *w_scales, int64_t N, int64_t K, const void *x_codes,
                         const void *x_scales, int64_t T, void *y, int32_t y_dtype, int64_t ldy,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * Low-rank adapters of many requests, added to a shared projection's result (mx4_gemm, q8_gemv or
 * any other):
 *     y[t] = base[t] + scales[a] B_a (A_a x[t]),  a = ids[t];   y[t] = base[t] where a token has none
 *   a       [n_adapters][R][K] bf16, b [n_adapters][N][R] bf16, contiguous, 16-byte aligned
 *   scales  [n_adapters] fp32, or NULL: 1
 *   ranks   [n_adapters] int32, or NULL: R.  Rows of A and columns of B past an adapter's rank are
 *           not used, whatever they hold (a rank above R counts as R, a negative one as 0)
 *   ids     [T] int32; an id outside [0, n_adapters) is a token without an adapter
 *   x       [T][K] bf16, row stride ldx, rows 16-byte aligned
 *   base    [T][N] of y's type, row stride ldb, or NULL: zeros
 *   y       [T][N], row stride ldy, y_dtype MOE_BF16 (rounded to nearest even) or MOE_F32; it may be base
 *           (same pointer and stride: in place, tokens without an adapter are not touched), or other
 *           columns of its matrix; any other overlap with an input is MOE_ERR_INVALID
 *   ws      device workspace of ws_bytes >= lora_workspace_size(T, R), 256-byte aligned, contents undefined
 *           before and after (one for T tokens also serves fewer), apart from every other buffer; calls
 *           that share it must not overlap in time.
 * Products are exact and sums fp32; A_a x[t] times its scale is carried to 2^-16 of itself for a bf16 y,
 * to 2^-24 for an fp32 one, as two or three parts: an infinity in B gives NaN where one of them is 0.  A token's result
 * does not depend on the other tokens.  More than 65536 tokens are not ordered by adapter: where adapters
 * change from token to token, such a call takes longer than pieces of 65536 (8 adapters: 2.5 times).
 * Limits (else MOE_ERR_UNSUPPORTED): R % 8 == 0, 8 <= R <= 256, K % 8 == 0, 8 <= K <= 65536, N <= 2^23,
 * 1 <= n_adapters <= 65536, T <= 2^20.  T == 0 or N == 0 enqueues nothing.
 */
size_t lora_workspace_size(int64_t T, int64_t R);
moe_status lora_gemm(const void *a, const void *b, const float *scales, const int32_t *ranks, int64_t n_adapters,
                     int64_t R, int64_t K, int64_t N, const int32_t *ids, const void *x, int64_t T, int64_t ldx,
                     const void *base, int64_t ldb, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes,
                     void *stream);
/* What lora_gemm would return for these arguments before it enqueues anything: for callers that enqueue
 * the base first. */
moe_status lora_gemm_check(const void *a, const void *b, const float *scales, const int32_t *ranks, int64_t n_adapters,
                           int64_t R, int64_t K, int64_t N, const int32_t *ids, const void *x, int64_t T, int64_t ldx,
                           const void *base, int64_t ldb, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes);

/*
 * Measured ceilings ([LILY] "Limits of further optimization": kernels are judged
 * against the fastest sustained rate of their resource, next to the data-sheet peak).
 * Measurement helpers only; they compute nothing the layer uses.
 *   moe_calib_read  one read-only pass over buf (bytes % 16 == 0, 16-byte aligned) with
 *                   16-byte nontemporal loads: time it to get the sustained HBM read
 *                   rate (use a buffer far larger than the 256 MB on-die cache).
 *   moe_calib_mfma  `blocks` workgroups of 4 waves, each wave issuing iters x 8
 *                   v_mfma_f32_16x16x32_f16 (16384 flops each) on register operands:
 *                   the sustained dense fp16 matrix rate.
 * Both enqueue one kernel on `stream` and store nothing.
 */
moe_status moe_calib_read(const void *buf, size_t bytes, void *stream);
moe_status moe_calib_mfma(int32_t iters, int32_t blocks, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QSMOE_H */
