// mx4_gemm.hip -- y = x W^T with W in MX4 tiles and x in bf16 or MX4 (format, layouts and the
// matrix instructions each takes: mx4.h).
#include "mx4.h"

namespace qs {

namespace {

struct GemmArgs {
    const uint8_t *wc, *ws;    // weight tiles and scales
    const uint8_t *xc, *xs;    // MX4 activations: tiles and scales
    const uint16_t *x;         // bf16 activations
    void *y;
    int64_t ldx, ldy;
    int N, T, K, KS, KQ, P;    // KS, KQ: steps and quads of K; P: weight panels
    int y_dtype;
    int qs;                    // waves that share a panel, taking quads wq, wq + qs, ...
    int ppw;                   // panels per workgroup
    float *part;               // [shares][T][part_pitch(N)] partial sums (shares > 1)
    int shares;                // workgroups that split the columns of a tile between them
};

constexpr int MAX_SHARES = 16;
// row pitch of the shares' partial sums: whole 16-byte pieces
__host__ __device__ inline int64_t part_pitch(int64_t N) { return (N + 3) / 4 * 4; }

// Up to 16 tokens: bound by the weight stream.  A wave multiplies one 16-row weight panel by the
// 16-token activation tile over its share of the columns; every weight tile is read once, with
// contiguous 16-byte loads straight into registers, a chunk (one quad per wave, 4 KB of codes)
// ahead of its use.  bf16 activations are staged in LDS with coalesced reads (an MFMA operand
// read from global memory touches 64 separate 16-byte pieces, which costs the address unit four
// times the 16 cycles of a contiguous one); MX4 activations come as tiles and need no staging.
// The qs waves of a panel meet in LDS, summed in wave order.  Measured: T = 1 x 2048 x 2048 3.6 us
// (a launch and one round trip to HBM), T = 5 x 16384 x 2048 6.6 to 7.3 (17.8 MB, 2.6 TB/s: too
// few bytes to fill the pipe between its first and last loads), MX4 x T = 3 x 2048 x 8192 6.3.
template <bool MX>
__global__ __launch_bounds__(512) void k_mx4_skinny(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nt = blockDim.x;
    const int n = lane & 15, g = lane >> 4;
    const int pw = wave / a.qs, wq = wave % a.qs;
    const int pp = blockIdx.x * a.ppw + pw;
    const int p = pp < a.P ? pp : a.P - 1;

    u32x4 b[4];
    uint32_t sb = 0;
    auto load_w = [&](int q) __attribute__((always_inline)) {
        const uint8_t *c = a.wc + ((int64_t)p * a.KS + 4 * q) * MX_TILE + 16 * lane;
        sb = __builtin_nontemporal_load((const uint32_t *)(a.ws + ((int64_t)p * a.KQ + q) * MX_QS + 4 * lane));
#pragma unroll
        for (int i = 0; i < 4; ++i)                          // (steps past K: a valid tile, not used)
            b[i] = __builtin_nontemporal_load((const u32x4 *)(c + (4 * q + i < a.KS ? i : 0) * MX_TILE));
    };
    if (wq < a.KQ) load_w(wq);

    const int pitch = a.KQ * 1024 + 16;                      // bytes of a staged row (padded: banks)
    if constexpr (!MX) {
        const int nc = a.KQ * 64;                            // 16-byte pieces per row
        for (int i = tid; i < a.T * nc; i += nt) {
            const int r = i / nc, c = i % nc;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (8 * c < a.K) v = *(const u32x4 *)(a.x + r * a.ldx + 8 * c);
            *(u32x4 *)(sm + r * pitch + 16 * c) = v;
        }
        __syncthreads();
    }
    const int r = n < a.T ? n : a.T - 1;                     // (past the tokens: repeated, discarded)
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int q = wq; q < a.KQ; q += a.qs) {
        u32x4 bb[4];
        const uint32_t sbb = sb;
#pragma unroll
        for (int i = 0; i < 4; ++i) bb[i] = b[i];
        if (q + a.qs < a.KQ) load_w(q + a.qs);
        uint32_t sa = 0;
        if constexpr (MX) sa = *(const uint32_t *)(a.xs + q * MX_QS + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * q + i >= a.KS) break;
            if constexpr (MX) {
                acc = mx_mfma(*(const u32x4 *)(a.xc + (4 * q + i) * MX_TILE + 16 * lane), bb[i], acc, i, sa, sbb);
            } else {
                const float sc = mx_scale(sbb, i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        *(const bf16x8 *)(sm + r * pitch + 1024 * q + 256 * i + 64 * g + 16 * j), mx_bf16(bb[i][j], sc),
                        acc, 0, 0, 0);
            }
        }
    }
    // join the panel's waves in wave order
    if (a.qs > 1) {
        f32x4 *red = (f32x4 *)sm;
        __syncthreads();
        red[wave * 64 + lane] = acc;
        __syncthreads();
        if (wq == 0)
            for (int w = 1; w < a.qs; ++w) acc += red[(wave + w) * 64 + lane];
    }
    const int col = 16 * p + n;
    if (wq == 0 && pp < a.P && col < a.N)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (4 * g + x < a.T) mx_store(a.y, (4 * g + x) * a.ldy + col, acc[x], a.y_dtype);
}

template <bool MX>
hipError_t launch_skinny(GemmArgs a, hipStream_t s) {
    a.qs = 1;
    while (a.qs < 8 && 2 * a.qs <= a.KQ) a.qs *= 2;
    a.ppw = 1;
    while (a.qs * a.ppw < 8 && a.P / (2 * a.ppw) >= 2 * n_compute_units()) a.ppw *= 2;
    const int waves = a.qs * a.ppw;
    const size_t red = a.qs > 1 ? (size_t)waves * 1024 : 16, stage = MX ? 0 : (size_t)a.T * (a.KQ * 1024 + 16);
    hipLaunchKernelGGL(k_mx4_skinny<MX>, dim3((a.P + a.ppw - 1) / a.ppw), dim3(64 * waves), red > stage ? red : stage, s,
                       a);
    return hipGetLastError();
}

// ------------------------------------------------------------------- many tokens
// Bound by the matrix cores: four waves, each FM x FN fragments of 32 tokens x 32 weight rows
// (v_mfma 32x32, the weights as first operand so that a lane's registers are neighbouring columns
// of y).  The waves split the weight rows and share the tokens: activations go global -> LDS by
// direct-to-LDS loads in a ring of three stages, each wave's weights, which no other multiplies,
// straight into its registers, both two steps ahead; one barrier a step.  Against weights through
// LDS too: 4096 x 16384 x 2048 in large tiles 242 -> 209 us with bf16 x and 97 -> 77 with MX4 x,
// 128 x 16384 x 2048 in small ones 15.5 -> 12.4 and 7.1 -> 6.1 (two waves to a weight row before).
//   bf16 x: a step is 64 columns.  128 bytes of a token's row, its eight 16-byte chunks XORed
//     by (row / 2) % 8: a 16-byte LDS read is served 16 lanes a cycle, those of one wave half
//     with equal parity of lane bits 2..4 (measured), and under this key they fall in 64
//     distinct banks.
//   MX4 x: a step is 128 columns, a tile of each panel of x as it lies in memory.
// Rates: 4096 x 16384 x 2048 196 to 209 us with bf16 x (1.3 to 1.4 PFLOP/s, a library bf16 product of
// the shape takes 194 to 213), 69 to 77 with MX4 x (3.6 to 4.0); 4096 x 16384 x 8192 4.25 PFLOP/s with
// MX4 x, where the loop without any of its loads from memory reaches 4.6.  An MFMA-only loop sustains
// 2.0 to 2.2 and 5.8 to 6.9; the matrix cores are busy 0.70 of the cycles with bf16 x, 0.45 with MX4 x
// (16 steps a tile, then 64 KB of y: waves wait 0.32 of theirs), LDS 0.21 and 0.24.
// Scales come a quad (512 columns) at a time; every wave has them in registers a step later, long
// before the next quad's arrive in their place.
constexpr int NW = 4;                                        // waves of a tile's workgroup
template <bool MX, int FM, int FN>
struct Tiled {
    static constexpr int BM = 32 * FM, BN = 32 * FN * NW;
    static constexpr int STEP = MX ? 128 : 64;                        // columns
    static constexpr int PER_Q = 512 / STEP;                          // steps per quad of scales
    static constexpr int STAGE = MX ? BM * 64 : BM * 128, NSTAGE = 3;  // of activations
    static constexpr int SC_BYTES = (MX ? BM * 16 : 0) + BN * 16;     // of a quad
    static constexpr int B_STEP = MX ? MX_TILE : MX_TILE / 2;         // bytes of a weight panel
    // per wave: 16-byte loads of activations and of weights a step, of scales a quad
    static constexpr int A_DMA = STAGE / (1024 * NW), BL = FN * (MX ? 2 : 1);
    static constexpr int XS = MX ? BM / (16 * NW) : 0, WS = BN / (16 * NW), SDMA = XS + WS;
    static constexpr int EP = 32 * (FN * 32 * 4 + 16);                // epilogue staging of a wave
    static constexpr int RING = NSTAGE * STAGE + SC_BYTES;
    static constexpr int LDS = RING > NW * EP ? RING : NW * EP;
    static_assert(STAGE % (1024 * NW) == 0 && (!MX || BM % (16 * NW) == 0), "whole loads per wave");
};

// Epilogue of a wave: 32 tokens at a time through its LDS area ep, then whole 16-byte pieces of
// y's rows.  acc[j][i][r]: token 32 i + lane % 32, weight row 32 j + 8 (r / 4) + 4 h + r % 4.
template <bool F32, bool PART, int FM, int FN>
__device__ __forceinline__ void tiled_store(const f32x16 (&acc)[FN][FM], uint8_t *ep, void *y, int64_t ldy, int T, int N,
                                            int t0, int n0) {
    constexpr int ESZ = F32 ? 4 : 2, PER = 16 / ESZ;         // elements of a 16-byte piece
    constexpr int PITCH = FN * 32 * ESZ + 16, PR = FN * 32 / PER;   // pieces of a row
    constexpr int RP = 64 / PR;                              // rows per store
    const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
    const int row = lane / PR, n = n0 + lane % PR * PER;
    const bool vec = ((uintptr_t)y & 15) == 0 && (ldy * ESZ & 15) == 0 && n + PER <= N;
    const uint8_t *src = ep + row * PITCH + lane % PR * 16;
    uint8_t *dst = (uint8_t *)y + ((t0 + row) * ldy + n) * ESZ;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                uint8_t *d = ep + r32 * PITCH + (32 * j + 8 * r4 + 4 * h) * ESZ;
                const f32x16 &v = acc[j][i];
                const f32x4 f = {v[4 * r4], v[4 * r4 + 1], v[4 * r4 + 2], v[4 * r4 + 3]};
                if constexpr (F32) *(f32x4 *)d = f;
                else *(bf16x4 *)d = __builtin_convertvector(f, bf16x4);   // (nearest even)
            }
        wave_lds_sync();
#pragma unroll
        for (int c = 0; c < 32 / RP; ++c) {
            const int t = t0 + 32 * i + RP * c + row;
            const u32x4 v = *(const u32x4 *)(src + RP * c * PITCH);
            if (t < T) {
                uint8_t *d = dst + (32 * i + RP * c) * ldy * ESZ;
                if (vec && PART) *(u32x4 *)d = v;
                else if (vec) __builtin_nontemporal_store(v, (u32x4 *)d);   // (y is not read here)
                else
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        if (n + q >= N) break;
                        if constexpr (F32) ((uint32_t *)d)[q] = v[q];
                        else ((uint16_t *)d)[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
                    }
            }
        }
        wave_lds_sync();
    }
}

template <bool MX, int FM, int FN>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void k_mx4_tiled(GemmArgs a) {
    using C = Tiled<MX, FM, FN>;
    __shared__ __attribute__((aligned(1024))) uint8_t sm[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r32 = lane & 31, h = lane >> 5;
    // ---- which tile: a contiguous range of tiles per XCD, eight column tiles wide, so that
    // the workgroups an XCD runs at a time share their rows of x and of W in its L2
    const int mtiles = (a.T + C::BM - 1) / C::BM, ntiles = (a.N + C::BN - 1) / C::BN, tiles = mtiles * ntiles;
    const int id = ((int)blockIdx.x & 7) * ((tiles + 7) >> 3) + ((int)blockIdx.x >> 3);
    if (id >= tiles || ((int)blockIdx.x >> 3) >= ((tiles + 7) >> 3)) return;
    const int ng = id / (8 * mtiles), gw = ntiles - 8 * ng < 8 ? ntiles - 8 * ng : 8;
    const int rem = id - ng * 8 * mtiles;
    const int t0 = rem / gw * C::BM, n0 = (8 * ng + rem % gw) * C::BN;

    const int steps = (a.K + C::STEP - 1) / C::STEP;
    // this workgroup's share of the steps (whole quads)
    const int qper = (a.KQ + a.shares - 1) / a.shares;
    const int k_lo = blockIdx.y * qper * C::PER_Q;
    const int k_hi = k_lo + qper * C::PER_Q < steps ? k_lo + qper * C::PER_Q : steps;

    // ---- sources of this wave's loads
    const int xp0 = t0 / 16, xpl = (a.T + 15) / 16 - 1, wp0 = n0 / 16;      // panels (xpl: the last of x)
    auto wpanel = [&](int p) __attribute__((always_inline)) { return wp0 + p < a.P ? p : a.P - 1 - wp0; };
    auto xpanel = [&](int p) __attribute__((always_inline)) { return xp0 + p <= xpl ? p : xpl - xp0; };
    // activations: piece i of a stage is 1024 bytes, through a resource of its own
    __amdgpu_buffer_rsrc_t abuf[C::A_DMA];
    uint32_t aoff[C::A_DMA];
    int kmax[C::A_DMA];                     // bf16 x: the last column offset at which the chunk is whole
#pragma unroll
    for (int i = 0; i < C::A_DMA; ++i) {
        const int piece = wave * C::A_DMA + i;
        if constexpr (MX) {
            abuf[i] = buffer_from(a.xc + (int64_t)(xp0 + xpanel(piece)) * a.KS * MX_TILE);
            aoff[i] = 16 * lane;
            kmax[i] = 0;
        } else {                            // eight rows (past the last: that one again)
            const int first = min(t0 + 8 * piece, a.T - 1), row = 8 * piece + (lane >> 3);
            const int c = (lane & 7) ^ ((row >> 1) & 7);
            abuf[i] = buffer_from(a.x + first * a.ldx);
            aoff[i] = (uint32_t)(min(t0 + row, a.T - 1) - first) * (uint32_t)(2 * a.ldx) + 16 * c;
            kmax[i] = a.K - 8 * c - 8;
        }
    }
    const uint8_t *bsrc[FN];                // weights of the next step, by fragment
#pragma unroll
    for (int j = 0; j < FN; ++j)
        bsrc[j] = a.wc + (int64_t)(wp0 + wpanel(2 * (wave * FN + j) + (r32 >> 4))) * a.KS * MX_TILE +
                  16 * ((r32 & 15) + 16 * h) + (int64_t)k_lo * C::B_STEP;
    // scales, 256 bytes (a panel) a piece: XS of x, then WS of the weights
    const __amdgpu_buffer_rsrc_t xsbuf = buffer_from(MX ? a.xs + (int64_t)xp0 * a.KQ * MX_QS : a.ws);
    const __amdgpu_buffer_rsrc_t wsbuf = buffer_from(a.ws + (int64_t)wp0 * a.KQ * MX_QS);
    int soff[C::SDMA];
#pragma unroll
    for (int i = 0; i < C::SDMA; ++i)
        soff[i] = (i < C::XS ? xpanel(wave * C::XS + i) : wpanel(wave * C::WS + i - C::XS)) * a.KQ * MX_QS + 4 * lane;
    auto issue = [&](int k, int s) __attribute__((always_inline)) {   // step k, the s-th of its quad
        uint8_t *st = sm + (k % C::NSTAGE) * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::A_DMA; ++i) {
            // (bf16 x: columns past K meet zero weights, any value of the row will do)
            const int off = C::STEP * k;
            dma16_buffer(abuf[i], st + (wave * C::A_DMA + i) * 1024,
                         MX ? aoff[i] : aoff[i] + 2 * (off <= kmax[i] ? off : kmax[i]), MX ? k * MX_TILE : 0);
        }
        if (s % C::PER_Q == 0) {
            const int q = k / C::PER_Q * MX_QS;
            uint8_t *ss = sm + C::NSTAGE * C::STAGE;
#pragma unroll
            for (int i = 0; i < C::SDMA; ++i)
                dma4_buffer(i < C::XS ? xsbuf : wsbuf,
                            ss + (i < C::XS ? (wave * C::XS + i) * 256
                                            : (MX ? C::BM * 16 : 0) + (wave * C::WS + i - C::XS) * 256),
                            soff[i], q);
        }
    };
    u32x4 bq[2][C::BL];                                      // weights, by the step's parity
    auto load_b = [&](u32x4 (&b)[C::BL]) __attribute__((always_inline)) {   // of the next step
#pragma unroll
        for (int i = 0; i < C::BL; ++i) b[i] = *(const u32x4 *)(bsrc[MX ? i >> 1 : i] + (MX ? 512 * (i & 1) : 0));
#pragma unroll
        for (int j = 0; j < FN; ++j) bsrc[j] += C::B_STEP;
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    // scales of a quad: lane (row, h) keeps blocks h and 2 + h of each step of 128
    uint32_t sw[FN][2], sx[FM][2];
    auto load_scales = [&]() __attribute__((always_inline)) {
        const uint8_t *ss = sm + C::NSTAGE * C::STAGE;
        const int e = (r32 >> 4) * 256 + 4 * ((r32 & 15) + 16 * h);
        const uint8_t *sb = ss + (MX ? C::BM * 16 : 0) + wave * FN * 512 + e;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            sw[j][0] = *(const uint32_t *)(sb + 512 * j);
            sw[j][1] = *(const uint32_t *)(sb + 512 * j + 128);
        }
        if constexpr (MX) {
            const uint8_t *sa = ss + e;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                sx[i][0] = *(const uint32_t *)(sa + 512 * i);
                sx[i][1] = *(const uint32_t *)(sa + 512 * i + 128);
            }
        }
    };
    // ahead: stage k + 2 exists
    auto sync_step = [&](int k, int s, bool ahead) __attribute__((always_inline)) {
        // stage k has landed once at most stage k + 1's loads are outstanding
        if (!ahead && k + 1 >= k_hi) wait_dma<0>();
        else if ((s + 1) % C::PER_Q == 0) wait_dma<C::A_DMA + C::BL + C::SDMA>();
        else wait_dma<C::A_DMA + C::BL>();
        block_sync();
        if (ahead) issue(k + 2, s + 2);
    };

    auto start = [&](int s) __attribute__((always_inline)) {
        issue(k_lo + s, s);
        load_b(bq[s]);
        __builtin_amdgcn_sched_barrier(0);                   // (and the next step's after these)
    };
    // step k, the s-th of its quad
    auto step = [&](int k, int s, bool ahead) __attribute__((always_inline)) {
        sync_step(k, s, ahead);
        const uint8_t *st = sm + (k % C::NSTAGE) * C::STAGE;
        u32x4(&bk)[C::BL] = bq[s & 1];
        if constexpr (MX) {
            if (s == 0) load_scales();
            const int e = (r32 >> 4) * MX_TILE + 16 * ((r32 & 15) + 16 * h);
#pragma unroll
            for (int f = 0; f < 2; ++f) {                    // columns 64 f .. 64 f + 63 of the step
                u32x4 A[FM];
#pragma unroll
                for (int i = 0; i < FM; ++i) A[i] = *(const u32x4 *)(st + i * 2 * MX_TILE + e + 512 * f);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[j][i] = mx_mfma32(bk[2 * j + f], A[i], acc[j][i], s, sw[j][f], sx[i][f]);
            }
        } else {
            if (s == 0) load_scales();
            float sc[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) sc[j] = mx_scale(sw[j][s & 1], s >> 1);
            // columns 32 h + 8 m .. + 7: x of m + 1 is read while m is multiplied
            bf16x8 A[2][FM];
            auto load_a = [&](int m) __attribute__((always_inline)) {
                const int pos = (4 * h + m) ^ ((r32 >> 1) & 7);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    A[m & 1][i] = *(const bf16x8 *)(st + (32 * i + r32) * 128 + 16 * pos);
            };
            load_a(0);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m < 3) load_a(m + 1);
                bf16x8 B[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j) B[j] = mx_bf16(bk[j][m], sc[j]);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(B[j], A[m & 1][i], acc[j][i], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);           // (no reads of later columns drawn ahead)
            }
        }
        if (ahead) load_b(bk);
    };
    // Whole quads load two steps ahead without a condition, so that the compiler knows how many
    // loads are outstanding wherever it waits for one; what is left of K takes the last loop.
    constexpr int U = C::PER_Q;
    int k0 = k_lo;
    if (k0 + U <= k_hi) {
        start(0);
        start(1);
        for (; k0 + U + 2 <= k_hi; k0 += U)
#pragma unroll
            for (int s = 0; s < U; ++s) step(k0 + s, s, true);
        if (k0 + U == k_hi) {
#pragma unroll
            for (int s = 0; s < U; ++s) step(k0 + s, s, s + 2 < U);
            k0 += U;
        }
    } else {
        if (k_lo < k_hi) start(0);
        if (k_lo + 1 < k_hi) start(1);
    }
    for (; k0 < k_hi; k0 += U)
#pragma unroll
        for (int s = 0; s < U; ++s) {
            if (k0 + s >= k_hi) break;
            step(k0 + s, s, k0 + s + 2 < k_hi);
        }
    block_sync();                                            // the ring is free

    const int nw = n0 + wave * FN * 32;
    if (a.shares > 1)
        tiled_store<true, true, FM, FN>(acc, sm + wave * C::EP, a.part + blockIdx.y * (a.T * part_pitch(a.N)),
                                  part_pitch(a.N), a.T, a.N, t0, nw);
    else if (a.y_dtype == MOE_F32)
        tiled_store<true, false, FM, FN>(acc, sm + wave * C::EP, a.y, a.ldy, a.T, a.N, t0, nw);
    else
        tiled_store<false, false, FM, FN>(acc, sm + wave * C::EP, a.y, a.ldy, a.T, a.N, t0, nw);
}

// The shares' partial sums, in share order: a thread adds four columns, all shares' loads in
// flight at once (T = 37 x 2048, 16 shares: 3.6 us, a launch and a round trip to the caches).
__global__ __launch_bounds__(256) void k_mx4_join(GemmArgs a) {
    const int64_t np = part_pitch(a.N), n4 = np / 4, total = a.T * n4, st = a.T * np;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / n4;
        const int n = (int)(i - t * n4) * 4;
        const float *p = a.part + t * np + n;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        f32x4 q[MAX_SHARES];
#pragma unroll
        for (int s = 0; s < MAX_SHARES; ++s)
            if (s < a.shares) q[s] = *(const f32x4 *)(p + s * st);
#pragma unroll
        for (int s = 0; s < MAX_SHARES; ++s)
            if (s < a.shares) v += q[s];
        const int64_t o = t * a.ldy + n;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n + c < a.N) mx_store(a.y, o + c, v[c], a.y_dtype);
    }
}

template <bool MX, int FM, int FN>
hipError_t launch_tiled(GemmArgs a, hipStream_t s) {
    using C = Tiled<MX, FM, FN>;
    const int tiles = ((a.T + C::BM - 1) / C::BM) * ((a.N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((k_mx4_tiled<MX, FM, FN>), dim3((tiles + 7) / 8 * 8, a.shares), dim3(64 * NW), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.shares == 1) return e;
    const int64_t b = (a.T * (part_pitch(a.N) / 4) + 255) / 256, cap = 8 * (int64_t)n_compute_units();
    hipLaunchKernelGGL(k_mx4_join, dim3((unsigned)(b < cap ? b : cap)), dim3(256), 0, s, a);
    return hipGetLastError();
}

GemmArgs make_args(const uint8_t *wc, const uint8_t *ws, int64_t N, int64_t K, int64_t T, void *y, int y_dtype,
                   int64_t ldy) {
    GemmArgs a{};
    a.wc = wc;
    a.ws = ws;
    a.N = (int)N;
    a.K = (int)K;
    a.T = (int)T;
    a.KS = (int)mx4_steps(K);
    a.KQ = (int)mx4_quads(K);
    a.P = (int)((N + 15) / 16);
    a.y = y;
    a.y_dtype = y_dtype;
    a.ldy = ldy;
    a.shares = 1;
    return a;
}

}  // namespace

// Which kernel (times: bf16 x, us):
//   skinny  up to 16 tokens, bf16 x only while all of it can be staged at once (64 KB): beyond,
//           staging between barriers costs more than reading the weights once saves
//           (T = 16 x 16384 x 2048: 7.5 against 13.0 in tiles; T = 16 x 2048 x 8192: 30.5 against 10.9)
//   large   tiles of 128 x 256, two workgroups a compute unit, if they fill their last round of the
//           device to 7/8 on average, and over 64 tokens (which one row of small tiles holds); times
//           in large and in small tiles at 16384 x 2048: T = 512, half a round, 35 and 33; T = 768,
//           3/4, 52 and 48; T = 1024, one round, 59 and 62 (MX4 x: 23 and 27); T = 1152 78 and 70
//   small   tiles of 64 x 128, and where those are fewer than the compute units, the columns
//           split into shares of at least one quad (T = 37 x 2048 x 8192: 11.4 with 16 shares,
//           12.7 with 8; T = 128 x 16384 x 2048, a tile per compute unit, 12.4, halved 22)
enum Plan { SKINNY, SMALL, LARGE };
struct Choice {
    Plan plan;
    int shares;
};
static Choice choose(bool mx, int64_t T, int64_t N, int64_t K) {
    if (T <= 16 && (mx || T * mx4_quads(K) <= 64)) return {SKINNY, 1};
    const int64_t cu = n_compute_units();
    auto tiles = [&](int64_t m, int64_t n) { return ((T + m - 1) / m) * ((N + n - 1) / n); };
    const int64_t large = tiles(128, 256), round = 2 * cu;
    if (T > 64 && 8 * large >= 7 * ((large + round - 1) / round * round)) return {LARGE, 1};
    const int64_t quads = mx4_quads(K);
    int64_t sh = cu / tiles(64, 128);
    if (sh > quads) sh = quads;
    if (sh > MAX_SHARES) sh = MAX_SHARES;
    if (sh <= 1) return {SMALL, 1};
    // (whole quads a share: no more shares than those leave something to)
    const int64_t per = (quads + sh - 1) / sh;
    return {SMALL, (int)((quads + per - 1) / per)};
}

// For either kind of x, and never less than for fewer tokens: the largest shares x tokens of the
// row counts up to T (within a row of tiles the shares are the same, so its last count is it).
size_t mx4_gemm_ws(int64_t T, int64_t N, int64_t K) {
    int64_t rows = 0;
    for (int64_t t = 64;; t += 64) {
        const int64_t n = t < T ? t : T, sh = choose(false, n, N, K).shares;
        if (sh > 1 && sh * n > rows) rows = sh * n;
        if (n == T || n_compute_units() < 2 * ((n + 63) / 64) * ((N + 127) / 128)) break;
    }
    return (size_t)(rows * part_pitch(N) * 4);
}

template <bool MX>
static hipError_t launch_product(GemmArgs a, uint8_t *ws, hipStream_t s) {
    const Choice c = choose(MX, a.T, a.N, a.K);
    a.shares = c.shares;
    a.part = (float *)ws;
    if (c.plan == SKINNY) return launch_skinny<MX>(a, s);
    if (c.plan == SMALL) return launch_tiled<MX, 2, 1>(a, s);
    return launch_tiled<MX, 4, 2>(a, s);
}

hipError_t launch_mx4_gemm(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint16_t *x, int64_t T,
                           int64_t ldx, void *y, int y_dtype, int64_t ldy, uint8_t *ws, hipStream_t s) {
    GemmArgs a = make_args(wc, wsc, N, K, T, y, y_dtype, ldy);
    a.x = x;
    a.ldx = ldx;
    return launch_product<false>(a, ws, s);
}

hipError_t launch_mx4_gemm_mx4x(const uint8_t *wc, const uint8_t *wsc, int64_t N, int64_t K, const uint8_t *xc,
                                const uint8_t *xs, int64_t T, void *y, int y_dtype, int64_t ldy, uint8_t *ws,
                                hipStream_t s) {
    GemmArgs a = make_args(wc, wsc, N, K, T, y, y_dtype, ldy);
    a.xc = xc;
    a.xs = xs;
    return launch_product<true>(a, ws, s);
}

}  // namespace qs
