// mx4_group.hip -- the expert products of a prompt with MX4 experts, on v_mfma 32x32x16 bf16.
//
// Work comes from the grouped path's block map: tiles of up to GEMM_BM = 160 rows of one
// expert's bin (or of the shared expert), each against column blocks of 256 weight rows, one
// launch for [gate; up] and one for down.  Four waves; a wave takes 64 weight rows (two
// fragments of 32) against the tile's rows (five fragments, only as many as the tile fills),
// the weights as first operand, so that a lane's registers are neighbouring columns.
//
// Data movement as in mx4_gemm.hip: everything global -> LDS by direct-to-LDS loads, steps of
// 64 columns, activation rows of 128 bytes with their chunks XORed by (row / 2) % 8; here a
// ring of two stages, so that two workgroups fit a compute unit and one's prologue and epilogue
// run under the other's products.  Each wave loads the weight tiles it multiplies itself.
//
//   gate/up  rows of x gathered through perm; the wave's fragments are 32 gate rows and the
//            same 32 up rows, so h = silu(g) u is formed in registers.  It leaves as the bf16
//            pair hi + lo (h to 2^-17), [row][hi, lo][I].
//   down     rows of h; the reduction runs over hi, then over lo, each against the same weights
//            (a third more matrix work than bf16 h, which would leave 2e-3 x RMS of error in the
//            layer).  Slot rows as the affine path writes them: w o in fp16 under a scale per row
//            and 64 columns (a wave's), for the same combine.
#include "mx4.h"

namespace qs {

namespace {

struct GroupArgs {
    Layer L;
    const uint16_t *x;
    int64_t T;
    uint16_t *h;
    const int32_t *perm;
    const Tile *tiles;
    int32_t *ntiles;
    const float *w, *sgate;
    uint16_t *slot;
    int8_t *sexp;
    int nb;                          // column blocks per tile
};

constexpr int FM = GEMM_BM / 32, FN = 2, GW = 4;
constexpr int A_STAGE = GEMM_BM * 128, B_STAGE = 256 * 32, STAGE = A_STAGE + B_STAGE;
constexpr int SC_SLOT = 256 * 16, RING = 2 * STAGE + 2 * SC_SLOT;
constexpr int A_DMA = A_STAGE / (1024 * GW), B_DMA = 2, S_DMA = 4;
constexpr int EP = 32 * (64 * 4 + 16);                       // a wave's epilogue staging
static_assert(GW * EP <= RING && GEMM_BM % 32 == 0 && A_STAGE % (1024 * GW) == 0, "tile shape");

template <bool DOWN>
__global__ __launch_bounds__(64 * GW) __attribute__((amdgpu_waves_per_eu(2))) void k_mx_group(GroupArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t sm[RING];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r32 = lane & 31, h = lane >> 5;
    const Layer &L = a.L;
    const int H = L.H, I = L.I, K = L.K;
    // the column blocks of a tile, which share its rows, run on one XCD
    const int bslot = (int)blockIdx.x >> 3, ti = bslot / a.nb * 8 + ((int)blockIdx.x & 7), nbi = bslot % a.nb;
    if (ti >= a.ntiles[1]) return;
    const Tile tile = a.tiles[ti];
    const bool sh = tile.expert == L.E;
    const int nrows = tile.nrows, nf = (nrows + 31) >> 5;
    const int64_t e = sh ? 0 : tile.expert, TK = a.T * K;
    const int Kdim = DOWN ? I : H, KS = (Kdim + 127) >> 7, KQ = (KS + 3) >> 2;
    const int S = Kdim / 64, steps = DOWN ? 2 * S : S;       // (H and I are multiples of 64)

    // ---- this wave's weight panels: four of 16 rows (gate/up: two of gate, two of up)
    const uint8_t *bsrc[B_DMA], *ssrc[S_DMA];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint8_t *codes, *scales;
        int64_t stride;
        if (DOWN) {
            codes = sh ? L.s_down.codes : L.down.codes;
            scales = (const uint8_t *)(sh ? L.s_down.scales : L.down.scales);
            stride = sh ? L.s_down.stride : L.down.stride;
        } else if (j == 0) {
            codes = sh ? L.s_gate.codes : L.gate.codes;
            scales = (const uint8_t *)(sh ? L.s_gate.scales : L.gate.scales);
            stride = sh ? L.s_gate.stride : L.gate.stride;
        } else {
            codes = sh ? L.s_up.codes : L.up.codes;
            scales = (const uint8_t *)(sh ? L.s_up.scales : L.up.scales);
            stride = sh ? L.s_up.stride : L.up.stride;
        }
        // (columns past the matrix: its last panel, discarded)
        const int first = DOWN ? nbi * 16 + wave * 4 + 2 * j : nbi * 8 + wave * 2, np = (DOWN ? H : I) / 16;
        const int64_t p0 = e * stride / 16;
        bsrc[j] = codes + (p0 + min(first + h, np - 1)) * KS * MX_TILE + 16 * r32;
#pragma unroll
        for (int i = 0; i < 2; ++i) ssrc[2 * j + i] = scales + (p0 + min(first + i, np - 1)) * KQ * MX_QS + 4 * lane;
    }
    // ---- activation rows: piece i of a stage is rows 8 (A_DMA wave + i) .. + 7
    const uint8_t *asrc[A_DMA];
#pragma unroll
    for (int i = 0; i < A_DMA; ++i) {
        const int row = 8 * (A_DMA * wave + i) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
        const int r = tile.row0 + (row < nrows ? row : nrows - 1);         // (past the tile: its last row)
        const uint16_t *src;
        if (DOWN) src = a.h + (int64_t)r * 2 * I;
        else src = a.x + (sh ? r - TK : (int64_t)(a.perm[r] / K)) * H;
        asrc[i] = (const uint8_t *)(src + 8 * c);
    }
    auto issue = [&](int k) __attribute__((always_inline)) {
        uint8_t *st = sm + (k & 1) * STAGE;
        const int kb = DOWN && k >= S ? k - S : k;
#pragma unroll
        for (int i = 0; i < A_DMA; ++i) dma16(asrc[i] + (int64_t)k * 128, st + (A_DMA * wave + i) * 1024);
#pragma unroll
        for (int j = 0; j < B_DMA; ++j)
            dma16(bsrc[j] + (int64_t)kb * (MX_TILE / 2), st + A_STAGE + (B_DMA * wave + j) * 1024);
        if (kb % 8 == 0) {                                   // a quad's scales; slots alternate
            const int n = kb / 8 + (DOWN && k >= S ? KQ : 0);
#pragma unroll
            for (int i = 0; i < S_DMA; ++i)
                dma4(ssrc[i] + (int64_t)(kb / 8) * MX_QS, sm + 2 * STAGE + (n & 1) * SC_SLOT + (S_DMA * wave + i) * 256);
        }
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
    uint32_t sw[FN][2];
    issue(0);
    for (int k = 0; k < steps; ++k) {
        wait_dma<0>();                                       // stage k has landed, and is read after the barrier,
        block_sync();                                        // which also frees stage k - 1 for the next loads
        if (k + 1 < steps) issue(k + 1);
        const int kb = DOWN && k >= S ? k - S : k;
        if (kb % 8 == 0) {
            const int n = kb / 8 + (DOWN && k >= S ? KQ : 0);
            const uint8_t *ss = sm + 2 * STAGE + (n & 1) * SC_SLOT + wave * 1024 + (r32 >> 4) * 256 + 4 * ((r32 & 15) + 16 * h);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                sw[j][0] = *(const uint32_t *)(ss + 512 * j);
                sw[j][1] = *(const uint32_t *)(ss + 512 * j + 128);
            }
        }
        const uint8_t *st = sm + (k & 1) * STAGE;
        u32x4 b[FN];
        float sc[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            b[j] = *(const u32x4 *)(st + A_STAGE + wave * 2048 + j * 1024 + (r32 >> 4) * 512 + 16 * ((r32 & 15) + 16 * h));
            sc[j] = mx_scale((kb & 1) ? sw[j][1] : sw[j][0], (kb >> 1) & 3);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {                        // columns 32 h + 8 m .. + 7
            bf16x8 A[FM], B[FN];
            const int pos = (4 * h + m) ^ ((r32 >> 1) & 7);
#pragma unroll
            for (int i = 0; i < FM; ++i) A[i] = *(const bf16x8 *)(st + (32 * i + r32) * 128 + 16 * pos);
#pragma unroll
            for (int j = 0; j < FN; ++j) B[j] = mx_bf16(b[j][m], sc[j]);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                if (i < nf)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(B[j], A[i], acc[j][i], 0, 0, 0);
        }
    }
    block_sync();                                            // the ring is free

    // ---- epilogues, 32 rows at a time through the wave's LDS area.  acc[j][i][r]: row
    // 32 i + lane % 32, weight row 32 j + 8 (r / 4) + 4 h + r % 4 of the wave's
    uint8_t *ep = sm + wave * EP;
    if constexpr (!DOWN) {
        constexpr int PITCH = 64 * 2 + 16;                   // hi of 32 columns, then lo
        const int col = nbi * 128 + wave * 32;
        if (col >= I) return;                                // (I % 128 == 64: the last block's upper waves)
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i >= nf) break;
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = silu(acc[0][i][4 * r4 + r]) * acc[1][i][4 * r4 + r];
                const bf16x4 hi = __builtin_convertvector(v, bf16x4);
                const bf16x4 lo = __builtin_convertvector(v - __builtin_convertvector(hi, f32x4), bf16x4);
                uint8_t *d = ep + r32 * PITCH + (8 * r4 + 4 * h) * 2;
                *(bf16x4 *)d = hi;
                *(bf16x4 *)(d + 64) = lo;
            }
            wave_lds_sync();
            // 8 lanes per row: four 16-byte pieces of hi, four of lo
            const int c = lane & 7;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = 8 * q + (lane >> 3);
                const u32x4 v = *(const u32x4 *)(ep + row * PITCH + 16 * c);
                if (32 * i + row < nrows)
                    *(u32x4 *)(a.h + ((int64_t)(tile.row0 + 32 * i + row) * 2 + (c >> 2)) * I + col + 8 * (c & 3)) = v;
            }
            wave_lds_sync();
        }
    } else {
        constexpr int PITCH = 64 * 4 + 16;
        const int col = nbi * 256 + wave * 64;
        if (col >= H) return;
        int8_t *sexp_blk = a.sexp + (int64_t)(col >> 6) * sexp_rows(a.T, K);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i >= nf) break;
            const int row = 32 * i + r32;
            const bool live = row < nrows;
            const int rr = tile.row0 + (live ? row : nrows - 1);
            const int64_t p = sh ? rr : a.perm[rr];           // slot row
            const float w = !sh ? a.w[p] : a.sgate ? a.sgate[p - TK] : 1.0f;
            float mx = 0.0f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) mx = __builtin_fmaxf(mx, __builtin_fabsf(acc[j][i][r]));
            // (the row's other columns are in lane ^ 32)
            const auto o = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
            mx = __builtin_fmaxf(__uint_as_float(o[0]), __uint_as_float(o[1])) * __builtin_fabsf(w);
            const int es = range_exp(mx);
            const float f = w * exp2i(es);
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    uint32_t q[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        q[r] = pack_f16x2(f32_to_f16_ftz(acc[j][i][4 * r4 + 2 * r] * f),
                                          f32_to_f16_ftz(acc[j][i][4 * r4 + 2 * r + 1] * f));
                    *(uint64_t *)(ep + r32 * PITCH + (32 * j + 8 * r4 + 4 * h) * 2) = q[0] | (uint64_t)q[1] << 32;
                }
            if (live && h == 0) sexp_blk[p] = (int8_t)es;
            // a nonzero scale anywhere sends the combine through its scaled path
            if (__builtin_amdgcn_ballot_w64(live && es != 0) != 0 && lane == 0) a.ntiles[2] = 1;
            wave_lds_sync();
            const int c = lane & 7;                          // 8 lanes per row of 64 columns
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int rw = 8 * q + (lane >> 3);
                const u32x4 v = *(const u32x4 *)(ep + rw * PITCH + 16 * c);
                const int64_t pr = __shfl((int)p, rw);
                if (32 * i + rw < nrows) *(u32x4 *)(a.slot + pr * H + col + 8 * c) = v;
            }
            wave_lds_sync();
        }
    }
}

}  // namespace

hipError_t launch_mx_group(const Layer &L, const uint16_t *x, int64_t T, const PrefillBufs &b, hipStream_t s) {
    GroupArgs a{};
    a.L = L;
    a.x = x;
    a.T = T;
    a.h = b.h;
    a.perm = b.perm;
    a.tiles = b.tiles;
    a.ntiles = b.ntiles;
    a.w = b.w;
    a.sgate = (L.shared_gate_w && L.has_shared) ? b.sgate : nullptr;
    a.slot = b.slot;
    a.sexp = b.sexp;
    const int64_t tiles = prefill_max_tiles(T, L.K, L.E);
    auto grid = [&](int nb) { return dim3((unsigned)((tiles + 7) / 8 * 8 * nb)); };
    a.nb = (L.I + 127) / 128;
    hipLaunchKernelGGL(k_mx_group<false>, grid(a.nb), dim3(64 * GW), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.nb = (L.H + 255) / 256;
    hipLaunchKernelGGL(k_mx_group<true>, grid(a.nb), dim3(64 * GW), 0, s, a);
    return hipGetLastError();
}

}  // namespace qs
