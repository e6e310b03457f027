// mx4_group.hip -- the expert products of a prompt with MX4 experts, on v_mfma 32x32x16 bf16.
//
// Work comes from the grouped path's block map: tiles of up to GEMM_BM = 160 rows of one
// expert's bin (or of the shared expert), each against column blocks of 256 weight rows, one
// launch for [gate; up] and one for down.  Four waves; a wave takes 64 weight rows (two
// fragments of 32) against the tile's rows (five fragments, only as many as the tile fills),
// the weights as first operand, so that a lane's registers are neighbouring columns.
//
// Data movement as in the large tiles of mx4_gemm.hip: activation rows global -> LDS in a ring of
// three stages of 64 columns (128 bytes a row, chunks XORed by (row / 2) % 8), each wave's weights
// straight into its registers, both two steps ahead; two workgroups fit a compute unit, and one's
// prologue and epilogue run under the other's products.  T = 4096, 2048 x 512, top 8 of 256 experts
// and a shared one, skewed router: 474 -> 425 us a layer against weights through LDS in a ring of two;
// fragments past a tile's rows skipped by a branch each (T = 512: 154 us; all five multiplied: 184).
// With every expert as likely T = 4096 takes 403 us: gate/up 170, matrix cores busy half of the
// cycles (about 128 rows a tile, 32 steps and then its h), down 193, busy 0.44 (16 steps, then its slot
// rows); the router, binning and combine the rest.  T = 512 takes 209: 91 and 85 for 430 MB of weights,
// with 16 rows a tile too little work to hide the wait for them (busy 0.15).
//
//   gate/up  rows of x gathered through perm; the wave's fragments are 32 gate rows and the
//            same 32 up rows, so h = silu(g) u is formed in registers.  It leaves as the bf16
//            pair hi + lo (h to 2^-17), [row][hi, lo][I].
//   down     rows of h; the reduction runs over hi, then over lo, each against the same weights
//            (a third more matrix work than bf16 h, which would leave 2e-3 x RMS of error in the
//            layer).  Slot rows as the affine path writes them: w o in fp16 under a scale per row
//            and 64 columns (a wave's), for the same combine.  One rounding of each summand of y
//            (2e-4 of y's norm; bf16 y alone rounds to 2e-3), for half the bytes of fp32 rows:
//            151 MB written and read again at T = 4096.
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
constexpr int STAGE = GEMM_BM * 128, NSTAGE = 3;
constexpr int SC_SLOT = 256 * 16, RING = NSTAGE * STAGE + 2 * SC_SLOT;
constexpr int A_DMA = STAGE / (1024 * GW), S_DMA = 4;
constexpr int EP = 32 * (64 * 4 + 16);                       // a wave's epilogue staging
static_assert(GW * EP <= RING && GEMM_BM % 32 == 0 && STAGE % (1024 * GW) == 0, "tile shape");

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
    const uint8_t *bsrc[FN], *sbase[2];
    int soff[S_DMA];
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
        bsrc[j] = codes + (p0 + min(first + (r32 >> 4), np - 1)) * KS * MX_TILE + 16 * ((r32 & 15) + 16 * h);
        sbase[j] = scales + p0 * KQ * MX_QS;
#pragma unroll
        for (int i = 0; i < 2; ++i) soff[2 * j + i] = min(first + i, np - 1) * KQ * MX_QS + 4 * lane;
    }
    // ---- activation rows: piece i of a stage is rows 8 (A_DMA wave + i) .. + 7; their offsets
    // from abase (gate/up: below 2^31, the caller's chunks see to it)
    const void *abase = DOWN ? (const void *)(a.h + (int64_t)tile.row0 * 2 * I) : a.x;
    uint32_t aoff[A_DMA];
#pragma unroll
    for (int i = 0; i < A_DMA; ++i) {
        const int row = 8 * (A_DMA * wave + i) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
        const int r = row < nrows ? row : nrows - 1;         // (past the tile: its last row)
        if (DOWN) aoff[i] = (uint32_t)(r * 4 * I + 16 * c);
        else aoff[i] = (uint32_t)(sh ? tile.row0 + r - TK : (int64_t)(a.perm[tile.row0 + r] / K)) * (uint32_t)(2 * H) + 16 * c;
    }
    // step k's columns are 64 kb .. of the weights; slot: of the quad's scales
    auto issue = [&](int k, int kb, int slot) __attribute__((always_inline)) {
        uint8_t *st = sm + (k % NSTAGE) * STAGE;
#pragma unroll
        for (int i = 0; i < A_DMA; ++i)
            dma16_buffer(buffer_from(abase), st + (A_DMA * wave + i) * 1024, aoff[i], k * 128);
        if (kb % 8 == 0)                                     // a quad's scales; slots alternate
#pragma unroll
            for (int i = 0; i < S_DMA; ++i)
                dma4_buffer(buffer_from(sbase[i >> 1]), sm + NSTAGE * STAGE + slot * SC_SLOT + (S_DMA * wave + i) * 256,
                            soff[i], kb / 8 * MX_QS);
    };
    u32x4 bq[2][FN];                                         // weights, by the step's parity
    auto load_b = [&](int kb, u32x4 (&b)[FN]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = *(const u32x4 *)(bsrc[j] + kb * (MX_TILE / 2));
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
    uint32_t sw0[FN], sw1[FN];                               // scales of the quad's even and odd steps
    // step k of parity par, columns 64 kb of the weights; the next two steps' kb and scale slots
    struct Next {
        int kb, slot;
    };
    auto step = [&](int k, int par, Next c, bool quad1, Next n2, bool ahead) __attribute__((always_inline)) {
        // stage k has landed once at most step k + 1's loads are outstanding (quad1: scales too)
        if (!ahead && k + 1 >= steps) wait_dma<0>();
        else if (quad1) wait_dma<A_DMA + FN + S_DMA>();
        else wait_dma<A_DMA + FN>();
        block_sync();                                        // and frees stage k - 1
        if (ahead) issue(k + 2, n2.kb, n2.slot);
        if (c.kb % 8 == 0) {
            const uint8_t *ss = sm + NSTAGE * STAGE + c.slot * SC_SLOT + wave * 1024 + (r32 >> 4) * 256 +
                                4 * ((r32 & 15) + 16 * h);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                sw0[j] = *(const uint32_t *)(ss + 512 * j);
                sw1[j] = *(const uint32_t *)(ss + 512 * j + 128);
            }
        }
        const uint8_t *st = sm + (k % NSTAGE) * STAGE;
        float sc[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) sc[j] = mx_scale((c.kb & 1) ? sw1[j] : sw0[j], (c.kb >> 1) & 3);
#pragma unroll
        for (int m = 0; m < 4; ++m) {                        // columns 32 h + 8 m .. + 7
            bf16x8 A[FM], B[FN];
            const int pos = (4 * h + m) ^ ((r32 >> 1) & 7);
#pragma unroll
            for (int i = 0; i < FM; ++i) A[i] = *(const bf16x8 *)(st + (32 * i + r32) * 128 + 16 * pos);
#pragma unroll
            for (int j = 0; j < FN; ++j) B[j] = mx_bf16(bq[par][j][m], sc[j]);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                // (read above for every fragment: inside the branches each read would be waited for)
                asm volatile("" : "+v"(A[i]));
                if (i < nf)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(B[j], A[i], acc[j][i], 0, 0, 0);
            }
        }
        if (ahead) load_b(n2.kb, bq[par]);
    };
    auto start = [&](int k, Next n) __attribute__((always_inline)) {
        issue(k, n.kb, n.slot);
        load_b(n.kb, bq[k]);
        __builtin_amdgcn_sched_barrier(0);                   // (and the next step's after these)
    };
    // Whole quads of columns: every step's place in its quad is known, and with it the number of
    // loads outstanding, wherever the compiler waits for one.
    if (S % 8 == 0) {
        start(0, {0, 0});
        start(1, {1, 0});
        const int quads = steps / 8;
        int qb = 0;                                          // the quad of the weights
        for (int q = 0; q + 1 < quads; ++q) {
            const int qn = qb + 1 == KQ ? 0 : qb + 1;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                step(8 * q + s, s & 1, {8 * qb + s, q & 1}, s == 7,
                     s < 6 ? Next{8 * qb + s + 2, q & 1} : Next{8 * qn + s - 6, (q + 1) & 1}, true);
            qb = qn;
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
            step(steps - 8 + s, s & 1, {8 * qb + s, (quads - 1) & 1}, false, {8 * qb + s + 2, 0}, s < 6);
    } else {
        auto at = [&](int k) __attribute__((always_inline)) {
            const int kb = k < S ? k : k - S;                // (k < steps <= 2 S)
            return Next{kb, (kb / 8 + (k < S ? 0 : KQ)) & 1};
        };
        start(0, at(0));
        if (steps > 1) start(1, at(1));
        for (int k = 0; k < steps; k += 2)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (k + s >= steps) break;
                const bool ahead = k + s + 2 < steps;
                step(k + s, s, at(k + s), k + s + 1 < steps && at(k + s + 1).kb % 8 == 0, ahead ? at(k + s + 2) : Next{0, 0}, ahead);
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
