// mx4.h -- device helpers shared by the microscaled 4-bit (MX4) kernels.
//
// MX4: FP4 E2M1 elements in blocks of 32 along the reduction axis, one E8M0 scale byte
// per block, v = 2^(s - 127) e2m1(code); s = 255 makes the whole block NaN.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128 columns and applies
// a scale per operand row and 32-column block.  Its fp4 operands on gfx950 (lane l = n + 16 g,
// measured with one-hot operands):
//   operand   row n, columns 32 g .. 32 g + 31 (16 bytes), one MX block
//   scale     the byte of that block; one of the four bytes of the scale register, chosen by
//             an immediate
//   result    rows 4 g .. 4 g + 3 of the first operand, row n of the second
//
// Tile layout of MX4 matrices: rows in panels of 16, columns in steps of 128; tile (p, s)
// is the 1024 bytes of the fp4 operand in lane order, so a wave reads a tile with one
// contiguous 16-byte load per lane.  Scales are grouped by four steps ("quads"): per (panel,
// quad) one dword per lane, byte i for step 4 q + i.
//
// Where both operands are MX4 the scaled MFMA multiplies the tiles as they are: its products
// are exact there, and so are their sums of 8 (a group of 8 products is aligned to its largest
// with 13 bits below it, and MX4 products span 7).  bf16 activations do not go that way: as two
// e4m3 parts they would, at one instruction each, but the same alignment drops bits of small
// products next to large ones (2e-5 of the result, measured).  They meet the weights on
// v_mfma_f32_16x16x32_bf16 instead: v_cvt_scalef32_pk_bf16_fp4 turns two codes and their
// block's scale into two bf16 (exact: an element has two significant bits and bf16 the range of
// the scale; the instruction takes the scale's exponent byte as it is, 0 and 255 included), so
// every product is exact and only the fp32 sums round.  A lane's 16 bytes of a tile are the
// operand of four such MFMAs: number j takes columns 32 g + 8 j .. + 7 of each lane group g.
#pragma once
#include "common.h"
#include "internal.h"

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

namespace qs {

namespace {

constexpr int MX_FP4 = 4;                   // operand format of the scaled MFMA
constexpr int MX_TILE = 1024;               // bytes of a 16 x 128 tile of codes
constexpr int MX_QS = 256;                  // bytes of a (panel, quad) of scales

__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {      // s <= 254
    return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// largest |value| of 8 bf16 as bf16 bits
__device__ __forceinline__ uint32_t absmax8_bf16(u32x4 v) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
    return m[0] > m[1] ? m[0] : m[1];
}

// 8 codes (one dword) under a scale (its byte in the exponent bits of an fp32) as bf16
__device__ __forceinline__ bf16x8 mx_bf16(uint32_t c, float s) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    return __builtin_bit_cast(bf16x8, r);
}
// byte i of a quad's scale dword as that fp32
__device__ __forceinline__ float mx_scale(uint32_t sw, int i) {
    return __uint_as_float(((sw >> (8 * i)) & 255u) << 23);
}

__device__ __forceinline__ i32x8 frag4(u32x4 a) {
    return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
}

// fp4 x fp4 over one step, with the scale bytes of step i (0..3) of a quad
__device__ __forceinline__ f32x4 mx_mfma(u32x4 a, u32x4 b, f32x4 c, int i, uint32_t sa, uint32_t sb) {
    const i32x8 A = frag4(a), B = frag4(b);
    switch (i) {
        case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, MX_FP4, MX_FP4, 0, (int)sa, 0, (int)sb);
        case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, MX_FP4, MX_FP4, 1, (int)sa, 1, (int)sb);
        case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, MX_FP4, MX_FP4, 2, (int)sa, 2, (int)sb);
        default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, MX_FP4, MX_FP4, 3, (int)sa, 3, (int)sb);
    }
}

// the 32 x 32 form over 64 columns: lane r + 32 h holds row r, columns 32 h .. 32 h + 31
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mx_mfma32(u32x4 a, u32x4 b, f32x16 c, int i, uint32_t sa, uint32_t sb) {
    const i32x8 A = frag4(a), B = frag4(b);
    switch (i) {
        case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, MX_FP4, MX_FP4, 0, (int)sa, 0, (int)sb);
        case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, MX_FP4, MX_FP4, 1, (int)sa, 1, (int)sb);
        case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, MX_FP4, MX_FP4, 2, (int)sa, 2, (int)sb);
        default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, MX_FP4, MX_FP4, 3, (int)sa, 3, (int)sb);
    }
}

// Direct-to-LDS loads (lane l's bytes land at l times their number) through a buffer resource over
// everything from a wave-uniform pointer on: voff per lane, soff uniform, both in bytes and below
// 2^31; and the waits for them.  Beside loads into registers only this form will do: the compiler
// cannot count global_load_lds among them (it may be LDS or memory that a flat instruction waits
// for) and would wait for every load there is.
typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const void *p) {
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(lo | (uint64_t)hi << 32), 0, 0xffffffffu, 0x00020000);
}
__device__ __forceinline__ void dma16_buffer(__amdgpu_buffer_rsrc_t r, void *l, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)l, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4_buffer(__amdgpu_buffer_rsrc_t r, void *l, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)l, 4, voff, soff, 0, 0);
}
template <int N>
__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// this wave's LDS reads are complete and every wave has arrived
__device__ __forceinline__ void block_sync() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// LDS writes of this wave before its later reads
__device__ __forceinline__ void wave_lds_sync() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ void mx_store(void *y, int64_t i, float v, int y_dtype) {
    if (y_dtype == MOE_F32) ((float *)y)[i] = v;
    else ((uint16_t *)y)[i] = f32_to_bf16(v);
}

}  // namespace

}  // namespace qs
