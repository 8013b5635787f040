// int4.cuh -- KV-cache rows of 4-bit whole numbers, one 8-bit scale per 32 values.
//
// A row of 128 values x is four groups of 32.  A group's scale s is the smallest UE5M3 number (5
// exponent and 3 mantissa bits: the upper byte of an fp16 without its sign, so that fp16(s) is
// the byte shifted left by 7) with 7 s >= max|x|, at most 896; a value is stored as
// n = x / s rounded to nearest, ties to even, |n| <= 7, and reads back as n s.  A uniform step
// instead of a 4-bit float's: on normal values of unit size the rms error is 0.104, against 0.115
// for 4-bit floats (E2M1) with a power-of-two scale per 32.
//
// n s has 3 + 4 significant bits, so it is exact in bf16 and in fp16 (below
// 2^-14 both count in multiples of 2^-17): the decode (fp16 operands) and the prefill (bf16
// operands) see the same values.
//
// Codes: 64 bytes a row; 32-bit word w holds the values 8 w .. 8 w + 7 as u = n + 8 (1 .. 15),
// value 8 w + 2 i in bits 4 i and value 8 w + 2 i + 1 in bits 16 + 4 i, so that one mask takes a
// pair of neighbours into the two halves of an fp16x2.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace inkattn {

constexpr int kI4Group = 32;                       // values of a scale
constexpr int kI4RowBytes = 64;                    // codes of a row of 128
constexpr int kI4RowScales = 4;                    // scales of a row of 128
constexpr uint32_t kI4ScaleMax = 0xC6u;            // 896: 72 * 896, the expansion's offset, is finite in fp16

constexpr float kI4Max = 7.f * 896.f;              // the largest value

__device__ __forceinline__ float i4_scale(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}
// The byte of the smallest scale s with 7 s >= amax, amax <= kI4Max.
__device__ __forceinline__ uint32_t i4_scale_byte(float amax) {
    // amax / 7 from below by at most two units of the last place, up to the next scale; a scale that lies
    // between the two is told by 7 s, which is exact
    const float t = __fmul_rd(amax, 0x1.249248p-3f);
    uint32_t b;
    if (t >= 0x1p-14f) b = ((__float_as_uint(t) + 0xFFFFFu) >> 20) - ((127u - 15u) << 3);   // mantissa up to 3 bits
    else b = (uint32_t)__float2int_ru(t * 0x1p17f);                                       // multiples of 2^-17
    return 7.f * i4_scale(b) < amax ? b + 1 : b;
}
// n = x / s to nearest, ties to even, of two values, as u = n + 8 in the low halves of the results; |x| <= 7 s,
// inv = 1 / s but for 2^-20 of it.  x / s is a tie or lies 2^-9 of it from one (x has 8 significant bits and so
// has (n + 1/2) s): rounded to multiples of 2^-11 first, by a sum that ends there, a tie is exact and the
// others stay on their side.
__device__ __forceinline__ float2 i4_codes2(float2 x, float inv) {
    constexpr float kStep = 0x1.8p12f;             // sums with it end at 2^-11
    constexpr float kMagic = 0x1.8p23f + 8.f;      // and with this at 1: the sum's low bits are those of n + 8
    const float2 t = ffma2(x, make_float2(inv, inv), make_float2(kStep, kStep));
    return fadd2(t, make_float2(kMagic - kStep, kMagic - kStep));
}
// A lane's eight values of a row (packed bf16, a group in four neighbouring lanes of a converged warp) as a word
// of codes, and the group's scale byte.
__device__ __forceinline__ void i4_encode(const uint4 &row, uint32_t &word, uint32_t &byte) {
    const uint32_t mag = 0x7FFF7FFFu;
    uint32_t m = max_u16x2(max_u16x2(row.x & mag, row.y & mag), max_u16x2(row.z & mag, row.w & mag));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    float amax = fmaxf(__uint_as_float(m & 0x7FFF0000u), __uint_as_float(m << 16));
    const uint32_t w[4] = {row.x, row.y, row.z, row.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
    // rare: a value beyond the largest, an infinity or a NaN (whose bits are larger still) in the group: a NaN
    // counts as 0, the others saturate
    if (max(m & 0x7FFFu, m >> 16) > (__float_as_uint(kI4Max) >> 16)) {
        amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] == x[e] ? fminf(fmaxf(x[e], -kI4Max), kI4Max) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        const uint32_t group = 0xFu << ((threadIdx.x & 31) & ~3);          // (the four lanes alike)
        amax = fmaxf(amax, __shfl_xor_sync(group, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(group, amax, 2));
    }
    byte = i4_scale_byte(amax);
    float inv = 0.f;
    if (byte) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(i4_scale(byte)));
    uint32_t pair[4];                              // of neighbours, a code in each half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = i4_codes2(make_float2(x[2 * i], x[2 * i + 1]), inv);
        pair[i] = __byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x5410);
    }
    word = (pair[0] | pair[1] << 4) | (pair[2] << 8 | pair[3] << 12);
}

// A group's scale as the two factors of i4_decode8: s and -72 s.
struct I4Scale {
    __half2 s, off;
};
__device__ __forceinline__ I4Scale i4_factors(uint32_t byte) {
    const uint32_t h = byte << 7;
    const uint32_t two = h | (h << 16);
    I4Scale f;
    f.s = *reinterpret_cast<const __half2 *>(&two);
    f.off = __hmul2(f.s, __float2half2_rn(-72.f));
    return f;
}
// Eight values of a word as four fp16x2 in order.  A code u placed in bits 4 .. 7 under the exponent of 64
// (16 units of the last place are 1) is 64 + u; (64 + u) s - 72 s = n s in one fused step, exact:
// 72 s = 9 s * 8 has at most 8 significant bits.  3 shifts, 4 masks and 4 multiply-adds a word, and
// the SM has 4096 words to expand for every 128 keys: with `mask` and `exponent` (kI4Mask, kI4Exponent)
// in registers or a kernel's parameters a mask is one instruction, with literals it is two (10 cycles a word
// of a scheduler against 15).
constexpr uint32_t kI4Mask = 0x00F000F0u, kI4Exponent = 0x54005400u;
__device__ __forceinline__ uint4 i4_decode8(uint32_t w, const I4Scale &f, uint32_t mask, uint32_t exponent) {
    const uint32_t at[4] = {w << 4, w, w >> 4, w >> 8};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t m;                                // (at & mask) | exponent
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(m) : "r"(at[i]), "r"(mask), "r"(exponent));
        const __half2 v = __hfma2(*reinterpret_cast<const __half2 *>(&m), f.s, f.off);
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace inkattn
