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

// The byte of the smallest scale that holds a group of largest magnitude amax (NaN counts as 0;
// above 7 * 896 the largest, and the values saturate).
__device__ __forceinline__ uint32_t i4_scale_byte(float amax) {
    if (!(amax > 0.f)) return 0u;
    // amax / 7 rounded up: no scale lies between the quotient and its rounding, since every
    // scale is a float
    const float t = __fdiv_ru(amax, 7.f);
    const uint32_t u = __float_as_uint(t);
    uint32_t b;
    if (t >= 0x1p-14f) b = ((u + 0xFFFFFu) >> 20) - ((127u - 15u) << 3);   // mantissa up to 3 bits
    else b = (uint32_t)__float2int_ru(t * 0x1p17f);                        // multiples of 2^-17
    return b < kI4ScaleMax ? b : kI4ScaleMax;
}
__device__ __forceinline__ float i4_scale(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}
// The word of eight values.  The quotient by division, not by a reciprocal's product: n + 1/2 is
// reached exactly by bf16 values, and a tie has to be seen as one.  (Any other quotient lies further
// from a tie than fp32's rounding, x having 8 significant bits and (n + 1/2) s as many.)
__device__ __forceinline__ uint32_t i4_encode8(const float (&x)[8], float s) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float n = s > 0.f ? rintf(__fdiv_rn(x[e], s)) : 0.f;
        n = n == n ? fminf(fmaxf(n, -7.f), 7.f) : 0.f;                     // (a NaN is stored as 0)
        w |= (uint32_t)((int)n + 8) << (4 * (e >> 1) + 16 * (e & 1));
    }
    return w;
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
