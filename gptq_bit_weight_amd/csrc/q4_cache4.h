// The cache held in 4 bits: what its codes stand for, in registers.
//
// A row of a head is dim / 2 bytes of codes, value 2 i in the low half of byte i and
// 2 i + 1 in the high half, and for each group of 32, 64, 128 or 256 neighbouring values a
// word of two binary16: the step s (low half) and the least value m. Code c stands for
// the binary16 value RNE(s c + m): one packed multiply-add for two values, which the
// matrix instructions take as they are.
//
// Codes become binary16 as in q4_device.h: or-ed into the fraction of 1024 (low halves of bytes)
// or, where they sit, of 64 (high halves), less 1024 or 64: exact.
#pragma once

#include "q4_device.h"

namespace q4cache4 {

using namespace q4dev;

constexpr float kLargest = 65440.f;     // finite values beyond it are held as it: s 15 + m, with s rounded up, stays finite

// A half of a word in both halves (the packed instructions select it).
__device__ __forceinline__ h2 low_half(uint32_t w)
{
    const h2 v = bitcast<h2>(w);
    return h2{v[0], v[0]};
}
__device__ __forceinline__ h2 high_half(uint32_t w)
{
    const h2 v = bitcast<h2>(w);
    return h2{v[1], v[1]};
}

// The constants that codes are or-ed into, 1024 and 64 in both halves. (One v_and_or_b32
// takes its mask from a scalar register and this from a vector one; the compiler must not see the values.)
struct Magic {
    uint32_t low, high;
};
__device__ __forceinline__ Magic magic()
{
    Magic m{0x64006400u, 0x54005400u};
    asm volatile("" : "+v"(m.low), "+v"(m.high));
    return m;
}

// (codes in bits 0..3 and 16..19; in bits 4..7 and 20..23)
__device__ __forceinline__ uint32_t value_low(uint32_t w, h2 step, h2 least, const Magic& g)
{
    const h2 c = bitcast<h2>(and_or(w, 0x000f000fu, g.low)) - bitcast<h2>(0x64006400u);
    return bitcast<uint32_t>(__builtin_elementwise_fma(c, step, least));
}
__device__ __forceinline__ uint32_t value_high(uint32_t w, h2 step, h2 least, const Magic& g)
{
    const h2 c = bitcast<h2>(and_or(w, 0x00f000f0u, g.high)) - bitcast<h2>(0x54005400u);
    return bitcast<uint32_t>(__builtin_elementwise_fma(c, step, least));
}

// A word's eight values, in the order 0 4, 1 5, 2 6, 3 7.
__device__ __forceinline__ u4 values8(uint32_t w, h2 step, h2 least, const Magic& g)
{
    return u4{value_low(w, step, least, g), value_high(w, step, least, g), value_low(w >> 8, step, least, g), value_high(w >> 8, step, least, g)};
}

// Eight 16-bit values in that order.
__device__ __forceinline__ u4 code_order(u4 x)
{
    return u4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
              __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}
// and back in their own.
__device__ __forceinline__ u4 own_order(u4 x)
{
    return u4{__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
              __builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}

// Two rows' values of byte b of a word of each: its first (even) and second (odd)
// column, in the low half the first row's, with the rows' steps and least values in pairs.
__device__ __forceinline__ u2 values_of_pair(uint32_t w0, uint32_t w1, int b, h2 step, h2 least, const Magic& g)
{
    const uint32_t x = __builtin_amdgcn_perm(w1, w0, 0x0c040c00u + 0x00010001u * (uint32_t)b);
    return u2{value_low(x, step, least, g), value_high(x, step, least, g)};
}

// Queries of bfloat16 as binary16: a row is multiplied by the power of two that brings its
// largest magnitude to 2^14 .. 2^15 (one within 2^-112 .. 2^127), so its values keep all their
// bits down to 2^-17, 2^-31 of the largest; the scores are multiplied by the inverse.
__device__ __forceinline__ uint32_t largest_bf16(u4 x)
{
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) t = max(t, max(x[e] << 16 & 0x7fff0000u, x[e] & 0x7fff0000u));
    return t;                           // (bits of a float)
}
__device__ __forceinline__ uint32_t exponent_of(float most) { return min(max(bitcast<uint32_t>(most) >> 23 & 255u, 15u), 254u); }
__device__ __forceinline__ float halve_range(float most) { return bitcast<float>((exponent_of(most) - 14u) << 23); }
// The scores' factor with that inverse, held within fp32's range: at 0 a masked score of -inf would
// be NaN, and at infinity one of 0. (Scores under the least factor are all 0 to what a weight is rounded to.)
__device__ __forceinline__ float row_scale(float scale, float most)
{
    return fminf(fmaxf(scale * halve_range(most), 1.1754943508222875e-38f), 3.4028234663852886e38f);
}
__device__ __forceinline__ u4 bf16_to_f16(u4 x, float most)
{
    const float f = bitcast<float>((268u - exponent_of(most)) << 23);
    u4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float lo = bitcast<float>(x[e] << 16) * f, hi = bitcast<float>(x[e] & 0xffff0000u) * f;
        r[e] = (uint32_t)f32_to_f16_bits(lo) | (uint32_t)f32_to_f16_bits(hi) << 16;
    }
    return r;
}

}  // namespace q4cache4
