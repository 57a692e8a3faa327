// Angles of rotary positions: cosine and sine of a fraction of a turn in 64-bit
// fixed point, and indexes of two widths.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace q4dev {

__device__ __forceinline__ long long index_at(const void* p, int wide, int i)
{
    return wide ? static_cast<const long long*>(p)[i] : (long long)static_cast<const int*>(p)[i];
}

__device__ __forceinline__ float2 turn_cos_sin(uint64_t f)
{
    const uint64_t g = f + (1ull << 61);
    const uint32_t quad = (uint32_t)(g >> 62);
    const uint64_t r = f - ((uint64_t)quad << 62);      // signed, in [-2^61, 2^61)
    const float t = __builtin_fmaf((float)(uint32_t)r, 0x1p-64f, (float)(int32_t)(uint32_t)(r >> 32) * 0x1p-32f);
    const float x = t * 6.283185307179586f, y = x * x;
    float s = __builtin_fmaf(y, 1.f / 362880, -1.f / 5040);
    s = __builtin_fmaf(y, s, 1.f / 120);
    s = __builtin_fmaf(y, s, -1.f / 6);
    s = __builtin_fmaf(x * y, s, x);
    float c = __builtin_fmaf(y, -1.f / 3628800, 1.f / 40320);
    c = __builtin_fmaf(y, c, -1.f / 720);
    c = __builtin_fmaf(y, c, 1.f / 24);
    c = __builtin_fmaf(y, c, -0.5f);
    c = __builtin_fmaf(y, c, 1.f);
    const float a = (quad & 1) ? s : c, b = (quad & 1) ? c : s;   // |cos|, |sin| of the quadrant
    return float2{(quad == 1 || quad == 2) ? -a : a, (quad & 2) ? -b : b};
}

// The same in 64 bits, off by some 2^-50: keys that are rounded to few bits next, where a value
// beside a border is decided by the last bits of fp32. (The first omitted terms, of x^19 / 19! and
// x^20 / 20! at pi / 4, are 8e-20 and 3e-21.)
__device__ __forceinline__ double2 turn_cos_sin64(uint64_t f)
{
    const uint64_t g = f + (1ull << 61);
    const uint32_t quad = (uint32_t)(g >> 62);
    const long long r = (long long)(f - ((uint64_t)quad << 62));      // in [-2^61, 2^61)
    const double x = (double)r * (6.283185307179586476925286766559 * 0x1p-64), y = x * x;
    double s = 0, c = 0;
    constexpr double S[] = {1. / 355687428096000, -1. / 1307674368000, 1. / 6227020800, -1. / 39916800, 1. / 362880, -1. / 5040, 1. / 120, -1. / 6};
    constexpr double C[] = {-1. / 6402373705728000, 1. / 20922789888000, -1. / 87178291200, 1. / 479001600, -1. / 3628800, 1. / 40320, -1. / 720, 1. / 24, -0.5};
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fma(y, s, S[i]);
#pragma unroll
    for (int i = 0; i < 9; ++i) c = __builtin_fma(y, c, C[i]);
    s = __builtin_fma(x * y, s, x);
    c = __builtin_fma(y, c, 1.);
    const double a = (quad & 1) ? s : c, b = (quad & 1) ? c : s;
    return double2{(quad == 1 || quad == 2) ? -a : a, (quad & 2) ? -b : b};
}

}  // namespace q4dev
