// Low-rank adapters of many requests beside one quantized product:
//   y[m] = x[m] W + bias + c_a B_a,p (A_a,p x[m]),  a = index[m],
// for the columns of part p (the layers a handle concatenates; one otherwise).
//
// The bank keeps A as [slot][part][rank][K] and B as [slot][N][rp], rp the rank
// rounded up to 8 with zeros. A first launch forms c A x (q4_adapters.hip), the
// product's own launch adds B (c A x) to its fp32 sums.
#pragma once

#include <hip/hip_runtime.h>

#include "q4_device.h"

namespace q4dev {

struct AdapterArgs {
    const uint16_t* B;       // [slots][N][rp]
    const uint8_t* part8;    // part of columns 8i .. 8i + 7, or null: one part
    int slots, rp, width;    // width = parts * rp: values of c A x a row
    // few rows: in their own order, fp32
    const int* index;        // [M]
    const float* t;          // [M][width]
    // many rows: in the order of their adapters (rows without one last)
    const int* rows;         // position -> row, padded to whole fours
    const int* slot_of;      // position -> adapter
    const int* seg;          // [slots + 2] first position of each adapter's rows
    const uint16_t *hi, *lo; // [positions][width], rounded and what that leaves
};

// What row m's adapter adds to column n: `rank` terms in fp32.
template <bool BF>
__device__ __forceinline__ float adapter_row(const AdapterArgs& a, int m, int n, int N)
{
    const int s = a.index[m];
    if ((unsigned)s >= (unsigned)a.slots) return 0.f;
    const int part = a.part8 ? a.part8[n >> 3] : 0;
    const float* t = a.t + (size_t)m * a.width + part * a.rp;
    const uint16_t* b = a.B + ((size_t)s * N + n) * a.rp;
    float y = 0.f;
    for (int j = 0; j < a.rp; j += 8) {
        const u4 v = *reinterpret_cast<const u4*>(b + j);
        const f4 t0 = *reinterpret_cast<const f4*>(t + j), t1 = *reinterpret_cast<const f4*>(t + j + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float t_lo = e < 2 ? t0[2 * e] : t1[2 * e - 4], t_hi = e < 2 ? t0[2 * e + 1] : t1[2 * e - 3];
            y = __builtin_fmaf(t_lo, act_to_f32<BF>((uint16_t)v[e]), y);
            y = __builtin_fmaf(t_hi, act_to_f32<BF>((uint16_t)(v[e] >> 16)), y);
        }
    }
    return y;
}

// Adds the adapters of positions m0 .. m0 + 32 MI - 1 to a wave's accumulators:
// acc(i) is the 32 x 32 tile of positions m0 + 32 i .. and columns n0 .. n0 + 31
// (lane: column n0 + l32, rows 8 (r / 4) + 4 lhi + r % 4). A tile that is one
// adapter's takes its products directly; one that several share (or whose
// columns are of several parts) takes each through a result of its own, so
// that values of one request that are not finite stay its own.
template <bool BF, int MI, class Acc>
__device__ __forceinline__ void adapter_tile(const AdapterArgs& a, int m0, int n0, int N, int l32, int lhi, Acc&& acc)
{
    const int end = min(m0 + 32 * MI, __builtin_amdgcn_readfirstlane(a.seg[a.slots]));
    if (m0 >= end) return;
    const int n = min(n0 + l32, N - 1);
    int mine = 0, first = 0, last = 0;
    if (a.part8) {
        mine = a.part8[n >> 3];
        first = __builtin_amdgcn_readfirstlane(a.part8[min(n0, N - 1) >> 3]);
        last = __builtin_amdgcn_readfirstlane(a.part8[min(n0 + 31, N - 1) >> 3]);
    }
    auto mma = [](u4 x, u4 y, f16x c) {
        if constexpr (BF) return mfma32(bitcast<b8>(x), bitcast<b8>(y), c);
        else return mfma32(bitcast<h8>(x), bitcast<h8>(y), c);
    };
    for (int r = m0; r < end;) {
        const int s = __builtin_amdgcn_readfirstlane(a.slot_of[r]);
        const int e = min(end, __builtin_amdgcn_readfirstlane(a.seg[s + 1]));
        const uint16_t* bn = a.B + ((size_t)s * N + n) * a.rp;
        for (int part = first; part <= last; ++part)
            for (int k = 0; k < a.rp; k += 16) {
                const int at = k + 8 * lhi;
                const bool in = at < a.rp;
                const u4 zero = u4{0, 0, 0, 0};
                const u4 b = in && mine == part ? *reinterpret_cast<const u4*>(bn + at) : zero;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const int t0 = m0 + 32 * i;
                    if (t0 + 32 <= r || t0 >= e) continue;
                    const size_t off = (size_t)(t0 + l32) * a.width + part * a.rp + at;
                    const u4 h = in ? *reinterpret_cast<const u4*>(a.hi + off) : zero;
                    const u4 l = in ? *reinterpret_cast<const u4*>(a.lo + off) : zero;
                    if (first == last && r <= t0 && e >= t0 + 32) {
                        acc(i) = mma(l, b, mma(h, b, acc(i)));
                    } else {
                        f16x y;
#pragma unroll
                        for (int q = 0; q < 16; ++q) y[q] = 0.f;
                        y = mma(l, b, mma(h, b, y));
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const int m = t0 + 8 * (q >> 2) + 4 * lhi + (q & 3);
                            if (m >= r && m < e && mine == part) acc(i)[q] += y[q];
                        }
                    }
                }
            }
        r = e;
    }
}

}  // namespace q4dev
