// Low-rank adapters of many requests beside one quantized product:
//   y[m] = x[m] W + bias + c_a B_a,p (A_a,p x[m]),  a = index[m],
// for the columns of part p (the layers a handle concatenates; one otherwise).
//
// The bank keeps A as [slot][part][rank][K] and B in the order in which the matrix
// instructions take it: [slot][32 columns][8 of rank][column][value], rank rounded up
// to rp, a multiple of 8, and columns to 32, with zeros. A first launch forms c A x
// (q4_adapters.hip), the product's own launch adds B (c A x) to its fp32 sums.
#pragma once

#include <hip/hip_runtime.h>

#include "q4_device.h"

namespace q4dev {

// A position in the order of the adapters: its row of the call, its adapter (-1:
// none) and the position at which that adapter's rows end.
struct AdapterRow {
    int row, slot, end, pad;
};

struct AdapterArgs {
    const uint16_t* B;       // [slots][b_slot]
    const uint8_t* part8;    // part of columns 8i .. 8i + 7, or null: one part
    size_t b_slot;           // values of a slot's B
    int slots, rp, width;    // width = parts * rp: values of c A x a row
    // few rows: in their own order, fp32
    const int* index;        // [M]
    const float* t;          // [M][width]
    // many rows: in the order of their adapters (rows without one last)
    const AdapterRow* rows;  // [positions]
    // c A x rounded, and what that leaves: [positions / 32][width / 8][position][value]
    const uint16_t *hi, *lo;
};

// Values between two 8-value chunks of one column of B, or of one position of c A x.
constexpr int kChunk = 32 * 8;

// What row m's adapter adds to column n: `rank` terms in fp32.
template <bool BF>
__device__ __forceinline__ float adapter_row(const AdapterArgs& a, int m, int n)
{
    const int s = a.index[m];
    if ((unsigned)s >= (unsigned)a.slots) return 0.f;
    const int part = a.part8 ? a.part8[n >> 3] : 0;
    const float* t = a.t + (size_t)m * a.width + part * a.rp;
    const uint16_t* b = a.B + s * a.b_slot + ((size_t)(n >> 5) * a.rp * 32 + (n & 31) * 8);
    float y = 0.f;
    for (int j = 0; j < a.rp; j += 8) {
        const u4 v = *reinterpret_cast<const u4*>(b + j / 8 * kChunk);
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
// (lane: column n0 + l32, rows 8 (r / 4) + 4 lhi + r % 4). seg[i], in LDS, is the
// adapter of position m0 + i (-1: none, or past the last) and where its rows end.
//
// Bound: latency, so operands are asked for ahead: 32 values of rank at a time, the
// next 32 positions' c A x and the next adapter's B while the present ones are
// multiplied. Each operand is one dense KiB of its 32 positions or columns.
//
// A tile that is one adapter's takes its products directly; one that several
// share (or whose columns are of several parts) takes each through a result of
// its own, so that values of one request that are not finite stay its own.
template <bool BF, int MI, class Acc>
__device__ __forceinline__ void adapter_tile(const AdapterArgs& a, const int2* seg, int m0, int n0, int N, int l32, int lhi, Acc&& acc)
{
    constexpr int KC = 2;               // 16-value steps of rank at a time
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    if (uniform(seg[0].x) < 0) return;
    int mine = 0, first = 0, last = 0;
    if (a.part8) {
        mine = a.part8[min(n0 + l32, N - 1) >> 3];
        first = uniform(a.part8[min(n0, N - 1) >> 3]);
        last = uniform(a.part8[min(n0 + 31, N - 1) >> 3]);
    }
    auto mma = [](u4 x, u4 y, f16x c) {
        if constexpr (BF) return mfma32(bitcast<b8>(x), bitcast<b8>(y), c);
        else return mfma32(bitcast<h8>(x), bitcast<h8>(y), c);
    };
    const u4 zero = u4{0, 0, 0, 0};
    const uint16_t* bn = a.B + (size_t)(min(n0, N - 1) >> 5) * a.rp * 32 + l32 * 8;
    const uint16_t* tn = a.hi + (size_t)(m0 >> 5) * a.width * 32 + l32 * 8;
    const ptrdiff_t to_lo = a.lo - a.hi;
    for (int part = first; part <= last; ++part)
        for (int k = 8 * lhi; k - 8 * lhi < a.rp; k += 16 * KC) {
            u4 h[KC], l[KC], nh[KC], nl[KC], nb[KC];
            auto load_t = [&](int i) {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const bool in = k + 16 * c < a.rp;
                    const uint16_t* t = tn + ((size_t)i * a.width + part * a.rp + k + 16 * c) * 32;
                    nh[c] = in ? *reinterpret_cast<const u4*>(t) : zero;
                    nl[c] = in ? *reinterpret_cast<const u4*>(t + to_lo) : zero;
                }
            };
            auto load_b = [&](int s) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    nb[c] = k + 16 * c < a.rp && mine == part
                                ? *reinterpret_cast<const u4*>(bn + s * a.b_slot + (size_t)(k + 16 * c) * 32) : zero;
            };
            int r = 0, s = uniform(seg[0].x);   // the next position, its adapter
            load_t(0);
            load_b(s);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
                for (int c = 0; c < KC; ++c) h[c] = nh[c], l[c] = nl[c];
                if (i + 1 < MI && s >= 0) load_t(i + 1);
#pragma clang loop unroll(disable)
                while (s >= 0 && r < 32 * i + 32) {
                    u4 b[KC];
#pragma unroll
                    for (int c = 0; c < KC; ++c) b[c] = nb[c];
                    const int from = r;
                    r = min(32 * i + 32, uniform(seg[r].y) - m0);
                    s = r < 32 * MI ? uniform(seg[r].x) : -1;
                    if (s >= 0) load_b(s);
                    if (first == last && r - from == 32) {
#pragma unroll
                        for (int c = 0; c < KC; ++c) acc(i) = mma(l[c], b[c], mma(h[c], b[c], acc(i)));
                    } else {
                        f16x y;
#pragma unroll
                        for (int v = 0; v < 16; ++v) y[v] = 0.f;
#pragma unroll
                        for (int c = 0; c < KC; ++c) y = mma(l[c], b[c], mma(h[c], b[c], y));
                        const int lo = from - 32 * i - 4 * lhi, hi = mine == part ? r - 32 * i - 4 * lhi : -1;
#pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const int m = 8 * (v >> 2) + (v & 3);
                            acc(i)[v] += m >= lo && m < hi ? y[v] : 0.f;
                        }
                    }
                }
            }
        }
}

}  // namespace q4dev
