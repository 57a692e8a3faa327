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

#include <type_traits>

#include "q4_device.h"

namespace q4dev {

// A position in the order of the adapters: its row of the call, its adapter (-1:
// none) and whether that adapter's B has values that are not finite.
struct AdapterRow {
    int row, slot, wild, pad;
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
    // binary16: [stretch][up_pitch] what a position's values of a stretch were divided by, a
    // power of two (1 where they are in reach of the type)
    const float* up;
    int up_pitch;
};

// Values of a stretch of a part's rank: what is in LDS at a time, and has one scale.
constexpr int kStretch = 64;

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

template <int I, int N, class F>
__device__ __forceinline__ void each(F&& f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<I + 1, N>(f);
    }
}

// Adds the adapters of positions m0 .. m0 + 32 MI - 1 to the accumulators of a
// workgroup of NW waves, whose columns are n0 .. n0 + 32 NW - 1, 32 a wave: acc(i) is
// the 32 x 32 tile of positions m0 + 32 i .. (lane: column l32 of the wave's, rows 8 (r
// / 4) + 4 lhi + r % 4). seg[i], in LDS, is the adapter of position m0 + i (-1: none,
// or past the last; kWild added where its B has values that are not finite). lds_up
// takes a factor for each (binary16); lds_hi and lds_lo take 64 values of c A x of every position each; no load into
// them is under way, and all waves come here.
//
// Bound: latency. 64 values of rank at a time, the positions' c A x comes to LDS once for
// all waves; then each wave goes by runs, the positions of one adapter inside one tile,
// with the B of the next PF runs under way. The runs are bit masks, and their adapters
// lanes of a register. The product's launch with adapters and without (medians in a
// trace; the rows' gathering and scattering included): 2048 rows x 11008 columns, 8
// adapters of rank 64: 205 us and 178 (with operands from memory in rows of rank values, a
// run at a time, some 65 more); 77 rows, 12 of rank 32: 33.1 us and 24.3, about 2 of them the
// rows' map, the rest the latency of 8 MiB of B.
//
// Other rows of a run's tile meet it with zeros for their c A x; where the run's B has
// values that are not finite, its products are a result of their own, of which only
// its rows are added: values of one request that are not finite stay its own. So are
// the products of a run with a position whose c A x was scaled into binary16's reach.
constexpr int kWild = 1 << 20;
template <bool BF, int MI, int NW, class Acc>
__device__ __forceinline__ void adapter_tile(const AdapterArgs& a, const int* seg, float* lds_up, char* lds_hi, char* lds_lo, int m0, int n0, int N,
                                             int wave, int lane, Acc&& acc)
{
    constexpr int RC = kStretch, KC = RC / 16;   // values of rank in LDS, and their 16-value steps
    // steps that runs are gone through for, runs ahead (the accumulators of 256 rows
    // leave room for less)
    constexpr int KB = 2, PF = MI <= 2 ? 4 : 2;
    constexpr int J = MI / 2;              // groups of 64 positions
    static_assert(MI % 2 == 0 && MI * 2 * KC % NW == 0, "whole groups; whole loads of a wave");
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    if (uniform(seg[0]) < 0) return;
    const int l32 = lane & 31, lhi = lane >> 5, own = n0 + 32 * wave;
    int mine = 0, first = 0, last = 0, wg_first = 0, wg_last = 0;
    if (a.part8) {
        mine = a.part8[min(own + l32, N - 1) >> 3];
        first = uniform(a.part8[min(own, N - 1) >> 3]);
        last = uniform(a.part8[min(own + 31, N - 1) >> 3]);
        wg_first = uniform(a.part8[n0 >> 3]);
        wg_last = uniform(a.part8[min(n0 + 32 * NW - 1, N - 1) >> 3]);
    }
    // the adapters of 64 positions and where runs begin (the first position without
    // one begins the last, which ends all)
    int slot[J];
    uint64_t starts[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        slot[j] = seg[64 * j + lane];
        const int before = seg[max(64 * j + lane - 1, 0)];
        starts[j] = __ballot((lane & 31) == 0 || slot[j] != before);
    }
    auto mma = [](u4 x, u4 y, f16x c) {
        if constexpr (BF) return mfma32(bitcast<b8>(x), bitcast<b8>(y), c);
        else return mfma32(bitcast<h8>(x), bitcast<h8>(y), c);
    };
    const u4 zero = u4{0, 0, 0, 0};
    const uint16_t* bn = a.B + (size_t)(min(own, N - 1) >> 5) * a.rp * 32 + l32 * 8;
    const uint32_t to_hi = lds_address(lds_hi), to_lo = lds_address(lds_lo);
    bool fresh = true;
    for (int part = wg_first; part <= wg_last; ++part)
        for (int k = 0; k < a.rp; k += RC) {
            const int chunks = min(RC, a.rp - k) >> 3;       // 8-value chunks of this stretch
            if (!fresh) __syncthreads();
            fresh = false;
            // (asked for before the values and written to LDS after B is asked for)
            float up_mine = 1.f;
            const int up_at = 64 * wave + lane;
            if constexpr (!BF) {
                const size_t of = (size_t)(part * ((a.rp + RC - 1) / RC) + k / RC) * a.up_pitch;
                if (up_at < 32 * MI) up_mine = a.up[of + m0 + up_at];
            }
#pragma unroll
            for (int e = 0; e < MI * KC / NW; ++e) {
                const int at = wave + NW * e, tile = at / KC, pair = at % KC;
                if (2 * pair >= chunks) continue;
                // (a chunk past an odd number's last repeats it; it meets zeros of B)
                const size_t off = ((size_t)((m0 >> 5) + tile) * a.width + part * a.rp + k + 8 * min(2 * pair + lhi, chunks - 1)) * 32 + l32 * 8;
                dma_lane(reinterpret_cast<const char*>(a.hi + off), to_hi + (uint32_t)at * 1024u);
                dma_lane(reinterpret_cast<const char*>(a.lo + off), to_lo + (uint32_t)at * 1024u);
            }
            const bool wanted = part >= first && part <= last;
            u4 b[PF][KB];
            uint64_t ahead = 0;
            int c0 = 0;
            // (as many loads in every run, of something where there is no run left, so that
            // the compiler can count those newer than the one it waits for; with a branch
            // every run waits for all: 77 rows of 12 adapters 35.5 us against 34.0, 2048 of 8,
            // whose runs are long, the same within 1%)
            auto load = [&](int q, int j) __attribute__((always_inline)) {
                const int s = ahead ? __builtin_amdgcn_readlane(slot[j], (int)__builtin_ctzll(ahead)) : 0;
                ahead &= ahead - 1;
                const uint16_t* of = bn + (s < 0 ? 0 : s & (kWild - 1)) * a.b_slot + (size_t)k * 32;
#pragma unroll
                for (int c = 0; c < KB; ++c)
                    b[q][c] = *reinterpret_cast<const u4*>(of + min(2 * (c0 + c) + lhi, chunks - 1) * kChunk);
            };
            if (wanted) {
                ahead = starts[0];
#pragma unroll
                for (int q = 0; q < PF; ++q) load(q, 0);
            }
            if constexpr (!BF)
                if (up_at < 32 * MI) lds_up[up_at] = seg[up_at] >= 0 ? up_mine : 1.f;   // (none without an adapter)
            wait_loads<0>();
            __syncthreads();
            if (!wanted) continue;
            uint64_t scaled[J];                              // positions with a factor
#pragma unroll
            for (int j = 0; j < J; ++j) scaled[j] = BF ? 0 : __ballot(lds_up[64 * j + lane] != 1.f);
            for (; 2 * c0 < chunks; c0 += KB) {
                each<0, J>([&](auto group) __attribute__((always_inline)) {
                    constexpr int j = decltype(group)::value;
                    uint64_t runs = starts[j];
                    if (j || c0) {
                        ahead = runs;
#pragma unroll
                        for (int q = 0; q < PF; ++q) load(q, j);
                    }
                    auto run = [&](int q) __attribute__((always_inline)) {
                        if (!runs) return false;
                        const int from = (int)__builtin_ctzll(runs);
                        const int s = __builtin_amdgcn_readlane(slot[j], from);
                        runs &= runs - 1;
                        if (s < 0) return false;
                        const int to = runs ? (int)__builtin_ctzll(runs) : 64;
                        const bool in = l32 >= (from & 31) && l32 < (from & 31) + to - from;
                        const int at = ((2 * j + (from >> 5)) * KC + c0) * 1024 + lane * 16;
                        auto products = [&](f16x y) __attribute__((always_inline)) {
#pragma unroll
                            for (int c = 0; c < KB; ++c)
                                if (2 * (c0 + c) < chunks) {
                                    u4 h = *reinterpret_cast<const u4*>(lds_hi + at + c * 1024);
                                    u4 l = *reinterpret_cast<const u4*>(lds_lo + at + c * 1024);
#pragma unroll
                                    for (int v = 0; v < 4; ++v) h[v] = in ? h[v] : 0u, l[v] = in ? l[v] : 0u;
                                    const u4 w = 2 * (c0 + c) + lhi < chunks ? b[q][c] : zero;
                                    y = mma(l, w, mma(h, w, y));
                                }
                            return y;
                        };
                        const bool up = !BF && (scaled[j] >> from << (from + 64 - to)) != 0;
                        // (256 rows' accumulators as operands in two branches would spill)
                        if (MI <= 2 && s < kWild && first == last && !up) {
                            if (from < 32) acc(2 * j) = products(acc(2 * j));
                            else acc(2 * j + 1) = products(acc(2 * j + 1));
                        } else {
                            f16x y;
#pragma unroll
                            for (int v = 0; v < 16; ++v) y[v] = 0.f;
                            y = products(y);
                            if (s >= kWild || first != last || up) {
                                const int lo = (from & 31) - 4 * lhi, hi = mine == part ? lo + to - from : -1;
                                const float* f = lds_up + 64 * j + (from & 32) + 4 * lhi;
#pragma unroll
                                for (int v = 0; v < 16; ++v) {
                                    const int m = 8 * (v >> 2) + (v & 3);
                                    y[v] = m >= lo && m < hi ? (BF ? y[v] : y[v] * f[m]) : 0.f;
                                }
                            }
                            // (the two ends differ, or the compiler makes one of them, of an
                            // address of either tile, and keeps the accumulators in memory)
                            if (from < 32) {
#pragma unroll
                                for (int v = 0; v < 16; ++v) acc(2 * j)[v] += y[v];
                                asm volatile("; first tile");
                            } else {
#pragma unroll
                                for (int v = 0; v < 16; ++v) acc(2 * j + 1)[v] += y[v];
                                asm volatile("; second tile");
                            }
                        }
                        load(q, j);
                        return true;
                    };
                    // (written out: as a loop it is not unrolled, and b is then in memory)
                    static_assert(PF == 2 || PF == 4, "runs by name");
#pragma clang loop unroll(disable)
                    while (run(0) && run(1) && (PF == 2 || (run(PF / 2) && run(PF - 1)))) {}
                });
            }
        }
}

}  // namespace q4dev
