// Shared parts of the few-row attention kernels: how the keys' tiles are shared
// out over the workgroups, and how a row tile's pieces are joined.
#pragma once

#include "q4_attend.h"

namespace q4attend {

constexpr int KT = 32;                 // keys of a tile
constexpr int ROWS = 16;               // rows (token, head of the group) of one

// What of a request the split goes by: its row tiles, its first key in the window,
// where the window's tiles begin (a multiple of 32), the tiles before it that hold sinks
// and the number of tiles (at least one: a tile of rows that see nothing still stores zeros).
struct Span {
    Request r;
    int rt, lo, base, ns, nt;
    // the first key of a tile: the sinks' come first, then the window's
    __device__ __forceinline__ int key_of(int tile) const { return tile < ns ? tile * KT : base + (tile - ns) * KT; }
};

template <bool SK>
__device__ __forceinline__ Span span(const Args& p, const Request& r)
{
    Span s;
    s.r = r;
    s.rt = (s.r.n * p.g + ROWS - 1) / ROWS;
    s.lo = p.window ? max(s.r.len - s.r.n - p.window + 1, 0) : 0;
    s.lo = min(s.lo, max(s.r.len - 1, 0));
    s.base = s.lo & ~(KT - 1);
    s.ns = SK ? min((p.sinks + KT - 1) / KT, s.base / KT) : 0;
    s.nt = s.ns + max((s.r.len - s.base + KT - 1) / KT, 1);
    return s;
}

// A key, or a block of 16, that no row sees is replaced by the window's first, before it is read.
template <bool SK>
__device__ __forceinline__ int seen_key(const Args& p, const Span& s, int key)
{
    return SK && key < p.sinks ? key : max(key, s.lo);
}
template <bool SK>
__device__ __forceinline__ int seen_block(const Args& p, const Span& s, int block)
{
    return SK && block * 16 < p.sinks ? block : max(block, s.lo >> 4);
}

// A workgroup's range of all tiles: `it` up to `end`, in shares of `per`; it begins
// in request b, which `before` tiles come before. A row tile counts as its tiles and `extra`
// before them, or as the next multiple of `pad`. (The first 64 requests stay in the lanes: each look at them in memory is one
// more latency before the first key.)
struct Share {
    Request first64;
    uint32_t per, it, end, before, pad, extra;
    int b;
    __device__ __forceinline__ uint32_t counted(int tiles) const
    {
        return pad == 1 ? (uint32_t)tiles + extra : ((uint32_t)tiles + pad - 1) / pad * pad;
    }
};

// (the lanes of a wave each look at a request; false: no work for this workgroup)
// EXTRA: the time that a piece of a row tile takes beside its tiles, in tiles; and where there are
// workgroups enough, every row tile gets whole shares of its own, so that no workgroup has pieces
// of two. (0: neither.)
template <bool SK, int WV, int EXTRA>
__device__ __forceinline__ bool share_of(const Args& p, int lane, Share& sh)
{
    auto request_at = [&](int b) { return b < p.B ? request(p, b) : Request{0, 0, 0}; };
    sh.pad = 1;
    sh.extra = EXTRA;
    auto cost = [&](const Request& r) {        // (0 without tokens)
        const Span s = span<SK>(p, r);
        return (uint32_t)s.rt * (uint32_t)p.KV * sh.counted(s.nt);
    };
    auto scan = [&](uint32_t v) {              // inclusive, over the lanes
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, d);
            if (lane >= d) v += o;
        }
        return v;
    };
    sh.first64 = request_at(lane);
    uint32_t cost64 = scan(cost(sh.first64));
    uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)cost64, 63);
    for (int b0 = 64; b0 < p.B; b0 += 64) total += (uint32_t)__builtin_amdgcn_readlane((int)scan(cost(request_at(b0 + lane))), 63);
    // equal shares, in whole rounds of the waves
    uint32_t per = (total + (uint32_t)p.workers - 1) / (uint32_t)p.workers;
    per = (max(per, (uint32_t)p.least) + WV - 1) / WV * WV;
    sh.per = per;
    if constexpr (EXTRA) {
        auto shares = [&](const Request& r) {
            const Span s = span<SK>(p, r);
            return (uint32_t)s.rt * (uint32_t)p.KV * (((uint32_t)s.nt + per - 1) / per);
        };
        uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)scan(shares(sh.first64)), 63);
        for (int b0 = 64; b0 < p.B; b0 += 64) n += (uint32_t)__builtin_amdgcn_readlane((int)scan(shares(request_at(b0 + lane))), 63);
        if (n <= (uint32_t)p.workers) {
            sh.pad = per;
            sh.extra = 0;
            total = n * per;
            cost64 = scan(cost(sh.first64));
        }
    }
    sh.it = (uint32_t)blockIdx.x * per;
    sh.end = min(sh.it + per, total);
    if (sh.it >= sh.end) return false;
    sh.b = 0;
    sh.before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        const uint32_t c = b0 ? scan(cost(request_at(b0 + lane))) : cost64;
        const unsigned long long past = __ballot(sh.before + c > sh.it);
        if (past) {
            const int f = (int)__builtin_ctzll(past);
            sh.b = b0 + f;
            if (f) sh.before += (uint32_t)__builtin_amdgcn_readlane((int)c, f - 1);
            break;
        }
        sh.before += (uint32_t)__builtin_amdgcn_readlane((int)c, 63);
        sh.b = b0 + 64;
    }
    return true;
}

// Request b's span, in scalar registers.
template <bool SK>
__device__ __forceinline__ Span span_of(const Args& p, const Share& sh, int b)
{
    Request r = b < 64 ? request_of_lane(sh.first64, b) : request(p, b);
    r.start = uniform(r.start);
    r.n = uniform(r.n);
    r.len = uniform(r.len);
    Span s = span<SK>(p, r);
    s.rt = uniform(s.rt);
    s.lo = uniform(s.lo);
    s.base = uniform(s.base);
    s.ns = uniform(s.ns);
    s.nt = uniform(s.nt);
    return s;
}

// A share's piece of a row tile: what comes before the row tile's first tile of all, and of
// the row tile `tiles` from `tile0`.
struct Segment {
    uint32_t pair_at;
    int tile0, tiles, head, row0, rows, pos0;
};

// Joins the waves' running maxima, sums and outputs of a segment, which lie in LDS
// (wave w's ROWS x D fp32 at out + w * out_pitch, four values u of row r at place u ^ r
// of the row; maxima and sums [w][ROWS]), and stores the rows if the segment is the whole row
// tile. Else its partial result goes to a slot of the workgroup, and the last workgroup of the
// row tile to arrive joins them in key order. Begins with a barrier; the caller has another
// before it writes to the buffers again.
template <int D, bool BF, int WV, bool SPREAD>
__device__ __forceinline__ void finish(const Args& p, const Share& sh, const Span& s, const Segment& g, char* out, int out_pitch,
                                       const float* lds_m, const float* lds_l, int* s_last)
{
    constexpr int NT = 64 * WV, UNITS = ROWS * (D / 4), UPT = UNITS < NT ? 1 : UNITS / NT;   // four values of a row each
    static_assert(UNITS % NT == 0 || UNITS < NT, "whole rounds");
    const int tid = SPREAD ? here((int)threadIdx.x) : (int)threadIdx.x;
    __syncthreads();
    const bool whole = g.tile0 == 0 && g.tiles == s.nt;
    // (workgroups there are, whatever `starts` says)
    const int wf = min((int)(g.pair_at / sh.per), p.workers - 1);
    const int wl = min((int)((g.pair_at + (uint32_t)s.nt - 1) / sh.per), p.workers - 1);
    constexpr size_t SLOT = (size_t)ROWS * (D + 2);
    auto slot_of = [&](int w) {
        return make_rsrc(p.slots + (size_t)(2 * w + (w == wf ? 1 : 0)) * SLOT, (uint32_t)(SLOT * 4));
    };
    const rsrc_t own = slot_of((int)blockIdx.x);
    const bool mine = UNITS >= NT || tid < UNITS;
    f4 o[UPT];
    float ol[UPT];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const int unit = u * NT + tid, row = UNITS < NT ? unit / (D / 4) % ROWS : unit / (D / 4), c = unit % (D / 4);
        float mm = lds_m[row];
#pragma unroll
        for (int w = 1; w < WV; ++w) mm = fmaxf(mm, lds_m[w * ROWS + row]);
        float ll = 0.f;
        f4 v = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WV; ++w) {
            const float a = exp2_fast(lds_m[w * ROWS + row] - mm);
            const f4 x = *reinterpret_cast<const f4*>(out + w * out_pitch + row * (4 * D) + ((c ^ row) << 4));
            ll += a * lds_l[w * ROWS + row];
            v += a * x;
        }
        o[u] = v;
        ol[u] = ll;
        if (!whole && row < g.rows && mine) {
            put16(own, (uint32_t)unit * 16u, v);
            if (c == 0) {
                put4(own, (uint32_t)(ROWS * D + row) * 4u, mm);
                put4(own, (uint32_t)(ROWS * D + ROWS + row) * 4u, ll);
            }
        }
    }
    bool all_here = whole;
    if (!whole) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0)
            *s_last = __hip_atomic_fetch_add(&p.counters[wf], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(wl - wf);
        __syncthreads();
        all_here = *s_last != 0;
        if (SPREAD && all_here) {
            // Unit `unit` (of `live` ones) of part `part` of the slots is lane unit + live part's, where there are
            // lanes for several parts.
            const int live = g.rows * (D / 4), parts = max(NT / live, 1), slots = wl - wf + 1;
            for (int u0 = 0; u0 < live; u0 += NT) {
                const int part = parts == 1 ? 0 : tid / live, unit = u0 + tid - part * live, row = unit / (D / 4);
                const bool on = part < parts && unit < live;
                const int w0 = wf + slots * part / parts, w1 = wf + slots * (part + 1) / parts;
                float mm = kLow, ll = 0.f;
                f4 v = f4{0.f, 0.f, 0.f, 0.f};
                // (FB slots whose loads are under way together)
                auto take = [&](int w, auto fb) {
                    constexpr int FB = decltype(fb)::value;
                    float pm[FB], pl[FB];
                    f4 po[FB];
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        const int x = min(w + f, w1 - 1);
                        const uint32_t at = (uint32_t)(2 * x + (x == wf ? 1 : 0)) * (uint32_t)(SLOT * 4);
                        const rsrc_t r = make_rsrc(p.slots, (uint32_t)(2 * p.workers * SLOT * 4));
                        pm[f] = take4(r, at + (uint32_t)(ROWS * D + row) * 4u);
                        pl[f] = take4(r, at + (uint32_t)(ROWS * D + ROWS + row) * 4u);
                        po[f] = take16(r, at + (uint32_t)unit * 16u);
                    }
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        if (w + f >= w1) continue;
                        const float mn = fmaxf(mm, pm[f]);
                        const float a = exp2_fast(mm - mn), c = exp2_fast(pm[f] - mn);
                        ll = a * ll + c * pl[f];
                        v = a * v + c * po[f];
                        mm = mn;
                    }
                };
                for (int w = w0; on && w < w1;) {
                    if (w1 - w > 4) {
                        take(w, std::integral_constant<int, 16>{});
                        w += 16;
                    } else {
                        take(w, std::integral_constant<int, 4>{});
                        w += 4;
                    }
                }
                if (parts > 1) {
                    f4* lv = reinterpret_cast<f4*>(out);
                    float *lm = reinterpret_cast<float*>(out + NT * 16), *lsum = lm + NT;
                    lv[tid] = v;
                    lm[tid] = mm;
                    lsum[tid] = ll;
                    __syncthreads();
                    for (int x = 1; part == 0 && x < parts; ++x) {
                        const int at = tid + x * live;
                        const float mn = fmaxf(mm, lm[at]);
                        const float a = exp2_fast(mm - mn), c = exp2_fast(lm[at] - mn);
                        ll = a * ll + c * lsum[at];
                        v = a * v + c * lv[at];
                        mm = mn;
                    }
                }
                const int at = unit % (D / 4) * 4;
                if (on && part == 0 && at < p.dim) {
                    const int r = g.row0 + row, token = (int)q4::fast_div((uint32_t)r, p.div_g);
                    const f4 y = output_of(v, ll, over_sum(ll, g.pos0 + token));
                    store_row4<BF>(p.out + (s.r.start + token) * p.o_t + (g.head * p.g + r - token * p.g) * p.o_h + at, y, p.dim - at, p.store8);
                }
            }
            if (tid == 0) __hip_atomic_store(&p.counters[wf], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            return;
        }
        if (all_here) {
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                const int unit = u * NT + tid, row = unit / (D / 4);
                float mm = kLow, ll = 0.f;
                f4 v = f4{0.f, 0.f, 0.f, 0.f};
                constexpr int FB = 16;     // slots whose loads are under way together
                for (int w0 = wf; row < g.rows && w0 <= wl; w0 += FB) {
                    float pm[FB], pl[FB];
                    f4 po[FB];
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        const rsrc_t r = slot_of(min(w0 + f, wl));
                        pm[f] = take4(r, (uint32_t)(ROWS * D + row) * 4u);
                        pl[f] = take4(r, (uint32_t)(ROWS * D + ROWS + row) * 4u);
                        po[f] = take16(r, (uint32_t)unit * 16u);
                    }
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        if (w0 + f > wl) continue;
                        const float mn = fmaxf(mm, pm[f]);
                        const float a = exp2_fast(mm - mn), c = exp2_fast(pm[f] - mn);
                        ll = a * ll + c * pl[f];
                        v = a * v + c * po[f];
                        mm = mn;
                    }
                }
                o[u] = v;
                ol[u] = ll;
            }
            if (tid == 0) __hip_atomic_store(&p.counters[wf], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (!all_here) return;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const int unit = u * NT + tid, row = unit / (D / 4), at = unit % (D / 4) * 4;
        if (row >= g.rows || at >= p.dim) continue;
        const int r = g.row0 + row, token = (int)q4::fast_div((uint32_t)r, p.div_g);
        const f4 y = output_of(o[u], ol[u], over_sum(ol[u], g.pos0 + token));
        store_row4<BF>(p.out + (s.r.start + token) * p.o_t + (g.head * p.g + r - token * p.g) * p.o_h + at, y, p.dim - at, p.store8);
    }
}

}  // namespace q4attend
