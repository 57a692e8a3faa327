// Attention over a paged cache for many rows a request: chunks of prompts.
//
// q4_attend_tiles_kernel<D, BF, PG>: head rows of D values in LDS, BF
// (bfloat16), PG (pages of a multiple of 16 rows).
//
// Bound: the matrix cores (4 dim flops for each visible key of a row), with the
// exponentials close behind: a 64-key tile of 32 rows is 32 products of 32 cycles
// and about 950 cycles of vector instructions (half of them the 16-cycle
// exponentials).
//
// A workgroup of NW waves takes NW x 32 rows (token, head of the group) of one
// request and cached head; a wave its 32. Tiles of KT keys and values go to two
// LDS stages by direct loads, each wave fetching 8 rows of both. Scores,
// weights, maxima, sums and outputs stay in registers (q4_attend.h).
//
// With eight waves each SIMD holds two, and the waves work in two groups a
// phase apart, so that one of the two multiplies (O += V^T P^T of tile j, then
// S^T = K Q^T of tile j + 1) while the other computes its weights; a barrier
// ends each phase. A head of 256 values takes four waves of 32-key tiles
// instead, whose outputs and queries fill the registers of two.
//
// The rescale of the outputs when a maximum grows is put off until it has grown by
// 2^8: a weight is then at most 256, far inside both types.
//
// Units of work are (request, row tile, cached head, split of the keys), the
// heads fastest, so that a head's row tiles run on one XCD (workgroup i on XCD i
// % 8) and share its L2. Requests' splits go by the whole call's work: with
// `target` workgroups wanted, no unit has more than 1 / target of all tiles (at
// least kLeast of them); where row tiles alone fill the chip there are none. A row tile's
// splits leave partial results, joined by the last to arrive, in key order.
#include "q4_attend.h"

namespace {

using namespace q4attend;

template <int D>
struct Shape {
    static constexpr int NW = D == 256 ? 4 : 8;      // waves
    static constexpr int KT = 8 * NW;                // keys of a tile
    static constexpr int BR = 32 * NW;               // rows of a workgroup
};

constexpr float kSlack = 8.f;    // log2 of the growth of a maximum that is let pass

template <int D>
struct Span {
    Request r;
    int rt, nt;                  // row tiles; most key tiles of one
};

template <int D>
__device__ __forceinline__ Span<D> span(const Args& p, int b)
{
    using S = Shape<D>;
    Span<D> s;
    s.r = request(p, b);
    s.rt = (s.r.n * p.g + S::BR - 1) / S::BR;
    const int lo = p.window ? min(max(s.r.len - s.r.n - p.window + 1, 0), max(s.r.len - 1, 0)) : 0;
    s.nt = max((s.r.len - (lo & ~(S::KT - 1)) + S::KT - 1) / S::KT, 1);
    return s;
}

template <int D, bool BF, bool PG>
__global__ __launch_bounds__(64 * Shape<D>::NW, D == 256 ? 1 : 2) void q4_attend_tiles_kernel(Args p)
{
    using SH = Shape<D>;
    constexpr int NW = SH::NW, KT = SH::KT, BR = SH::BR, NT = 64 * NW;
    constexpr int HH = KT / 32;                // 32-key halves of a tile
    constexpr int PITCH = 2 * D, CPR = D / 8, RPI = 64 / CPR;
    constexpr int NI = 8 / RPI;                // direct loads of a wave's 8 rows
    constexpr int KS = D / 16, DT = D / 32;    // k-steps of the scores, 32-value tiles of the output
    __shared__ __attribute__((aligned(1024))) char lds_k[2][KT * PITCH];
    __shared__ __attribute__((aligned(1024))) char lds_v[2][KT * PITCH];
    __shared__ int s_last;

    const int tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int lane = tid & 63, l32 = lane & 31, lhi = lane >> 5;

    // ---- the unit
    auto scan = [&](uint32_t v) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, d);
            if (lane >= d) v += o;
        }
        return v;
    };
    auto last_of = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); };
    uint32_t total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        uint32_t c = 0;
        if (b0 + lane < p.B) {
            const Span<D> s = span<D>(p, b0 + lane);
            c = (uint32_t)s.rt * (uint32_t)s.nt * (uint32_t)p.KV;
        }
        total += last_of(scan(c));
    }
    const int chunk = (int)max((total + (uint32_t)p.workers - 1) / (uint32_t)p.workers, (uint32_t)p.least);
    const uint32_t me = blockIdx.x;
    uint32_t before = 0, slots_before = 0;
    int b = -1;
    for (int b0 = 0; b0 < p.B && b < 0; b0 += 64) {
        uint32_t u = 0, sl = 0;
        if (b0 + lane < p.B) {
            const Span<D> s = span<D>(p, b0 + lane);
            const int splits = (s.nt + chunk - 1) / chunk;
            u = (uint32_t)s.rt * (uint32_t)splits * (uint32_t)p.KV;
            sl = splits > 1 ? u : 0;
        }
        const uint32_t uc = scan(u), sc = scan(sl);
        const unsigned long long past = __ballot(before + uc > me);
        if (past) {
            const int f = (int)__builtin_ctzll(past);
            b = b0 + f;
            before += (uint32_t)__builtin_amdgcn_readlane((int)(uc - u), f);
            slots_before += (uint32_t)__builtin_amdgcn_readlane((int)(sc - sl), f);
        } else {
            before += last_of(uc);
            slots_before += last_of(sc);
        }
    }
    if (b < 0) return;
    const Span<D> sp = span<D>(p, b);
    const int start = uniform(sp.r.start), n = uniform(sp.r.n), len = uniform(sp.r.len), rt = uniform(sp.rt);
    const int splits = (uniform(sp.nt) + chunk - 1) / chunk;
    const uint32_t unit = me - before;
    const int head = (int)(unit % (uint32_t)p.KV);
    const uint32_t rest = unit / (uint32_t)p.KV;
    const int split = (int)(rest % (uint32_t)splits);
    const int row_tile = rt - 1 - (int)(rest / (uint32_t)splits);    // the most keys first
    const int row0 = row_tile * BR, rows = min(BR, n * p.g - row0);
    const int pos0 = len - n;
    // the row tile's visible keys, its tiles, and this split's
    const int tok0 = (int)q4::fast_div((uint32_t)row0, p.div_g), tok1 = (int)q4::fast_div((uint32_t)(row0 + rows - 1), p.div_g);
    const int hi = max(min(len, pos0 + tok1 + 1), 0);
    const int lo = p.window ? min(max(pos0 + tok0 - p.window + 1, 0), max(hi - 1, 0)) : 0;
    const int base = lo & ~(KT - 1);
    const int nt = max((hi - base + KT - 1) / KT, 1);
    const int parts = (nt + chunk - 1) / chunk;
    if (split >= parts) return;
    const int j0 = (int)((long long)nt * split / parts), j1 = (int)((long long)nt * (split + 1) / parts);

    // ---- loads: rows 8 wave .. 8 wave + 7 of each tile
    const int last_key = max(hi - 1, 0);
    const char* kh = reinterpret_cast<const char*>(p.k + head * p.ks1);
    const char* vh = reinterpret_cast<const char*>(p.v + head * p.vs1);
    const int sub = lane / CPR;                // row of a direct load
    uint32_t koff[NI], voff[NI];
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int row = 8 * wave + e * RPI + sub;
        const uint32_t c = (uint32_t)min((lane % CPR) ^ spread<D>(row), p.chunks - 1) * 16u;
        koff[e] = (uint32_t)((row & 15) * p.ks2) + c;
        voff[e] = (uint32_t)((row & 15) * p.vs2) + c;
    }
    const uint32_t at_k = lds_address(lds_k[0]) + (uint32_t)(8 * wave) * PITCH;
    const uint32_t at_v = lds_address(lds_v[0]) + (uint32_t)(8 * wave) * PITCH;
    long long ko = 0, vo = 0;
    auto locate = [&](int key) {
        const int slot = (int)q4::fast_div((uint32_t)key, p.div_page);
        const uint32_t page = min((uint32_t)p.table[(long long)b * p.table_stride + slot], (uint32_t)p.pages - 1u);
        const int row = key - slot * p.page_size;
        ko = page * p.ks0 * 2 + (long long)row * p.ks2;
        vo = page * p.vs0 * 2 + (long long)row * p.vs2;
    };
    // (lane l: the wave's 16-row block of tile j + l)
    auto batch = [&](int j) {
        if constexpr (PG) locate(min(max((base + (j + lane) * KT) / 16 + (wave >> 1), lo >> 4), last_key >> 4) * 16);
    };
    auto load = [&](int j, auto values_tag) {
        constexpr bool values = decltype(values_tag)::value;
        const int first = base + j * KT + 8 * wave;          // key of the wave's first row
        const uint32_t dst = (values ? at_v : at_k) + (uint32_t)(j & 1) * (KT * PITCH);
        const char* src = values ? vh : kh;
        if constexpr (PG) {
            const long long off = values ? vo : ko;
            const int from = (j - j0) & 63;
            const uint32_t o0 = (uint32_t)__builtin_amdgcn_readlane((int)off, from);
            const uint32_t o1 = (uint32_t)__builtin_amdgcn_readlane((int)(off >> 32), from);
            const char* base_at = src + (long long)((uint64_t)o1 << 32 | o0);
            uint32_t at[NI];
#pragma unroll
            for (int e = 0; e < NI; ++e) at[e] = values ? voff[e] : koff[e];
            // rows past the last key repeat it (nothing unwritten is read)
            const int limit = last_key - 16 * min(max(first >> 4, lo >> 4), last_key >> 4);
            if (limit < 15) {
#pragma unroll
                for (int e = 0; e < NI; ++e) {
                    const int row = (8 * wave + e * RPI + sub) & 15;
                    at[e] -= (uint32_t)((row - min(row, limit)) * (values ? p.vs2 : p.ks2));
                }
            }
            dma<NI>(base_at, at, dst);
        } else {
#pragma unroll
            for (int e = 0; e < NI; ++e) {
                const int row = 8 * wave + e * RPI + sub;
                const int c = min((lane % CPR) ^ spread<D>(row), p.chunks - 1);
                locate(min(max(first + e * RPI + sub, lo), last_key));
                dma_lane(src + (values ? vo : ko) + c * 16, dst + e * 1024u);
            }
        }
    };
    constexpr std::false_type KEYS;
    constexpr std::true_type VALUES;
    batch(j0);
    load(j0, KEYS);
    load(j0, VALUES);
    if (j0 + 1 < j1) load(j0 + 1, KEYS);

    // ---- queries: lane holds row l32, values 16 ks + 8 lhi ..
    u4 qf[KS];
    const int wrow = 32 * wave + l32;
    const bool live = wrow < rows;
    const int token = (int)q4::fast_div((uint32_t)(row0 + (live ? wrow : 0)), p.div_g);
    const int qh = head * p.g + row0 + (live ? wrow : 0) - token * p.g;
    const int pos = pos0 + token;
    {
        const uint16_t* qp = p.q + (start + token) * p.q_t + qh * p.q_h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int at = 16 * ks + 8 * lhi;
            qf[ks] = at < p.dim ? *reinterpret_cast<const u4*>(qp + at) : u4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[ks][e] = (qf[ks][e] & p.q_and) ^ p.q_xor;
        }
    }
    const int klo = p.window ? pos - p.window + 1 : 0;
    // keys that all of the wave's rows see
    const int w0 = min(32 * wave, rows - 1), w1 = min(32 * wave + 31, rows - 1);
    const int all_hi = pos0 + (int)q4::fast_div((uint32_t)(row0 + w0), p.div_g);
    const int all_lo = p.window ? pos0 + (int)q4::fast_div((uint32_t)(row0 + w1), p.div_g) - p.window + 1 : 0;

    f16x acc[DT], sc[HH];
    u4 pt[2 * HH];
    float m = kLow, l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;

    const int kx = l32 * PITCH + ((lhi ^ spread<D>(l32)) << 4);
    const int j16 = lane & 15, dh = (lane >> 4) & 1;
    int vx[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + 4 * lhi + (j16 >> 2);
        vx[q] = row * PITCH + (((2 * dh + ((j16 >> 1) & 1)) ^ spread<D>(row)) << 4) + (j16 & 1) * 8;
    }

    auto scores = [&](int j) {
        const char* kb = lds_k[j & 1];
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[h][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < HH; ++h) {
                const u4 a = *reinterpret_cast<const u4*>(kb + h * 32 * PITCH + (kx ^ (ks << 5)));
                if constexpr (BF) sc[h] = mfma32(bitcast<b8>(a), bitcast<b8>(qf[ks]), sc[h]);
                else sc[h] = mfma32(bitcast<h8>(a), bitcast<h8>(qf[ks]), sc[h]);
            }
    };
    auto weights = [&](int j) {
        const int first = base + j * KT;
        if (first + KT - 1 > all_hi || first < all_lo) {
#pragma unroll
            for (int h = 0; h < HH; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int key = first + 32 * h + 8 * (e >> 2) + 4 * lhi + (e & 3);
                    sc[h][e] = key >= klo && key <= pos ? sc[h][e] : -INFINITY;
                }
        }
        float top = sc[0][0];
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[h][e]);
        const float mn = fmaxf(m, max_halves(top) * p.scale);
        if (__any(mn > m + kSlack)) {
            const float a = exp2_fast(m - mn);
            l *= a;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[d][e] *= a;
            m = mn;
        }
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                sc[h][e] = exp2_fast(__builtin_fmaf(sc[h][e], p.scale, -m));
                l += sc[h][e];
            }
#pragma unroll
        for (int s = 0; s < 2 * HH; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 8 * (s & 1) + 2 * e;
                pt[s][e] = pack2<BF>(sc[s >> 1][at], sc[s >> 1][at + 1]);
            }
    };
    auto output = [&](int j) {
        const char* vb = lds_v[j & 1];
#pragma unroll
        for (int s = 0; s < 2 * HH; ++s)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u2 a0 = read_tr(vb + s * 16 * PITCH + (vx[0] ^ (d << 6)));
                const u2 a1 = read_tr(vb + s * 16 * PITCH + (vx[1] ^ (d << 6)));
                const u4 a = u4{a0[0], a0[1], a1[0], a1[1]};
                if constexpr (BF) acc[d] = mfma32(bitcast<b8>(a), bitcast<b8>(pt[s]), acc[d]);
                else acc[d] = mfma32(bitcast<h8>(a), bitcast<h8>(pt[s]), acc[d]);
            }
    };
    auto barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Phases. Group 0 forms scores in phase 0, weights of tile j in phase 2 (j -
    // j0) + 1, its output and the next scores in the one after; group 1 a phase
    // later. Loads of tile j + 2's keys and tile j + 1's values start in phase 2
    // (j - j0) + 2, where their stages are free (both groups have read tile j's
    // keys and tile j - 1's values), and have landed two phases later.
    const bool late = NW == 8 && wave >= 4;
    auto fetch = [&](int j) {
        if (j + 1 < j1) load(j + 1, VALUES);
        if (j + 2 >= j1) return;
        if (((j + 2 - j0) & 63) == 0) batch(j + 2);     // (its keys are the batch's first use)
        load(j + 2, KEYS);
    };
    wait_loads<0>();
    barrier();
    if (late) barrier();
    scores(j0);
    barrier();
    for (int j = j0; j < j1; ++j) {
        if (late) fetch(j);
        weights(j);
        if (!late) wait_loads<0>();
        barrier();
        if (!late) fetch(j);
        output(j);
        if (j + 1 < j1) scores(j + 1);
        if (late) wait_loads<0>();
        barrier();
    }
    if (NW == 8 && !late) barrier();

    // ---- store, or leave a partial result
    const float ls = sum_halves(l);
    if (parts == 1) {
        if (live) {
            const float inv = ls == 0.f ? 0.f : 1.f / ls;       // (a row that sees no key: zeros)
            uint16_t* o = p.out + (start + token) * p.o_t + qh * p.o_h;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 32 * d + 8 * e + 4 * lhi;
                    if (at >= p.dim) continue;
                    f4 y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = ls == 0.f ? 0.f : acc[d][4 * e + i] * inv;
                    store_row4<BF>(o + at, y, p.dim - at, p.store8);
                }
        }
        return;
    }
    constexpr size_t SLOT = (size_t)BR * (D + 2);
    // (never more slots than the workspace has, whatever `starts` says)
    const uint32_t slot0 = slots_before + ((uint32_t)row_tile * (uint32_t)p.KV + (uint32_t)head) * (uint32_t)splits;
    if (slot0 + (uint32_t)splits > 2u * (uint32_t)p.workers) return;
    auto slot_of = [&](int s) { return make_rsrc(p.slots + (size_t)(slot0 + (uint32_t)s) * SLOT, (uint32_t)(SLOT * 4)); };
    if (live) {
        const rsrc_t own = slot_of(split);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                put16(own, (uint32_t)(wrow * D + 32 * d + 8 * e + 4 * lhi) * 4u,
                      f4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]});
        if (lhi == 0) {
            put4(own, (uint32_t)(BR * D + wrow) * 4u, m);
            put4(own, (uint32_t)(BR * D + BR + wrow) * 4u, ls);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
        s_last = __hip_atomic_fetch_add(&p.counters[slot0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(parts - 1);
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) __hip_atomic_store(&p.counters[slot0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int u = tid; u < rows * (D / 4); u += NT) {
        const int row = u / (D / 4), at = u % (D / 4) * 4;
        float mm = kLow, ll = 0.f;
        f4 v = f4{0.f, 0.f, 0.f, 0.f};
        constexpr int FB = 4;
        for (int s0 = 0; s0 < parts; s0 += FB) {
            float pm[FB], pl[FB];
            f4 po[FB];
#pragma unroll
            for (int f = 0; f < FB; ++f) {
                const rsrc_t r = slot_of(min(s0 + f, parts - 1));
                pm[f] = take4(r, (uint32_t)(BR * D + row) * 4u);
                pl[f] = take4(r, (uint32_t)(BR * D + BR + row) * 4u);
                po[f] = take16(r, (uint32_t)u * 16u);
            }
#pragma unroll
            for (int f = 0; f < FB; ++f) {
                if (s0 + f >= parts) continue;
                const float mx = fmaxf(mm, pm[f]);
                const float a = exp2_fast(mm - mx), c = exp2_fast(pm[f] - mx);
                ll = a * ll + c * pl[f];
                v = a * v + c * po[f];
                mm = mx;
            }
        }
        if (at >= p.dim) continue;
        const int r = row0 + row, tk = (int)q4::fast_div((uint32_t)r, p.div_g);
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const f4 y = ll == 0.f ? f4{0.f, 0.f, 0.f, 0.f} : v * inv;
        store_row4<BF>(p.out + (start + tk) * p.o_t + (head * p.g + r - tk * p.g) * p.o_h + at, y, p.dim - at, p.store8);
    }
}

template <int D>
hipError_t launch_tiles(const Args& p, int grid, bool bf16, bool pg, hipStream_t stream)
{
    const dim3 g(grid), block(64 * Shape<D>::NW);
    if (bf16 && pg) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, true, true>), g, block, 0, stream, p);
    else if (bf16) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, true, false>), g, block, 0, stream, p);
    else if (pg) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, false, true>), g, block, 0, stream, p);
    else hipLaunchKernelGGL((q4_attend_tiles_kernel<D, false, false>), g, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

namespace q4 {

hipError_t launch_attend_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream)
{
    if (p.dim < 8 || p.dim > 256 || p.dim % 8 || grid < 1 || p.workers < 1) return hipErrorInvalidValue;
    if (p.dim <= 64) return launch_tiles<64>(p, grid, bf16, pages_of_16, stream);
    if (p.dim <= 128) return launch_tiles<128>(p, grid, bf16, pages_of_16, stream);
    return launch_tiles<256>(p, grid, bf16, pages_of_16, stream);
}

}  // namespace q4
