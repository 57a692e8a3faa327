// Attention over a paged cache for many rows a request: chunks of prompts.
//
// q4_attend_tiles_kernel<D, BF, PG, SK, C4, H16>: head rows of D values in LDS, BF
// (bfloat16), PG (pages of a multiple of 16 rows), SK (sinks: first keys that stay
// visible beside a window), C4 (a cache held in 4 bits, q4_cache4.h), H16 (keys and values
// of binary16 whatever the queries are).
//
// Bound: the matrix cores (4 dim flops for each visible key of a row), with the
// exponentials close behind: a 64-key tile of 32 rows is 32 products of 32 cycles
// and about 950 cycles of vector instructions (half of them the 16-cycle
// exponentials). 4096 new tokens over 8192 keys, 32 heads of 128, bfloat16: 381 us, 1080
// TFLOP/s (a large product of the library reaches 1240).
//
// A workgroup of NW waves takes NW x 32 rows (token, head of the group) of one
// request and cached head; a wave its 32. Tiles of KT keys and values go to two
// LDS stages by direct loads, each wave fetching 8 rows of both. Scores,
// weights, maxima, sums and outputs stay in registers (q4_attend.h).
//
// Each step of a wave multiplies for two tiles while it computes the weights of
// the tile between them (below); one barrier a step. A head of 256 values takes
// four waves of 32-key tiles, whose outputs and queries fill the registers of two: one
// workgroup a CU, a wave a SIMD, with no second one to issue beside it (2048 new tokens over
// 4096 keys, bfloat16: 16 heads of 256 221 us, 470 TFLOP/s; 32 of 128 115 us, 900).
//
// The rescale of the outputs when a maximum grows is put off until it has grown by
// 2^8: a weight is then at most 2^15 in binary16, 2^8 in bfloat16 (lift in q4_attend.h).
//
// Units of work are (request, row tile, cached head, split of the keys), the
// heads fastest, so that a head's row tiles run on one XCD (workgroup i on XCD i
// % 8) and share its L2. Requests' splits go by the whole call's work: with
// `target` workgroups wanted, no unit has more than 1 / target of all tiles (at
// least `least` of them); where row tiles alone fill the chip there are none. A row
// tile's splits leave partial results and its first one an entry in a list, which
// a second launch goes through.
//
// Over 4 bits the tiles in LDS are of binary16: each wave makes its KT / NW rows of them out of the
// codes, one packed multiply-add for two values, so the products
// are those of a binary16 cache whatever the queries' type (bfloat16 queries brought into binary16's
// range by a power of two a row). Codes and scales are asked for at a step's start (by direct loads into LDS
// for heads of 128, into registers for the others), waited for at its end, all of them, and unpacked there into
// the stage that they are for: only the step's own products stand between a load and its use. The unpacking is some 126 vector instructions a wave and 64-key tile beside
// the 950: 2048 new tokens over 8192 keys, 32 heads of 128 over 8, 290 us, 830 TFLOP/s, of
// which 5 join; over tiles that were unpacked once before (q4_attend4_halves.hip) 265 with the unpacking.
#pragma once

#include "q4_attend.h"
#include "q4_cache4.h"

namespace {

using namespace q4attend;

constexpr int NW = 4;            // waves of a workgroup
constexpr int BR = 32 * NW;      // its rows

template <int D>
struct Shape {
    static constexpr int KT = D == 256 ? 32 : 64;    // keys of a tile
    static constexpr int NS = D == 128 ? 2 : 4;      // LDS stages
    static constexpr int WR = KT / NW;               // rows of a tile that a wave loads
    static_assert(WR <= 16, "in one block of 16 rows");
};

constexpr float kSlack = 8.f;    // log2 of the growth of a maximum that is let pass

struct Span {
    Request r;
    int rt, nt;                  // row tiles; most key tiles of one
};

// Tiles that hold sinks, of those before the window's first.
template <int KT, bool SK>
__device__ __forceinline__ int sink_tiles(const Args& p, int base)
{
    return SK ? min((p.sinks + KT - 1) / KT, base / KT) : 0;
}

template <class S, bool SK>
__device__ __forceinline__ Span span(const Args& p, const Request& r)
{
    Span s;
    s.r = r;
    s.rt = (s.r.n * p.g + BR - 1) / BR;
    const int lo = p.window ? min(max(s.r.len - s.r.n - p.window + 1, 0), max(s.r.len - 1, 0)) : 0;
    s.nt = max((s.r.len - (lo & ~(S::KT - 1)) + S::KT - 1) / S::KT, 1);
    // (a later row tile's window leaves more of the sinks before it)
    if constexpr (SK) s.nt = min(s.nt + (p.sinks + S::KT - 1) / S::KT, max((s.r.len + S::KT - 1) / S::KT, 1));
    return s;
}

template <int D, bool BF, bool PG, bool SK, bool C4, bool H16>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void q4_attend_tiles_kernel(Args p)
{
    using SH = Shape<D>;
    constexpr bool BI = BF && !H16;            // the products' operands are bfloat16
    constexpr int KT = SH::KT, NS = SH::NS, WR = SH::WR;
    constexpr int HH = KT / 32;                // 32-key halves of a tile
    constexpr int PITCH = 2 * D, CPR = D / 8, RPI = 64 / CPR;
    constexpr int NI = WR / RPI;               // direct loads of a wave's rows
    constexpr int KS = D / 16, DT = D / 32;    // k-steps of the scores, 32-value tiles of the output
    __shared__ __attribute__((aligned(1024))) char lds_k[NS][KT * PITCH];
    __shared__ __attribute__((aligned(1024))) char lds_v[NS][KT * PITCH];
    // 4 bits, heads of 128: codes and scales on their way, a wave's 16 rows of keys and of values.
    // (In registers, ten of them for the time of a step, they left the compiler none to read the
    // products' operands ahead with, and every product waited for its own.)
    constexpr bool RAW = C4 && D == 128;
    constexpr int RAW_PIECES = 1024 + 256;
    __shared__ __attribute__((aligned(1024))) char lds_raw[RAW ? NW : 1][RAW ? 2 * RAW_PIECES : 16];

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
    // (the first 64 requests stay in the lanes: each look at them in memory is one
    // more latency before the first key)
    auto request_at = [&](int b) { return b < p.B ? request(p, b) : Request{0, 0, 0}; };
    auto cost = [&](const Request& r) {        // (0 without tokens)
        const Span s = span<SH, SK>(p, r);
        return (uint32_t)s.rt * (uint32_t)s.nt * (uint32_t)p.KV;
    };
    const Request first64 = request_at(lane);
    uint32_t total = last_of(scan(cost(first64)));
    for (int b0 = 64; b0 < p.B; b0 += 64) total += last_of(scan(cost(request_at(b0 + lane))));
    const int chunk = (int)max((total + (uint32_t)p.workers - 1) / (uint32_t)p.workers, (uint32_t)p.least);
    const uint32_t me = blockIdx.x;
    uint32_t before = 0, slots_before = 0;
    int b = -1;
    for (int b0 = 0; b0 < p.B && b < 0; b0 += 64) {
        uint32_t u = 0, sl = 0;
        if (b0 + lane < p.B) {
            const Span s = span<SH, SK>(p, b0 ? request(p, b0 + lane) : first64);
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
    const Span sp = span<SH, SK>(p, b < 64 ? request_of_lane(first64, b) : request(p, b));
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
    const int ns = sink_tiles<KT, SK>(p, base);
    const int nt = ns + max((hi - base + KT - 1) / KT, 1);
    const int parts = (nt + chunk - 1) / chunk;
    if (split >= parts) return;
    const int j0 = (int)((long long)nt * split / parts), j1 = (int)((long long)nt * (split + 1) / parts);

    // a tile's first key: the sinks' tiles come first, then the window's
    auto key_of = [&](int j) { return SK && j < ns ? j * KT : base + (j - ns) * KT; };
    // (a block of 16 keys that no row sees is replaced by the window's first before it is read)
    auto seen_block = [&](int block) { return SK && block * 16 < p.sinks ? block : max(block, lo >> 4); };

    // ---- loads: rows WR wave .. WR wave + WR - 1 of each tile (in one 16-row block)
    const int last_key = max(hi - 1, 0);
    const char* kh = reinterpret_cast<const char*>(p.k + head * p.ks1);
    const char* vh = reinterpret_cast<const char*>(p.v + head * p.vs1);
    const int sub = lane / CPR;                // row of a direct load
    uint32_t koff[NI], voff[NI];
    if constexpr (!C4)
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int row = WR * wave + e * RPI + sub;
        const uint32_t c = (uint32_t)min((lane % CPR) ^ spread<D>(row), p.chunks - 1) * 16u;
        koff[e] = (uint32_t)((row & 15) * p.ks2) + c;
        voff[e] = (uint32_t)((row & 15) * p.vs2) + c;
    }
    const uint32_t at_k = lds_address(lds_k[0]) + (uint32_t)(WR * wave) * PITCH;
    const uint32_t at_v = lds_address(lds_v[0]) + (uint32_t)(WR * wave) * PITCH;
    // bytes of a row of the cache from kh or vh, by its key
    auto locate = [&](int key, long long page_stride, int row_stride) {
        const int slot = (int)q4::fast_div((uint32_t)key, p.div_page);
        const uint32_t page = min((uint32_t)p.table[(long long)b * p.table_stride + slot], (uint32_t)p.pages - 1u);
        return page * page_stride * 2 + (long long)(key - slot * p.page_size) * row_stride;
    };
    // 4 bits: a lane has PD neighbouring values of one of the wave's rows. They go through
    // registers; a row's keys lie in LDS in
    // the order of the unpacked codes (the queries' values too), its values in their own.
    constexpr int PR = 64 / WR, PD = D / PR;   // pieces of a row, values of one
    struct Piece {
        uint32_t code[PD / 8], scale;
    };
    // (in an order in which the pieces that 8 lanes write together, and 16, fall on banks of their own:
    // row by row 4 of them met, which took a quarter of the kernel's time; of heads of 256 two still do)
    const int pq = D == 128 ? (lane >> 1 & 3) | lane >> 4 << 2 : lane / PR;
    const int prow = WR * wave + (D == 64 ? (pq & 1) << 2 | (pq & 6) >> 1 | (pq & 8) : D == 128 ? (pq & 3) << 2 | pq >> 2 : (pq & 1) << 2 | pq >> 1);
    const int pdim = (D == 128 ? (lane & 1) | (lane >> 3 & 1) << 1 : lane % PR) * PD;
    const bool pin = pdim < p.dim;
    const uint32_t pcol = pin ? (uint32_t)pdim / 2u : 0u, pscol = pin ? (uint32_t)(pdim >> p.group_shift) * 4u : 0u;
    const uint32_t raw = RAW ? lds_address(lds_raw[wave]) : 0u;
    uint32_t pkoff = 0, pksoff = 0, pvoff = 0, pvsoff = 0;     // the lane's bytes in the 16 rows
    if constexpr (C4) {
        pkoff = (uint32_t)((prow & 15) * p.k4.row) + pcol;
        pksoff = (uint32_t)((prow & 15) * p.k4.scale_row) + pscol;
        pvoff = (uint32_t)((prow & 15) * p.v4.row) + pcol;
        pvsoff = (uint32_t)((prow & 15) * p.v4.scale_row) + pscol;
    }
    auto locate4 = [&](int key, int& row) {
        const int slot = (int)q4::fast_div((uint32_t)key, p.div_page);
        row = key - slot * p.page_size;
        return (int)min((uint32_t)p.table[(long long)b * p.table_stride + slot], (uint32_t)p.pages - 1u);
    };
    // (lane l: of the wave's 16-row block of tile j + l, for 64 tiles at a time)
    long long ko = 0, vo = 0;
    auto block_of = [&](int j) { return min(seen_block(key_of(j + lane) / 16 + WR * wave / 16), last_key >> 4) * 16; };
    auto batch = [&](int j, auto values_tag) {
        if constexpr (PG && !C4) {
            if constexpr (decltype(values_tag)::value) vo = locate(block_of(j), p.vs0, p.vs2);
            else ko = locate(block_of(j), p.ks0, p.ks2);
        }
    };
    auto load = [&](int j, auto values_tag, int stage) {
        constexpr bool values = decltype(values_tag)::value;
        const int first = key_of(j) + WR * wave;         // key of the wave's first row
        const uint32_t dst = (values ? at_v : at_k) + (uint32_t)stage * (KT * PITCH);
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
            const int limit = last_key - 16 * min(seen_block(first >> 4), last_key >> 4);
            if (limit < 15) {
#pragma unroll
                for (int e = 0; e < NI; ++e) {
                    const int row = (WR * wave + e * RPI + sub) & 15;
                    at[e] -= (uint32_t)((row - min(row, limit)) * (values ? p.vs2 : p.ks2));
                }
            }
            dma<NI>(base_at, at, dst);
        } else {
#pragma unroll
            for (int e = 0; e < NI; ++e) {
                const int row = WR * wave + e * RPI + sub;
                const int c = min((lane % CPR) ^ spread<D>(row), p.chunks - 1);
                const int at = first + e * RPI + sub;
                const int key = min(SK && at < p.sinks ? at : max(at, lo), last_key);
                dma_lane(src + (values ? locate(key, p.vs0, p.vs2) : locate(key, p.ks0, p.ks2)) + c * 16, dst + e * 1024u);
            }
        }
    };
    // Pages of 16 rows: the lane's block (block_of), in units of the codes' 16 bytes and the scales' 4
    // (the host sees to it that they fit in 32 bits).
    uint32_t kblock = 0, ksblock = 0, vblock = 0, vsblock = 0;
    auto batch4 = [&](int j, auto values_tag) {
        if constexpr (PG && C4) {
            const Args& a = args_again();
            const Side& side = decltype(values_tag)::value ? a.v4 : a.k4;
            int row;
            const uint64_t page = (uint64_t)locate4(block_of(j), row);
            const uint32_t at = (uint32_t)((page * (uint64_t)side.page + (uint64_t)row * (uint64_t)side.row) >> 4);
            const uint32_t scale_at = (uint32_t)((page * (uint64_t)side.scale_page + (uint64_t)row * (uint64_t)side.scale_row) >> 2);
            if constexpr (decltype(values_tag)::value) {
                vblock = at;
                vsblock = scale_at;
            } else {
                kblock = at;
                ksblock = scale_at;
            }
        }
    };
    const char *kh4 = p.k4.at + head * p.k4.head, *ksh4 = p.k4.scale + head * p.k4.scale_head;
    const char *vh4 = p.v4.at + head * p.v4.head, *vsh4 = p.v4.scale + head * p.v4.scale_head;
    auto fetch = [&](int j, auto values_tag, Piece& x) {
        constexpr bool values = decltype(values_tag)::value;
        const int first = key_of(j) + WR * wave;
        const char *at = values ? vh4 : kh4, *scale_at = values ? vsh4 : ksh4;
        uint64_t ro, so;
        if constexpr (PG) {
            const int from = (j - j0) & 63;
            at += (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(values ? vblock : kblock), from) << 4;
            scale_at += (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(values ? vsblock : ksblock), from) << 2;
            uint32_t r = values ? pvoff : pkoff, q = values ? pvsoff : pksoff;
            // rows past the last key repeat it (nothing unwritten is read)
            const int limit = last_key - 16 * min(seen_block(first >> 4), last_key >> 4);
            if (limit < 15) {
                const Side& side = values ? args_again().v4 : args_again().k4;
                const int back = (prow & 15) - min(prow & 15, limit);
                r -= (uint32_t)(back * side.row);
                q -= (uint32_t)(back * side.scale_row);
            }
            ro = r;
            so = q;
        } else {
            const Side& side = values ? args_again().v4 : args_again().k4;
            const int key = first + prow - WR * wave;
            int row;
            const uint64_t page = (uint64_t)locate4(min(key < p.sinks ? key : max(key, lo), last_key), row);
            ro = page * (uint64_t)side.page + (uint64_t)row * (uint64_t)side.row + pcol;
            so = page * (uint64_t)side.scale_page + (uint64_t)row * (uint64_t)side.scale_row + pscol;
        }
        if constexpr (RAW) {
            const uint32_t to = raw + (values ? RAW_PIECES : 0);
            if constexpr (PG) {
                const uint32_t off[1] = {(uint32_t)ro};
                dma<1>(at, off, to);
                dma_words(scale_at, (uint32_t)so, to + 1024u);
            } else {
                dma_lane(at + ro, to);
                dma_words_lane(scale_at + so, to + 1024u);
            }
        } else if constexpr (PD == 16) {
            const u2 w = *reinterpret_cast<const u2*>(at + ro);
            x.code[0] = w[0];
            x.code[1] = w[1];
        } else {
            const u4 w = *reinterpret_cast<const u4*>(at + ro);
#pragma unroll
            for (int e = 0; e < 4; ++e) x.code[e] = w[e];
        }
        if constexpr (!RAW) x.scale = *reinterpret_cast<const uint32_t*>(scale_at + so);
    };
    // (piece e of the lane's, from a multiple of their number, is at place (pdim / 8 ^ spread) ^ e of the row)
    const int pplace = prow * PITCH + (((pdim / 8) ^ spread<D>(prow)) << 4);
    auto put = [&](Piece x, auto values_tag, int stage) {
        constexpr bool values = decltype(values_tag)::value;
        if constexpr (RAW) {
            const char* from = lds_raw[wave] + (values ? RAW_PIECES : 0);
            const u4 w = *reinterpret_cast<const u4*>(from + lane * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) x.code[e] = w[e];
            x.scale = *reinterpret_cast<const uint32_t*>(from + 1024 + lane * 4);
        }
        const int place = here(pplace);
        const q4cache4::Magic magic = q4cache4::magic();
        const uint32_t sm = pin ? x.scale : 0u;
        const h2 step = q4cache4::low_half(sm), least = q4cache4::high_half(sm);
#pragma unroll
        for (int e = 0; e < PD / 8; ++e) {
            const u4 w = q4cache4::values8(x.code[e], step, least, magic);
            *reinterpret_cast<u4*>((values ? lds_v[0] : lds_k[0]) + (place ^ (e << 4)) + stage * (KT * PITCH)) =
                values ? q4cache4::own_order(w) : w;
        }
    };
    constexpr std::false_type KEYS;
    constexpr std::true_type VALUES;
    Piece pk = {}, pv = {};
    if constexpr (C4) {
        batch4(j0, KEYS);
        batch4(j0, VALUES);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            fetch(min(j0 + i, j1 - 1), KEYS, pk);
            if (i < NS - 2) fetch(min(j0 + i, j1 - 1), VALUES, pv);
            if constexpr (RAW) wait_loads<0>();
            put(pk, KEYS, i);
            if (i < NS - 2) put(pv, VALUES, i);
            wait_lds();
        }
    } else {
    batch(j0, KEYS);
    batch(j0, VALUES);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        load(min(j0 + i, j1 - 1), KEYS, i);
        if (i < NS - 2) load(min(j0 + i, j1 - 1), VALUES, i);
    }
    }

    // ---- queries: lane holds row l32, values 16 ks + 8 lhi ..
    u4 qf[KS];
    const int wrow = 32 * wave + l32;
    const bool live = wrow < rows;
    const int token = (int)q4::fast_div((uint32_t)(row0 + (live ? wrow : 0)), p.div_g);
    const int qh = head * p.g + row0 + (live ? wrow : 0) - token * p.g;
    const int pos = pos0 + token;
    float scale = p.scale;
    {
        const uint16_t* qp = p.q + (start + token) * p.q_t + qh * p.q_h;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int at = 16 * ks + 8 * lhi;
            qf[ks] = at < p.dim ? *reinterpret_cast<const u4*>(qp + at) : u4{0, 0, 0, 0};
        }
        if constexpr (H16 && BF) {
            uint32_t top = 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) top = max(top, q4cache4::largest_bf16(qf[ks]));
            const float most = max_halves(bitcast<float>(top));
            scale = q4cache4::row_scale(scale, most);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks] = q4cache4::bf16_to_f16(qf[ks], most);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[ks][e] = (qf[ks][e] & p.q_and) ^ p.q_xor;
            if constexpr (C4) qf[ks] = q4cache4::code_order(qf[ks]);
        }
    }
    const bool alive = 32 * wave < rows;       // (a wave without rows only loads)
    const int klo = p.window ? pos - p.window + 1 : 0;
    // keys that all of the wave's rows see
    const int w0 = min(32 * wave, rows - 1), w1 = min(32 * wave + 31, rows - 1);
    const int all_hi = pos0 + (int)q4::fast_div((uint32_t)(row0 + w0), p.div_g);
    const int all_lo = p.window ? pos0 + (int)q4::fast_div((uint32_t)(row0 + w1), p.div_g) - p.window + 1 : 0;

    auto partly = [&](int first) { return first + KT - 1 > all_hi || (first < all_lo && !(SK && first + KT <= p.sinks)); };

    f16x acc[DT], sa[HH], sb[HH];
    u4 pt[2 * HH];
    float m = kLow, l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
#pragma unroll
    for (int s = 0; s < 2 * HH; ++s) pt[s] = u4{0, 0, 0, 0};

    // LDS places of the lane's operands: of the keys by k-step, of the values by
    // 8-key half and output tile; stages and 16-key steps are immediate offsets
    constexpr int STAGE = KT * PITCH;
    const char *ka[KS], *va[2][DT];
    {
        const int j16 = lane & 15, dh = (lane >> 4) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) ka[ks] = lds_k[0] + ((l32 * PITCH + ((lhi ^ spread<D>(l32)) << 4)) ^ (ks << 5));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 8 * q + 4 * lhi + (j16 >> 2);
            const int at = row * PITCH + (((2 * dh + ((j16 >> 1) & 1)) ^ spread<D>(row)) << 4) + (j16 & 1) * 8;
#pragma unroll
            for (int d = 0; d < DT; ++d) va[q][d] = lds_v[0] + (at ^ (d << 6));
        }
    }
    auto mma = [](u4 x, u4 y, f16x c) {
        if constexpr (BI) return mfma32(bitcast<b8>(x), bitcast<b8>(y), c);
        else return mfma32(bitcast<h8>(x), bitcast<h8>(y), c);
    };
    auto scores = [&](int stage, f16x (&sc)[HH]) {
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[h][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < HH; ++h)
                sc[h] = mma(*reinterpret_cast<const u4*>(ka[ks] + stage * STAGE + h * 32 * PITCH), qf[ks], sc[h]);
    };
    auto output = [&](int stage) {
#pragma unroll
        for (int s = 0; s < 2 * HH; ++s)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u2 a0 = read_tr(va[0][d] + stage * STAGE + s * 16 * PITCH);
                const u2 a1 = read_tr(va[1][d] + stage * STAGE + s * 16 * PITCH);
                acc[d] = mma(u4{a0[0], a0[1], a1[0], a1[1]}, pt[s], acc[d]);
            }
    };
    auto barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Step i, tile j = j0 + i: the products of its neighbours, O^T += V^T P^T of
    // tile j - 1 and the scores of tile j + 1, with the weights of tile j between
    // them, which depend on neither. (A wave alone issues a vector instruction
    // each 8 cycles, two waves together one each 2 to 5, a product takes 32: the
    // two waves of a SIMD (heads of 64 and 128) fill both pipes this way, where weights and
    // products in turn leave each idle for half of the time.) The first step multiplies weights
    // of zero with a stage of zeros, the last one's scores are not used.
    //
    // Loads of keys run NS tiles ahead and of values NS - 2, into the stages that step
    // i - 1 read last; those that step i + 1 reads have landed at the end of step
    // i, the newer ones stay under way. (A load's latency is longer than a step, 1.7
    // to 2 us against 1: with two stages every step took that. Past the last tile the
    // loads repeat it, so that the count of those under way holds.) Over 4 bits no load stays under way from one
    // step to the next: what is fetched in step i is in its stage at the end of it.
    auto step = [&](auto par, int i, f16x (&cur)[HH], f16x (&nxt)[HH]) {
        constexpr int ST = decltype(par)::value;      // i % NS
        const int j = j0 + i;
        if constexpr (C4) {
            // (asked for here, unpacked into LDS at the end of the step: a step later would be
            // ten registers more, which the reads of the operands ahead of the products need)
            if (((i + NS) & 63) == 0 && j + NS < j1) batch4(j + NS, KEYS);
            fetch(min(j + NS, j1 - 1), KEYS, pk);
            if (((i + NS - 2) & 63) == 0 && j + NS - 2 < j1) batch4(j + NS - 2, VALUES);
            fetch(min(j + NS - 2, j1 - 1), VALUES, pv);
        } else {
        if (((i + NS - 2) & 63) == 0 && j + NS - 2 < j1) batch(j + NS - 2, VALUES);
        load(min(j + NS - 2, j1 - 1), VALUES, (ST + NS - 2) % NS);
        if (((i + NS) & 63) == 0 && j + NS < j1) batch(j + NS, KEYS);
        load(min(j + NS, j1 - 1), KEYS, ST);
        }
        if (alive) {
        const int first = key_of(j);
        if (partly(first)) {
#pragma unroll
            for (int h = 0; h < HH; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int key = first + 32 * h + 8 * (e >> 2) + 4 * lhi + (e & 3);
                    cur[h][e] = (key >= klo || (SK && key < p.sinks)) && key <= pos ? cur[h][e] : -INFINITY;
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        output((ST + NS - 1) % NS);
        scores((ST + 1) % NS, nxt);
        float top = cur[0][0];
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, cur[h][e]);
        const float mn = fmaxf(m, max_halves(top) * scale - lift<BI>(kSlack));
        const bool grow = __any(mn > m + kSlack);
        const float m1 = grow ? mn : m, a = exp2_fast(m - m1);
        float ls[2] = {l * a, 0.f};
#pragma unroll
        for (int h = 0; h < HH; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                cur[h][e] = exp2_fast(__builtin_fmaf(cur[h][e], scale, -m1));
                ls[e & 1] += cur[h][e];
            }
#pragma unroll
        for (int s = 0; s < 2 * HH; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 8 * (s & 1) + 2 * e;
                pt[s][e] = pack2<BI>(cur[s >> 1][at], cur[s >> 1][at + 1]);
            }
        l = ls[0] + ls[1];
        m = m1;
        // (held here: the compiler otherwise moves the weights past the barrier, to
        // where they are used)
#pragma unroll
        for (int s = 0; s < 2 * HH; ++s) asm volatile("" : "+v"(pt[s]));
        asm volatile("" : "+v"(l));
        __builtin_amdgcn_sched_group_barrier(0x100, D == 64 ? 16 : D == 128 ? 6 : 12, 0);
#pragma unroll
        for (int q = 0; q < 2 * HH * DT; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        }
#pragma unroll
        for (int q = 0; q < HH * KS; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (grow) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[d][e] *= a;
        }
        }
        if constexpr (C4) {
            if constexpr (RAW) wait_loads<0>();
            put(pk, KEYS, ST);
            put(pv, VALUES, (ST + NS - 2) % NS);
            wait_lds();
        } else {
            wait_loads<(NS - 2) * 2 * NI>();
        }
        barrier();
    };
    {
        // zeros where the first step's values would be
        u4* z = reinterpret_cast<u4*>(lds_v[NS - 1]);
        for (int i = tid; i < STAGE / 16; i += 64 * NW) z[i] = u4{0, 0, 0, 0};
    }
    wait_loads<0>();
    __syncthreads();
    if (alive) scores(0, sa);
    barrier();
    const int steps = j1 - j0;
    static_assert(NS == 4 || NS == 2, "stages by name");
    for (int i = 0;;) {
        step(std::integral_constant<int, 0>{}, i, sa, sb);
        if (++i == steps) break;
        step(std::integral_constant<int, 1>{}, i, sb, sa);
        if (++i == steps) break;
        if constexpr (NS == 4) {
            step(std::integral_constant<int, 2>{}, i, sa, sb);
            if (++i == steps) break;
            step(std::integral_constant<int, 3>{}, i, sb, sa);
            if (++i == steps) break;
        }
    }
    if (alive) output((steps - 1) & (NS - 1));
    wait_loads<0>();      // (no load may land in LDS that is no longer this workgroup's)

    // ---- outputs that are not finite, and keys that not all of the rows see: a
    // row may have them from a key that it does not see (q4_attend.h). The workgroup
    // then goes through its tiles again one by one, the partly visible ones key by key.
    const bool edges = key_of(j0) < all_lo || key_of(j1 - 1) + KT - 1 > all_hi;
    bool again = false;
    if (alive && edges) {
        float z = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) z = __builtin_fmaf(acc[d][e], 0.f, z);
        again = !(z == 0.f);
    }
    if (__syncthreads_or(again)) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
        m = kLow;
        l = 0.f;
#pragma clang loop unroll(disable)
        for (int j = j0; j < j1; ++j) {
            if constexpr (C4) {
                if (((j - j0) & 63) == 0) {
                    batch4(j, KEYS);
                    batch4(j, VALUES);
                }
                fetch(j, KEYS, pk);
                fetch(j, VALUES, pv);
                if constexpr (RAW) wait_loads<0>();
                put(pk, KEYS, 0);
                put(pv, VALUES, 0);
            } else {
                if (((j - j0) & 63) == 0) {
                    batch(j, KEYS);
                    batch(j, VALUES);
                }
                load(j, KEYS, 0);
                load(j, VALUES, 0);
                wait_loads<0>();
            }
            __syncthreads();
            if (alive) {
                scores(0, sa);
                __builtin_amdgcn_sched_barrier(0);
                const int first = key_of(j);
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < HH; ++h)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int key = first + 32 * h + 8 * (e >> 2) + 4 * lhi + (e & 3);
                        sa[h][e] = (key >= klo || (SK && key < p.sinks)) && key <= pos ? sa[h][e] : -INFINITY;
                        top = fmaxf(top, sa[h][e]);
                    }
                const float m1 = fmaxf(m, max_halves(top) * scale - lift<BI>(kSlack)), a = exp2_fast(m - m1);
                m = m1;
                l *= a;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[d][e] *= a;
#pragma unroll
                for (int h = 0; h < HH; ++h)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        sa[h][e] = exp2_fast(__builtin_fmaf(sa[h][e], scale, -m1));
                        l += sa[h][e];
                    }
#pragma unroll
                for (int s = 0; s < 2 * HH; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = 8 * (s & 1) + 2 * e;
                        pt[s][e] = pack2<BI>(sa[s >> 1][at], sa[s >> 1][at + 1]);
                    }
                if (partly(first)) {
                    // (key 16 s + 8 q + 4 h + e of the tile is value 4 q + e of pt[s] in lanes of half h)
#pragma unroll
                    for (int s = 0; s < 2 * HH; ++s)
#pragma clang loop unroll(disable)
                        for (int x = 0; x < 16; ++x) {
                            const int key = first + 16 * s + x;
                            const bool sees = (key >= klo || (SK && key < p.sinks)) && key <= pos;
#pragma unroll
                            for (int d = 0; d < DT; ++d) {
                                f16x y;
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = 0.f;
                                y = mma(lone(read_tr(va[0][d] + s * 16 * PITCH), read_tr(va[1][d] + s * 16 * PITCH),
                                             x >> 3 << 2 | (x & 3), lhi == (x >> 2 & 1)), pt[s], y);
#pragma unroll
                                for (int e = 0; e < 16; ++e) acc[d][e] += sees ? y[e] : 0.f;
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                } else {
                    output(0);
                }
            }
            __syncthreads();
        }
    }

    // ---- store, or leave a partial result
    const float ls = sum_halves(l);
    if (parts == 1) {
        if (live) {
            const float inv = over_sum(ls, pos);
            uint16_t* o = p.out + (start + token) * p.o_t + qh * p.o_h;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 32 * d + 8 * e + 4 * lhi;
                    if (at >= p.dim) continue;
                    const f4 y = f4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]};
                    store_row4<BF>(o + at, output_of(y, ls, inv), p.dim - at, p.store8);
                }
        }
        return;
    }
    // (never more slots than the workspace has, whatever `starts` says)
    const uint32_t slot0 = slots_before + ((uint32_t)row_tile * (uint32_t)p.KV + (uint32_t)head) * (uint32_t)splits;
    if (slot0 + (uint32_t)splits > 2u * (uint32_t)p.workers) return;
    if (split == 0 && tid == 0) {
        const uint32_t i = atomicAdd(&p.joins->count, 1u);
        if (i < (uint32_t)kMaxJoins) p.joins->item[i] = Join{start, row0, rows, head, (int)slot0, parts, pos0};
    }
    if (!live) return;
    constexpr size_t SLOT = (size_t)BR * (D + 2);
    float* own = p.slots + (size_t)(slot0 + (uint32_t)split) * SLOT;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f4*>(own + wrow * D + 32 * d + 8 * e + 4 * lhi) =
                f4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]};
    if (lhi == 0) {
        own[BR * D + wrow] = m;
        own[BR * D + BR + wrow] = ls;
    }
}

// Joins the splits of row tiles, in the order of the keys. A lane group of D / 4
// lanes takes a row, 4 values a lane; a launch of its own, because the one
// workgroup that arrives last at a row tile would take many microseconds for what
// every CU can share.
constexpr int JW = 4;            // waves of a workgroup
constexpr int kJoinGrid = 2048;

template <int D, bool BF>
__global__ __launch_bounds__(64 * JW) void q4_attend_join_kernel(Args p)
{
    constexpr int LG = D / 4, ROWS = JW * 64 / LG;   // rows of a workgroup at a time
    constexpr size_t SLOT = (size_t)BR * (D + 2);
    const int sub = (int)threadIdx.x / LG, at = (int)threadIdx.x % LG * 4;
    const int count = min(uniform((int)p.joins->count), kMaxJoins);
    for (int x = blockIdx.x; x < count * (BR / ROWS); x += kJoinGrid) {
        const Join& j = p.joins->item[x / (BR / ROWS)];
        const int row = x % (BR / ROWS) * ROWS + sub, parts = j.parts;
        if (row >= j.rows) continue;
        const float* slot = p.slots + (size_t)j.slot * SLOT;
        float m = kLow, l = 0.f;
        f4 v = f4{0.f, 0.f, 0.f, 0.f};
        constexpr int U = 8;               // splits whose loads are under way together
        for (int s0 = 0; s0 < parts; s0 += U) {
            f4 o[U];
            float w[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float* f = slot + (size_t)min(s0 + u, parts - 1) * SLOT;
                o[u] = *reinterpret_cast<const f4*>(f + row * D + at);
                w[u] = f[BR * D + row];
                q[u] = f[BR * D + BR + row];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s0 + u >= parts) continue;
                const float mx = fmaxf(m, w[u]), a = exp2_fast(m - mx), c = exp2_fast(w[u] - mx);
                l = a * l + c * q[u];
                v = a * v + c * o[u];
                m = mx;
            }
        }
        if (at >= p.dim) continue;
        const int r = j.row0 + row, token = (int)q4::fast_div((uint32_t)r, p.div_g);
        const f4 y = output_of(v, l, over_sum(l, j.pos0 + token));
        store_row4<BF>(p.out + (j.start + token) * p.o_t + (j.head * p.g + r - token * p.g) * p.o_h + at, y, p.dim - at, p.store8);
    }
    // The last workgroup that had work leaves the list empty (counted in groups:
    // thousands of additions to one address take tens of microseconds). One that
    // reads the count after that has none either.
    __syncthreads();
    const int active = min(kJoinGrid, count * (BR / ROWS)), group = (int)blockIdx.x % kJoinGroups;
    if (threadIdx.x || (int)blockIdx.x >= active) return;
    const uint32_t members = (uint32_t)((active - group + kJoinGroups - 1) / kJoinGroups), groups = (uint32_t)min(active, kJoinGroups);
    if (atomicAdd(&p.joins->group[group].done, 1u) != members - 1) return;
    p.joins->group[group].done = 0;
    if (atomicAdd(&p.joins->done, 1u) != groups - 1) return;
    p.joins->done = 0;
    p.joins->count = 0;
}

// What joins the splits of a launch before it.
template <int D>
hipError_t launch_join(const Args& p, bool bf16, hipStream_t stream)
{
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.unsplit) return e;
    if (bf16) hipLaunchKernelGGL((q4_attend_join_kernel<D, true>), dim3(kJoinGrid), dim3(64 * JW), 0, stream, p);
    else hipLaunchKernelGGL((q4_attend_join_kernel<D, false>), dim3(kJoinGrid), dim3(64 * JW), 0, stream, p);
    return hipGetLastError();
}

template <int D, bool SK, bool C4>
hipError_t launch_tiles(const Args& p, int grid, bool bf16, bool pg, hipStream_t stream)
{
    const dim3 g(grid), block(64 * NW);
    if (bf16 && pg) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, true, true, SK, C4, C4>), g, block, 0, stream, p);
    else if (bf16) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, true, false, SK, C4, C4>), g, block, 0, stream, p);
    else if (pg) hipLaunchKernelGGL((q4_attend_tiles_kernel<D, false, true, SK, C4, C4>), g, block, 0, stream, p);
    else hipLaunchKernelGGL((q4_attend_tiles_kernel<D, false, false, SK, C4, C4>), g, block, 0, stream, p);
    return launch_join<D>(p, bf16, stream);
}

// Queries of bfloat16 over keys and values of binary16, in pages of a multiple of 16 rows.
template <int D, bool SK>
hipError_t launch_halves(const Args& p, int grid, hipStream_t stream)
{
    hipLaunchKernelGGL((q4_attend_tiles_kernel<D, true, true, SK, false, true>), dim3(grid), dim3(64 * NW), 0, stream, p);
    return launch_join<D>(p, true, stream);
}

}  // namespace
