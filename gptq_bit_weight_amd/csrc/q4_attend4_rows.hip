// Attention over a paged cache held in 4 bits for few rows a request: single
// tokens and short runs of them.
//
// q4_attend4_rows_kernel<D, BF, PG, WV>: heads of up to D values (64, 128, 256), BF
// (bfloat16 queries and outputs), PG (pages of a multiple of 16 rows), WV waves a
// workgroup. A row tile is 16 rows (token, head of the group).
//
// The cache stands for binary16 values v = RNE(s c + m) (q4_cache4.h), which one packed
// multiply-add makes of two codes, so the products are those of a binary16 cache whatever
// the queries' type; queries of bfloat16 are brought into binary16's range by a power of two a
// row, which the scores are multiplied by again: exact but for values below 2^-31 of the row's largest.
//
// Bound: HBM, with the vector instructions that unpack close behind: a 32-key tile of a head of
// 128 is 4 KiB of codes and up to 1 KiB of scales, and takes a wave some 300 vector instructions
// (unpacking 13 for 8 values of a key, 7 for 4 of a value). A wave's tile of codes lies in LDS of its own,
// filled by direct loads, and the next one is asked for as soon as the present one is in registers; no
// barrier stands in the loop. Two waves a SIMD take turns: a workgroup of eight, or two of four, of which
// one multiplies while the other begins or joins a piece. (A second tile a wave in LDS, so that its loads
// are out for longer, takes the place of half of the waves: 123 us against 115.)
// 64 single tokens, 32 heads of 128 over 8, 384 MB of cache: 87 us, 4.4 TB/s (a large copy reaches 4.75 to 6);
// one token over 131000 keys, 143 MB: 42 us.
//
// With the scores taken as S^T = K Q^T a lane's operand is a piece of one key's row, and its 8
// values an instruction may be any 8 of the head as long as the queries' are the same 8: D / 4
// neighbouring ones a lane, one LDS read and one scale. For O^T = V^T P^T a lane's operand is 8 keys'
// values of one column; it reads 8 keys' codes of D / 16 neighbouring columns and pairs the keys
// by byte permutes, which makes D / 16 operands. Row i of the scores' product is key i / 4 +
// 4 (i % 4) of 16, so that the four rows which the lanes of a read touch are neighbours and fall on
// banks of their own; pieces of 16 bytes lie at place piece ^ spread4(row) of a row for the reads of keys.
//
// Work is shared out, joined and stored as in the kernel for 16 bits (q4_attend_rows.h).
#include "q4_attend_rows.h"
#include "q4_cache4.h"

namespace {

using namespace q4attend;
using namespace q4cache4;

// A piece of a row tile takes 4 to 5 us beside its tiles (the first loads, the join), a tile of a
// workgroup 0.5.
constexpr int kExtra = 8;

constexpr float kSlack = 8.f;    // log2 of the growth of a maximum that is let pass: a weight is at most 2^15

template <int D>
struct Shape {
    static constexpr int ROW = D / 2;                  // bytes of a row of codes
    static constexpr int CPR = D / 32;                 // pieces of 16 bytes of it, and scales of it in LDS (one for 32 values)
    static constexpr int RPI = 64 / CPR > 16 ? 16 : 64 / CPR;      // rows that one direct load fills
    static constexpr int NL = 16 / RPI;                // direct loads of 16 rows of codes; of scales as many
    static constexpr int NI = 4 * NL;                  // and of a tile's keys (or values)
    static constexpr int CODES = KT * ROW, SCALES = KT * CPR * 4, TILE = 2 * (CODES + SCALES);
    static constexpr bool OVER = D == 256;             // a wave's outputs take the place of its tiles in the end
    static constexpr int OUT = ROWS * 4 * D;           // bytes of its outputs
    static constexpr int KS = D / 32;                  // k-steps of the scores: words of a lane's piece of a key
    static constexpr int KG = D == 256 ? 2 : 1;        // scales of that piece
    static constexpr int VD = D / 16;                  // columns of a lane's piece of a value row
    static constexpr int VB = VD / 2;                  // its bytes: 2, 4, 8
    static constexpr int VW = VD > 8 ? 2 : 1;          // and words
};

template <int D>
__device__ __forceinline__ int spread4(int row)        // (of 16)
{
    return D == 64 ? row >> 3 & 1 : D == 128 ? row >> 2 & 3 : row >> 1 & 7;
}

template <int D, bool BF, bool PG, int WV>
__global__ __launch_bounds__(64 * WV, D == 256 ? 2 : 3) void q4_attend4_rows_kernel(Args p)
{
    using S = Shape<D>;
    constexpr int KS = S::KS, KG = S::KG, VD = S::VD, NL = S::NL, CPR = S::CPR;
    constexpr int WAVE = S::OVER && S::OUT > S::TILE ? S::OUT : S::TILE;
    __shared__ __attribute__((aligned(1024))) char lds[WV][WAVE];
    __shared__ __attribute__((aligned(1024))) char lds_other[S::OVER ? 1 : WV][S::OUT];
    auto& lds_o = [&]() -> auto& {
        if constexpr (S::OVER) return lds;
        else return lds_other;
    }();
    __shared__ float lds_m[WV][ROWS], lds_l[WV][ROWS];
    __shared__ int s_last;

    const int tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int lane = tid & 63;
    const int c16 = lane & 15, quad = lane >> 4;

    // ---- direct loads: the lane's bytes in 16 rows of keys and of values (the queries are
    // zero where the head has ended, and the outputs not stored: a piece past its end is the first one)
    const int lrow = lane / CPR, lpiece = lane % CPR;        // (of D = 64 half of the lanes load)
    const bool loads = D > 64 || lane < 32;
    auto column = [&](int piece) { return 32 * piece < p.dim ? piece : 0; };
    uint32_t koff[NL], voff[NL], ksoff[NL], vsoff[NL];
#pragma unroll
    for (int e = 0; e < NL; ++e) {
        const int row = e * S::RPI + lrow;
        const int c = column(lpiece ^ spread4<D>(row)) * 16, sc = (32 * column(lpiece) >> p.group_shift) * 4;
        koff[e] = (uint32_t)(row * p.k4.row + c);
        voff[e] = (uint32_t)(row * p.v4.row + c);
        ksoff[e] = (uint32_t)(row * p.k4.scale_row + sc);
        vsoff[e] = (uint32_t)(row * p.v4.scale_row + sc);
    }
    const uint32_t own = lds_address(lds[wave]);
    // ---- reads of them: key 16 h + krow, dims D / 4 quad ..; values 16 h + 4 e + quad, columns VD c16 ..
    const int krow = (c16 >> 2) + 4 * (c16 & 3);
    const char* kb = lds[wave] + krow * S::ROW;
    const char* ksb = lds[wave] + S::CODES + krow * (CPR * 4) + (D / 4 * quad / 32) * 4;
    const char* vb = lds[wave] + S::CODES + S::SCALES + quad * S::ROW;
    const char* vsb = lds[wave] + 2 * S::CODES + S::SCALES + quad * (CPR * 4) + (VD * c16 / 32) * 4;

    const Magic mg = magic();

    Share sh;
    if (!share_of<true, WV, kExtra>(p, lane, sh)) return;
    uint32_t it = sh.it;
    // ---- the share's next piece of a row tile
    Span s;
    Segment g;
    int b = sh.b;                              // its request
    uint32_t before = sh.before;               // tiles of the requests before it
    bool more = true;
    auto next_segment = [&]() __attribute__((always_inline)) {
        for (;; ++b) {
            if (it >= sh.end || b >= p.B) {
                more = false;
                return;
            }
            s = span_of<true>(p, sh, b);
            const uint32_t pairs = (uint32_t)s.rt * (uint32_t)p.KV, nt = sh.counted(s.nt);
            const uint32_t after = before + pairs * nt;
            while (it < after && it < sh.end) {
                const uint32_t pair = (it - before) / nt, from = before + pair * nt;
                g.pair_at = from + sh.extra;
                g.tile0 = max((int)(it - g.pair_at), 0);
                g.tiles = min((int)(min(sh.end, from + nt) - g.pair_at), s.nt) - g.tile0;
                it = from + nt;
                if (g.tiles <= 0) continue;        // (what comes before a row tile's first only)
                // (row tiles of one head side by side: they read the same keys)
                g.head = (int)(pair / (uint32_t)s.rt);
                g.row0 = (int)(pair - (uint32_t)g.head * (uint32_t)s.rt) * ROWS;
                g.rows = min(ROWS, s.r.n * p.g - g.row0);
                g.pos0 = s.r.len - s.r.n;
                return;
            }
            before = after;
        }
    };

    // ---- the wave's tiles of it: tile0 + wave, + WV, ... (0 or less: none)
    auto count_of = [&]() { return (g.tiles - wave + WV - 1) / WV; };
    auto last_key = [&]() { return max(s.r.len - 1, 0); };
    // addresses of the 16-row block that lane l / 2 steps on, half l % 2 (one load of
    // page numbers for 32 tiles)
    const char *kat = nullptr, *ksat = nullptr, *vat = nullptr, *vsat = nullptr;
    auto locate = [&](int key) __attribute__((always_inline)) {
        const Args& a = args_again();
        const int slot = (int)q4::fast_div((uint32_t)key, a.div_page);
        const long long page = min((uint32_t)a.table[(long long)b * a.table_stride + slot], (uint32_t)a.pages - 1u);
        const long long row = key - slot * a.page_size;
        kat = a.k4.at + g.head * a.k4.head + page * a.k4.page + row * a.k4.row;
        ksat = a.k4.scale + g.head * a.k4.scale_head + page * a.k4.scale_page + row * a.k4.scale_row;
        vat = a.v4.at + g.head * a.v4.head + page * a.v4.page + row * a.v4.row;
        vsat = a.v4.scale + g.head * a.v4.scale_head + page * a.v4.scale_page + row * a.v4.scale_row;
    };
    auto batch = [&](int i) __attribute__((always_inline)) {
        if constexpr (PG) {
            const int at = here(lane), tile = g.tile0 + wave + WV * (i + (at >> 1));
            locate(16 * min(seen_block<true>(p, s, s.key_of(tile) / 16 + (at & 1)), last_key() >> 4));
        }
    };
    auto at_lane = [](const char* p, int from) {
        const uint64_t v = reinterpret_cast<uint64_t>(p);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)v, from), hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), from);
        return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
    };
    auto load = [&](int i, auto values_tag) __attribute__((always_inline)) {
        constexpr bool values = decltype(values_tag)::value;
        const int first = s.key_of(g.tile0 + wave + WV * i);
        const uint32_t to = own + (uint32_t)(values ? S::CODES + S::SCALES : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (PG) {
                const int from = 2 * (i & 31) + h;
                const char *base = at_lane(values ? vat : kat, from), *scale_base = at_lane(values ? vsat : ksat, from);
                // rows past the last key repeat it (nothing unwritten is read)
                const int limit = last_key() - 16 * min(seen_block<true>(p, s, (first >> 4) + h), last_key() >> 4);
#pragma unroll
                for (int e = 0; e < NL; ++e) {
                    uint32_t at[1] = {values ? voff[e] : koff[e]}, sat = values ? vsoff[e] : ksoff[e];
                    if (limit < 15) {
                        const Side& side = values ? args_again().v4 : args_again().k4;
                        const int row = e * S::RPI + here(lane) / CPR, back = row - min(row, limit);
                        at[0] -= (uint32_t)(back * side.row);
                        sat -= (uint32_t)(back * side.scale_row);
                    }
                    if (loads) {
                        dma<1>(base, at, to + (uint32_t)(h * NL + e) * (S::RPI * S::ROW));
                        dma_words(scale_base, sat, to + S::CODES + (uint32_t)(h * NL + e) * (S::RPI * CPR * 4));
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < NL; ++e) {
                    const int row = e * S::RPI + lrow;
                    locate(min(seen_key<true>(p, s, first + 16 * h + (row & 15)), last_key()));
                    const int c = column(lpiece ^ spread4<D>(row)) * 16, sc = (32 * column(lpiece) >> p.group_shift) * 4;
                    if (loads) {
                        dma_lane((values ? vat : kat) + c, to + (uint32_t)(h * NL + e) * (S::RPI * S::ROW));
                        dma_words_lane((values ? vsat : ksat) + sc, to + S::CODES + (uint32_t)(h * NL + e) * (S::RPI * CPR * 4));
                    }
                }
            }
        }
    };
    constexpr std::false_type KEYS;
    constexpr std::true_type VALUES;
    auto begin = [&]() __attribute__((always_inline)) {
        const int count = count_of();
        if (count <= 0) return;
        batch(0);
        load(0, KEYS);
        load(0, VALUES);
    };

    next_segment();
    if (more) begin();
    while (more) {
        const int count = count_of();
        const int row0 = g.row0, rows = g.rows, pos0 = g.pos0, head = g.head;
        // ---- queries: lane holds row c16, values D / 4 quad + 8 ks .. in the order of the unpacked codes
        u4 qf[KS];
        int khi;                           // the row's last visible key (-1: a row that is none)
        float scale = p.scale;
        {
            const int c16 = here(lane) & 15, quad = here(lane) >> 4;
            const int r = row0 + c16;
            const bool live = c16 < rows;
            const int token = (int)q4::fast_div((uint32_t)r, p.div_g);
            const int pos = pos0 + token;
            khi = live ? pos : -1;
            const uint16_t* qp = p.q + (s.r.start + (live ? token : 0)) * p.q_t
                               + (head * p.g + (live ? r - token * p.g : 0)) * p.q_h;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int at = D / 4 * quad + 8 * ks;
                qf[ks] = at < p.dim ? *reinterpret_cast<const u4*>(qp + at) : u4{0, 0, 0, 0};
            }
            if constexpr (BF) {
                uint32_t top = 0;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) top = max(top, largest_bf16(qf[ks]));
                const float most = max_quarters(bitcast<float>(top));
                scale = row_scale(scale, most);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) qf[ks] = bf16_to_f16(qf[ks], most);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                for (int e = 0; e < 4; ++e) qf[ks][e] = (qf[ks][e] & p.q_and) ^ p.q_xor;
                qf[ks] = code_order(qf[ks]);
            }
        }
        f4 acc[VD];
        float m = kLow, l = 0.f;
#pragma unroll
        for (int d = 0; d < VD; ++d) acc[d] = f4{0.f, 0.f, 0.f, 0.f};
        // keys of a tile that every live row sees
        const int all_hi = pos0 + (int)q4::fast_div((uint32_t)row0, p.div_g);
        const int back = p.window ? p.window : 1 << 30;
        auto visible = [&](int key) { return (key > khi - back || key < p.sinks) && key <= khi; };
        const int all_lo = p.window ? pos0 + (int)q4::fast_div((uint32_t)(row0 + rows - 1), p.div_g) - p.window + 1 : 0;

        // Tile i; the next one is asked for into its place, its keys as soon as these keys are in
        // registers, its values when these values are.
        for (int i = 0; i < count; ++i) {
            const int after = count - 1 - i;       // tiles after this one
            const bool more = after >= 1;
            const int first = s.key_of(g.tile0 + wave + WV * i);
            // (the waves of a SIMD would be served in the order of their age, and the oldest be done when
            // the youngest has half of its tiles left: who has more of them left goes first)
            if (4 * after >= 3 * count) __builtin_amdgcn_s_setprio(3);
            else if (2 * after >= count) __builtin_amdgcn_s_setprio(2);
            else if (4 * after >= count) __builtin_amdgcn_s_setprio(1);
            else __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            // the keys have landed (the values, issued later, may be out)
            wait_loads<S::NI>();
            __builtin_amdgcn_sched_barrier(0);
            uint32_t kc[2][KS], ksm[2][KG];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char* at = kb + h * 16 * S::ROW;
                if constexpr (D == 64) {
                    const u2 w = *reinterpret_cast<const u2*>(at + (((quad >> 1) ^ spread4<D>(krow)) << 4) + (quad & 1) * 8);
                    kc[h][0] = w[0];
                    kc[h][1] = w[1];
                } else {
#pragma unroll
                    for (int t = 0; t < KG; ++t) {
                        const u4 w = *reinterpret_cast<const u4*>(at + (((KG * quad + t) ^ spread4<D>(krow)) << 4));
#pragma unroll
                        for (int e = 0; e < 4; ++e) kc[h][4 * t + e] = w[e];
                    }
                }
#pragma unroll
                for (int t = 0; t < KG; ++t) ksm[h][t] = *reinterpret_cast<const uint32_t*>(ksb + h * 16 * CPR * 4 + 4 * t);
            }
            wait_lds();
            if (more) {
                if (((i + 1) & 31) == 0) batch(i + 1);
                load(i + 1, KEYS);
            }
            __builtin_amdgcn_sched_barrier(0);
            f4 sc[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    const h2 step = low_half(ksm[h][g]), least = high_half(ksm[h][g]);
#pragma unroll
                    for (int e = 0; e < KS / KG; ++e) {
                        const int ks = g * (KS / KG) + e;
                        sc[h] = mfma16(bitcast<h8>(values8(kc[h][ks], step, least, mg)), bitcast<h8>(qf[ks]), sc[h]);
                    }
                }
            // ---- softmax: lane holds keys first + 16 h + 4 e + quad of row c16
            const bool edge = first + KT - 1 > all_hi || (first < all_lo && first + KT > p.sinks);
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = first + 16 * h + 4 * e + quad;
                        sc[h][e] = visible(key) ? sc[h][e] : -INFINITY;
                    }
            }
            float top = sc[0][0];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[h][e]);
            const float mn = fmaxf(m, max_quarters(top) * scale - lift<false>(kSlack));
            if (__any(mn > m + kSlack)) {
                const float a = exp2_fast(m - mn);
                l *= a;
#pragma unroll
                for (int d = 0; d < VD; ++d) acc[d] *= a;
                m = mn;
            }
            float w[8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[4 * h + e] = exp2_fast(__builtin_fmaf(sc[h][e], scale, -m));
                    l += w[4 * h + e];
                }
            const u4 pt = u4{pack2<false>(w[0], w[1]), pack2<false>(w[2], w[3]), pack2<false>(w[4], w[5]), pack2<false>(w[6], w[7])};
            __builtin_amdgcn_sched_barrier(0);
            if (more) wait_loads<S::NI>();
            else wait_loads<0>();
            __builtin_amdgcn_sched_barrier(0);
            uint32_t vc[8][S::VW], vsm[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int row = 16 * (x >> 2) + 4 * (x & 3);             // (and quad)
                const char* at = vb + row * S::ROW;
                const int byte = S::VB * c16, place = ((byte >> 4) ^ spread4<D>((row & 15) + quad)) << 4 | (byte & 15);
                if constexpr (S::VB == 2) vc[x][0] = *reinterpret_cast<const uint16_t*>(at + place);
                else if constexpr (S::VB == 4) vc[x][0] = *reinterpret_cast<const uint32_t*>(at + place);
                else {
                    const u2 w = *reinterpret_cast<const u2*>(at + place);
                    vc[x][0] = w[0];
                    vc[x][1] = w[1];
                }
                vsm[x] = *reinterpret_cast<const uint32_t*>(vsb + row * (CPR * 4));
            }
            wait_lds();
            if (more) load(i + 1, VALUES);
            __builtin_amdgcn_sched_barrier(0);
            // ---- O^T += V^T P^T: column VD c16 + d of the lane's eight keys, in the order in which the lanes hold P^T
            h2 step[4], least[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                step[x] = bitcast<h2>(__builtin_amdgcn_perm(vsm[2 * x + 1], vsm[2 * x], 0x05040100u));
                least[x] = bitcast<h2>(__builtin_amdgcn_perm(vsm[2 * x + 1], vsm[2 * x], 0x07060302u));
            }
            if (edge) {
                // A weight of zero does not keep a group that is not finite out of a sum. Such a group (its values
                // lie between those of its codes 0 and 15) is left out here, and what rows see of it is
                // NaN: counted by a product of marks, of the keys in the lane's columns and of what its row sees.
                uint32_t bad[4];
                bool any = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const h2 most = __builtin_elementwise_fma(bitcast<h2>(0x4b804b80u), step[x], least[x]);
                    const uint32_t a = bitcast<uint32_t>(most), c = bitcast<uint32_t>(least[x]);
                    const bool lo = (a & 0x7c00u) == 0x7c00u || (c & 0x7c00u) == 0x7c00u;
                    const bool hi = (a & 0x7c000000u) == 0x7c000000u || (c & 0x7c000000u) == 0x7c000000u;
                    bad[x] = (lo ? 0x3c00u : 0u) | (hi ? 0x3c000000u : 0u);
                    any |= lo || hi;
                }
                if (__any(any)) {
                    u4 sees;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t mark[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int key = first + 16 * (x >> 1) + 4 * (2 * (x & 1) + y) + quad;
                            mark[y] = visible(key) ? 0x3c00u : 0u;
                        }
                        sees[x] = mark[0] | mark[1] << 16;
                        const uint32_t keep = (bad[x] & 0x3c00u ? 0u : 0xffffu) | (bad[x] >> 16 ? 0u : 0xffff0000u);
                        step[x] = bitcast<h2>(bitcast<uint32_t>(step[x]) & keep);
                        least[x] = bitcast<h2>(bitcast<uint32_t>(least[x]) & keep);
                    }
                    const f4 seen = mfma16(bitcast<h8>(u4{bad[0], bad[1], bad[2], bad[3]}), bitcast<h8>(sees), f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int d = 0; d < VD; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[d][e] = seen[e] > 0.f ? __builtin_nanf("") : acc[d][e];
                }
            }
#pragma unroll
            for (int y = 0; y < VD / 2; ++y) {
                u4 even, odd;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const u2 w = values_of_pair(vc[2 * x][y / 4], vc[2 * x + 1][y / 4], y % 4, step[x], least[x], mg);
                    even[x] = w[0];
                    odd[x] = w[1];
                }
                acc[2 * y] = mfma16(bitcast<h8>(even), bitcast<h8>(pt), acc[2 * y]);
                acc[2 * y + 1] = mfma16(bitcast<h8>(odd), bitcast<h8>(pt), acc[2 * y + 1]);
            }
        }
        // ---- join the waves. The next piece's first tiles are asked for before.
        {
            const int c16 = here(lane) & 15, quad = here(lane) >> 4;
            const float ls = sum_quarters(l);
            if (quad == 0) {
                lds_m[wave][c16] = m;
                lds_l[wave][c16] = ls;
            }
            // (row 4 quad + e of acc[d] is column VD (4 quad + e) + d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int d = 0; d < VD; d += 4)
                    *reinterpret_cast<f4*>(lds_o[wave] + c16 * (4 * D) + (((VD / 4 * (4 * quad + e) + d / 4) ^ c16) << 4)) =
                        f4{acc[d][e], acc[d + 1][e], acc[d + 2][e], acc[d + 3][e]};
        }
        const Span s_done = s;
        const Segment g_done = g;
        next_segment();
        if (more && !S::OVER) begin();
        finish<D, BF, WV, true>(args_again(), sh, s_done, g_done, lds_o[0], S::OVER ? WAVE : S::OUT, lds_m[0], lds_l[0], &s_last);
        __syncthreads();    // the buffers are free for the next piece
        if (more && S::OVER) begin();
    }
}

template <int D, int WV>
hipError_t launch_rows(const Args& p, bool bf16, bool pg, hipStream_t stream)
{
    const dim3 grid(p.workers), block(64 * WV);
    if (bf16 && pg) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, true, true, WV>), grid, block, 0, stream, p);
    else if (bf16) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, true, false, WV>), grid, block, 0, stream, p);
    else if (pg) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, false, true, WV>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((q4_attend4_rows_kernel<D, false, false, WV>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

namespace q4 {

hipError_t launch_attend4_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, bool wide, hipStream_t stream)
{
    if (p.dim < 32 || p.dim > 256 || p.dim % 32 || p.workers < 1) return hipErrorInvalidValue;
    if (wide) {
        if (p.dim <= 64) return launch_rows<64, 8>(p, bf16, pages_of_16, stream);
        if (p.dim <= 128) return launch_rows<128, 8>(p, bf16, pages_of_16, stream);
        return launch_rows<256, 8>(p, bf16, pages_of_16, stream);
    }
    if (p.dim <= 64) return launch_rows<64, 4>(p, bf16, pages_of_16, stream);
    if (p.dim <= 128) return launch_rows<128, 4>(p, bf16, pages_of_16, stream);
    return launch_rows<256, 4>(p, bf16, pages_of_16, stream);
}

}  // namespace q4
