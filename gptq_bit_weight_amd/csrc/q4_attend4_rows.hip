// Attention over a paged cache held in 4 bits for few rows a request: single
// tokens and short runs of them.
//
// q4_attend4_rows_kernel<D, BF, PG>: heads of up to D values (64, 128, 256), BF
// (bfloat16 queries and outputs), PG (pages of a multiple of 16 rows). A row tile is 16
// rows (token, head of the group).
//
// The cache stands for binary16 values v = RNE(s c + m) (q4_cache4.h), which one packed
// multiply-add makes of two codes, so the products are those of a binary16 cache whatever
// the queries' type; queries of bfloat16 are brought into binary16's range by a power of two a
// row, which the scores are multiplied by again: exact but for values below 2^-32 of the row's largest.
//
// Bound: HBM, with the vector instructions that unpack close behind. A 32-key tile of a head of
// 128 is 4 KiB of codes and up to 1 KiB of scales, and takes a wave some 350 vector instructions
// (1.7 a value), so the codes go from memory straight to registers: with the scores' products
// taken as S^T = K Q^T, a lane's operand is a piece of one key's row, and its 8 values per
// instruction may be any 8 of the head as long as the queries' are the same 8. For O^T = V^T P^T a
// lane's operand is 8 keys' values of one column; it loads 8 keys' codes of D / 16 neighbouring
// columns and pairs the keys by byte permutes, which makes D / 16 operands.
//
// Work is shared out, joined and stored as in the kernel for 16 bits (q4_attend_rows.h).
// Each wave has the next tile's codes under way while it computes with the present one's.
#include "q4_attend_rows.h"
#include "q4_cache4.h"

namespace {

using namespace q4attend;
using namespace q4cache4;

template <int D>
struct Shape {
    static constexpr int WV = D == 256 ? 4 : 8;        // waves of a workgroup
    static constexpr int KS = D / 32;                  // k-steps of the scores: words of a lane's piece of a key
    static constexpr int KG = D == 256 ? 2 : 1;        // scales of that piece
    static constexpr int VD = D / 16;                  // columns of a lane's piece of a value row
    static constexpr int VB = VD / 2;                  // its bytes: 2, 4, 8
    static constexpr int VW = VD > 8 ? 2 : 1;          // and words
};

// Codes and scales of a tile in a lane's registers: of keys c16 and 16 + c16, dims
// D / 4 quad ..; of values 4 quad + e and 16 + 4 quad + e, columns VD c16 ..
template <int D>
struct Tile {
    using S = Shape<D>;
    uint32_t k[2][S::KS], ks[2][S::KG], v[8][S::VW], vs[8];
};

template <int D, bool BF, bool PG>
__global__ __launch_bounds__(64 * Shape<D>::WV, D == 256 ? 1 : 2) void q4_attend4_rows_kernel(Args p)
{
    using S = Shape<D>;
    constexpr int WV = S::WV, KS = S::KS, KG = S::KG, VD = S::VD;
    __shared__ __attribute__((aligned(1024))) char lds_o[WV][ROWS * 4 * D];
    __shared__ float lds_m[WV][ROWS], lds_l[WV][ROWS];
    __shared__ int s_last;

    const int tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int lane = tid & 63;
    const int c16 = lane & 15, quad = lane >> 4;

    // the lane's bytes of a row: a piece past the head's end is another one, with
    // scales of zero
    uint32_t kcol[KG], kscol[KG], vcol, vscol;
    bool kin[KG], vin;
#pragma unroll
    for (int t = 0; t < KG; ++t) {
        const int d = D / 4 * quad + 32 * t;
        kin[t] = d < p.dim;
        kcol[t] = kin[t] ? (uint32_t)d / 2u : 0u;
        kscol[t] = kin[t] ? (uint32_t)(d >> p.group_shift) * 4u : 0u;
    }
    {
        const int d = VD * c16;
        vin = d < p.dim;
        vcol = vin ? (uint32_t)d / 2u : 0u;
        vscol = vin ? (uint32_t)(d >> p.group_shift) * 4u : 0u;
    }

    Share sh;
    if (!share_of<true, WV>(p, lane, sh)) return;
    uint32_t it = sh.it;
    uint32_t before = sh.before;
    int b = sh.b;
    for (; it < sh.end && b < p.B; ++b) {
        const Span s = span_of<true>(p, sh, b);
        const uint32_t pairs = (uint32_t)s.rt * (uint32_t)p.KV;
        const uint32_t mine = min(sh.end, before + pairs * (uint32_t)s.nt);
        while (it < mine) {
            const uint32_t pair = (it - before) / (uint32_t)s.nt;
            const int tile0 = (int)(it - before - pair * (uint32_t)s.nt);
            const int tiles = min(s.nt - tile0, (int)(mine - it));
            // (row tiles of one head side by side: they read the same keys)
            const int head = (int)(pair / (uint32_t)s.rt), row0 = (int)(pair - (uint32_t)head * (uint32_t)s.rt) * ROWS;
            const int rows = min(ROWS, s.r.n * p.g - row0);
            const int pos0 = s.r.len - s.r.n;

            // ---- the wave's tiles: tile0 + wave, + WV, ...
            const int count = (tiles - wave + WV - 1) / WV;      // (0 or less: none)
            const int last_key = max(s.r.len - 1, 0), last_block = last_key >> 4;
            const char *kh = p.k4.at + head * p.k4.head, *ksh = p.k4.scale + head * p.k4.scale_head;
            const char *vh = p.v4.at + head * p.v4.head, *vsh = p.v4.scale + head * p.v4.scale_head;
            // page and row of a key
            auto locate = [&](int key, int& row) {
                const int slot = (int)q4::fast_div((uint32_t)key, p.div_page);
                row = key - slot * p.page_size;
                return (int)min((uint32_t)p.table[(long long)b * p.table_stride + slot], (uint32_t)p.pages - 1u);
            };
            // of the 16-row block that lane l / 2 steps on, half l % 2 (one load of
            // page numbers for 32 tiles)
            int page_of = 0, row_of = 0;
            auto batch = [&](int i) {
                if constexpr (PG) {
                    const int tile = tile0 + wave + WV * (i + (lane >> 1));
                    page_of = locate(16 * min(seen_block<true>(p, s, s.key_of(tile) / 16 + (lane & 1)), last_block), row_of);
                }
            };
            auto take_v = [&](uint32_t (&v)[S::VW], const char* at) {
                if constexpr (S::VB == 2) v[0] = *reinterpret_cast<const uint16_t*>(at);
                else if constexpr (S::VB == 4) v[0] = *reinterpret_cast<const uint32_t*>(at);
                else {
                    const u2 w = *reinterpret_cast<const u2*>(at);
                    v[0] = w[0];
                    v[1] = w[1];
                }
            };
            auto take_k = [&](uint32_t (&k)[KS], const char* at, const uint32_t (&off)[KG]) {
                if constexpr (KS == 2) {
                    const u2 w = *reinterpret_cast<const u2*>(at + off[0]);
                    k[0] = w[0];
                    k[1] = w[1];
                } else {
#pragma unroll
                    for (int t = 0; t < KG; ++t) {
                        const u4 w = *reinterpret_cast<const u4*>(at + off[t]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) k[4 * t + e] = w[e];
                    }
                }
            };
            auto load = [&](int i, Tile<D>& t) {
                if constexpr (PG) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int from = 2 * (i & 31) + h;
                        const long long page = __builtin_amdgcn_readlane(page_of, from);
                        const long long row = __builtin_amdgcn_readlane(row_of, from);
                        const char* kb = kh + page * p.k4.page + row * p.k4.row;
                        const char* ksb = ksh + page * p.k4.scale_page + row * p.k4.scale_row;
                        const char* vb = vh + page * p.v4.page + row * p.v4.row;
                        const char* vsb = vsh + page * p.v4.scale_page + row * p.v4.scale_row;
                        const int first = s.key_of(tile0 + wave + WV * i) / 16 + h;
                        // rows past the last key repeat it (nothing unwritten is read)
                        const int limit = last_key - 16 * min(seen_block<true>(p, s, first), last_block);
                        const uint32_t kr = (uint32_t)min(c16, limit);
                        uint32_t koff[KG];
#pragma unroll
                        for (int g = 0; g < KG; ++g) koff[g] = kr * (uint32_t)p.k4.row + kcol[g];
                        take_k(t.k[h], kb, koff);
#pragma unroll
                        for (int g = 0; g < KG; ++g)
                            t.ks[h][g] = *reinterpret_cast<const uint32_t*>(ksb + (kr * (uint32_t)p.k4.scale_row + kscol[g]));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t vr = (uint32_t)min(4 * quad + e, limit);
                            take_v(t.v[4 * h + e], vb + (vr * (uint32_t)p.v4.row + vcol));
                            t.vs[4 * h + e] = *reinterpret_cast<const uint32_t*>(vsb + (vr * (uint32_t)p.v4.scale_row + vscol));
                        }
                    }
                } else {
                    const int first = s.key_of(tile0 + wave + WV * i);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        int row;
                        long long page = locate(min(seen_key<true>(p, s, first + 16 * h + c16), last_key), row);
                        take_k(t.k[h], kh + page * p.k4.page + (long long)row * p.k4.row, kcol);
#pragma unroll
                        for (int g = 0; g < KG; ++g)
                            t.ks[h][g] = *reinterpret_cast<const uint32_t*>(ksh + page * p.k4.scale_page + (long long)row * p.k4.scale_row + kscol[g]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            page = locate(min(seen_key<true>(p, s, first + 16 * h + 4 * quad + e), last_key), row);
                            take_v(t.v[4 * h + e], vh + page * p.v4.page + (long long)row * p.v4.row + vcol);
                            t.vs[4 * h + e] = *reinterpret_cast<const uint32_t*>(vsh + page * p.v4.scale_page + (long long)row * p.v4.scale_row + vscol);
                        }
                    }
                }
            };
            Tile<D> ta, tb;
            if (count > 0) {
                batch(0);
                load(0, ta);
            }

            // ---- queries: lane holds row c16, values D / 4 quad + 8 ks .. in the order of the unpacked codes
            u4 qf[KS];
            int klo, khi;                      // the row's visible keys
            float scale = p.scale;
            {
                const int r = row0 + c16;
                const bool live = c16 < rows;
                const int token = (int)q4::fast_div((uint32_t)r, p.div_g);
                const int pos = pos0 + token;
                khi = live ? pos : -1;
                klo = p.window ? pos - p.window + 1 : 0;
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
                    scale *= halve_range(most);
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
            const int all_lo = p.window ? pos0 + (int)q4::fast_div((uint32_t)(row0 + rows - 1), p.div_g) - p.window + 1 : 0;

            auto compute = [&](int i, const Tile<D>& t) {
                const int first = s.key_of(tile0 + wave + WV * i);
                f4 sc[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < KG; ++g) {
                        const uint32_t sm = kin[g] ? t.ks[h][g] : 0u;
                        const h2 step = both(sm), least = both(sm >> 16);
#pragma unroll
                        for (int e = 0; e < KS / KG; ++e) {
                            const int ks = g * (KS / KG) + e;
                            sc[h] = mfma16(bitcast<h8>(values8(t.k[h][ks], step, least)), bitcast<h8>(qf[ks]), sc[h]);
                        }
                    }
                // ---- softmax: lane holds keys first + 16 h + 4 quad + e of row c16
                sc[0] *= scale;
                sc[1] *= scale;
                const bool edge = first + KT - 1 > all_hi || (first < all_lo && first + KT > p.sinks);
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = first + 16 * h + 4 * quad + e;
                            sc[h][e] = (key >= klo || key < p.sinks) && key <= khi ? sc[h][e] : -INFINITY;
                        }
                }
                float top = kLow;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[h][e]);
                const float mn = fmaxf(m, max_quarters(top) - lift<false>(0.f));
                if (__any(mn > m)) {
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
                        w[4 * h + e] = exp2_fast(sc[h][e] - m);
                        l += w[4 * h + e];
                    }
                const u4 pt = u4{pack2<false>(w[0], w[1]), pack2<false>(w[2], w[3]), pack2<false>(w[4], w[5]), pack2<false>(w[6], w[7])};
                // ---- O^T += V^T P^T: column VD c16 + d of the lane's eight keys, in the order in which the lanes hold P^T
                h2 step[4], least[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t s0 = vin ? t.vs[2 * x] : 0u, s1 = vin ? t.vs[2 * x + 1] : 0u;
                    step[x] = bitcast<h2>(__builtin_amdgcn_perm(s1, s0, 0x05040100u));
                    least[x] = bitcast<h2>(__builtin_amdgcn_perm(s1, s0, 0x07060302u));
                }
                auto columns = [&](int byte, u4& even, u4& odd) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const u2 y = values_of_pair(t.v[2 * x][byte / 4], t.v[2 * x + 1][byte / 4], byte % 4, step[x], least[x]);
                        even[x] = y[0];
                        odd[x] = y[1];
                    }
                };
                auto mma = [&](u4 a, f4 c) { return mfma16(bitcast<h8>(a), bitcast<h8>(pt), c); };
                bool apart = false;
                if (edge) {
#pragma unroll
                    for (int y = 0; y < VD / 2; ++y) {
                        u4 e, o;
                        columns(y, e, o);
#pragma unroll
                        for (int x = 0; x < 4; x += 2) apart |= not_finite<false>(u2{e[x], e[x + 1]}) || not_finite<false>(u2{o[x], o[x + 1]});
                    }
                    apart = __any(apart);
                }
                if (!apart) {
#pragma unroll
                    for (int y = 0; y < VD / 2; ++y) {
                        u4 e, o;
                        columns(y, e, o);
                        acc[2 * y] = mma(e, acc[2 * y]);
                        acc[2 * y + 1] = mma(o, acc[2 * y + 1]);
                    }
                } else {
                    // (key 16 h + 4 q + e of the tile is value 4 h + e of the lanes of quad q)
#pragma clang loop unroll(disable)
                    for (int x = 0; x < KT; ++x) {
                        const bool sees = (first + x >= klo || first + x < p.sinks) && first + x <= khi;
                        const int key = x >> 4 << 2 | (x & 3);
                        const bool lanes = quad == (x >> 2 & 3);
#pragma unroll
                        for (int y = 0; y < VD / 2; ++y) {
                            u4 e, o;
                            columns(y, e, o);
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const u4 a = z ? o : e;
                                const f4 r = mma(lone(u2{a[0], a[1]}, u2{a[2], a[3]}, key, lanes), f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                                for (int q = 0; q < 4; ++q) acc[2 * y + z][q] += sees ? r[q] : 0.f;
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
            };
            for (int i = 0; i < count; i += 2) {
                if (i + 1 < count) load(i + 1, tb);
                __builtin_amdgcn_sched_barrier(0);
                compute(i, ta);
                if (i + 1 >= count) break;
                __builtin_amdgcn_sched_barrier(0);
                if (i + 2 < count) {
                    if (((i + 2) & 31) == 0) batch(i + 2);
                    load(i + 2, ta);
                }
                __builtin_amdgcn_sched_barrier(0);
                compute(i + 1, tb);
                __builtin_amdgcn_sched_barrier(0);
            }
            it += (uint32_t)tiles;

            // ---- join the waves
            {
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
            finish<D, BF, WV>(p, sh, s, Segment{before + pair * (uint32_t)s.nt, tile0, tiles, head, row0, rows, pos0}, lds_o[0],
                              ROWS * 4 * D, lds_m[0], lds_l[0], &s_last);
            __syncthreads();    // the buffers are free for the next segment
        }
        before += pairs * (uint32_t)s.nt;
    }
}

template <int D>
hipError_t launch_rows(const Args& p, bool bf16, bool pg, hipStream_t stream)
{
    const dim3 grid(p.workers), block(64 * Shape<D>::WV);
    if (bf16 && pg) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, true, true>), grid, block, 0, stream, p);
    else if (bf16) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, true, false>), grid, block, 0, stream, p);
    else if (pg) hipLaunchKernelGGL((q4_attend4_rows_kernel<D, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((q4_attend4_rows_kernel<D, false, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

namespace q4 {

hipError_t launch_attend4_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, hipStream_t stream)
{
    if (p.dim < 32 || p.dim > 256 || p.dim % 32 || p.workers < 1) return hipErrorInvalidValue;
    if (p.dim <= 64) return launch_rows<64>(p, bf16, pages_of_16, stream);
    if (p.dim <= 128) return launch_rows<128>(p, bf16, pages_of_16, stream);
    return launch_rows<256>(p, bf16, pages_of_16, stream);
}

}  // namespace q4
