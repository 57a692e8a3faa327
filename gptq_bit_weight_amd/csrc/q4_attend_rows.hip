// Attention over a paged cache for few rows a request: single tokens and
// short runs of them.
//
// q4_attend_rows_kernel<D, BF, PG>: head rows of D values in LDS (64, 128,
// 256; a head's own dim may be less), BF (bfloat16), PG (pages of a multiple
// of 16 rows). A row tile is 16 rows (token, head of the group).
//
// Bound: HBM. Each key and value is read once for all rows of its tile and
// does 4 rows flops a value, far under the matrix rate. So the work is split
// by bytes: every (request, cached head, row tile) has its keys' 32-key tiles,
// and the workgroups take equal contiguous ranges of all of them, whatever the
// requests' lengths; a range's pieces of a row tile are segments. The ranges
// follow from starts and lengths, which each workgroup reads itself, so there
// is no planning launch and the host need not know them.
//
// A segment's tiles go round its four waves. A wave has one 32-key tile of
// keys and one of values in LDS of its own, filled by direct loads; the next
// keys are under way as soon as the scores of the present ones are formed,
// the next values when the present ones are multiplied, so the wave waits for
// memory alone and no barrier stands in the loop. One workgroup a CU has 32 to
// 64 KiB under way (D = 128), which suffices: 64 single tokens over 4600 keys on
// average take 221 us with one or with two (5.5 TB/s), and one token over 131000
// 106 us against 114, since each workgroup's share is one more partial result to join.
//
// At a segment's end the waves' running maxima, sums and outputs are joined
// in LDS. A segment that is its whole row tile is stored; else its partial
// result goes to a slot of its workgroup, and the last workgroup of the row
// tile to arrive joins them in key order (the same bits whichever it is).
#include "q4_attend.h"

namespace {

using namespace q4attend;

constexpr int WV = 4, NT = 64 * WV;
constexpr int KT = 32;                 // keys of a tile
constexpr int ROWS = 16;               // rows of one

// What of a request the kernel's split goes by: its row tiles, its first
// visible key, where its tiles begin (a multiple of 32) and their number (at least
// one: a tile of rows that see nothing still stores zeros).
struct Span {
    Request r;
    int rt, lo, base, nt;
};

__device__ __forceinline__ Span span(const Args& p, const Request& r)
{
    Span s;
    s.r = r;
    s.rt = (s.r.n * p.g + ROWS - 1) / ROWS;
    s.lo = p.window ? max(s.r.len - s.r.n - p.window + 1, 0) : 0;
    s.lo = min(s.lo, max(s.r.len - 1, 0));
    s.base = s.lo & ~(KT - 1);
    s.nt = max((s.r.len - s.base + KT - 1) / KT, 1);
    return s;
}

template <int D, bool BF, bool PG>
__global__ __launch_bounds__(NT, D == 256 ? 1 : 2) void q4_attend_rows_kernel(Args p)
{
    constexpr int PITCH = 2 * D;               // bytes of a row in LDS
    constexpr int CPR = D / 8;                 // 16-byte chunks of a row
    constexpr int RPI = 64 / CPR;              // rows one direct load fills
    constexpr int NI = KT / RPI;               // direct loads of a tile
    constexpr int KS = D / 32, DT = D / 16;    // k-steps of the scores; 16-value tiles of the output
    __shared__ __attribute__((aligned(1024))) char lds_k[WV][KT * PITCH];
    __shared__ __attribute__((aligned(1024))) char lds_v[WV][KT * PITCH];
    __shared__ float lds_m[WV][ROWS], lds_l[WV][ROWS];
    __shared__ int s_last;

    const int tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int lane = tid & 63;
    const int c16 = lane & 15, quad = lane >> 4;

    const uint32_t own_k = lds_address(lds_k[wave]), own_v = lds_address(lds_v[wave]);
    // the lane's byte offsets in 16 rows of keys and of values, one for each
    // direct load of them (a chunk past the head's end repeats its last one: it
    // meets zeros of the query, or makes output values that are not stored)
    constexpr int NB = NI / 2 < 4 ? NI / 2 : 4;
    uint32_t koff[NI / 2], voff[NI / 2];
#pragma unroll
    for (int e = 0; e < NI / 2; ++e) {
        const int row = e * RPI + lane / CPR;
        const uint32_t chunk = (uint32_t)min((lane % CPR) ^ spread<D>(row), p.chunks - 1) * 16u;
        koff[e] = (uint32_t)(row * p.ks2) + chunk;
        voff[e] = (uint32_t)(row * p.vs2) + chunk;
    }

    // ---- this workgroup's range of tiles
    // (the first 64 requests stay in the lanes: each look at them in memory is one
    // more latency before the first key)
    auto request_at = [&](int b) { return b < p.B ? request(p, b) : Request{0, 0, 0}; };
    auto cost = [&](const Request& r) {        // (0 without tokens)
        const Span s = span(p, r);
        return (uint32_t)s.rt * (uint32_t)p.KV * (uint32_t)s.nt;
    };
    auto scan = [&](uint32_t v) {              // inclusive, over the lanes
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)v, d);
            if (lane >= d) v += o;
        }
        return v;
    };
    const Request first64 = request_at(lane);
    const uint32_t cost64 = scan(cost(first64));
    uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)cost64, 63);
    for (int b0 = 64; b0 < p.B; b0 += 64) total += (uint32_t)__builtin_amdgcn_readlane((int)scan(cost(request_at(b0 + lane))), 63);
    // equal shares, in whole rounds of the waves
    uint32_t per = (total + (uint32_t)p.workers - 1) / (uint32_t)p.workers;
    per = (max(per, (uint32_t)p.least) + WV - 1) / WV * WV;
    const int me = (int)blockIdx.x;
    uint32_t it = (uint32_t)me * per;
    const uint32_t it_end = min(it + per, total);
    if (it >= it_end) return;
    int b = 0;
    uint32_t before = 0;                       // tiles of the requests before b
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        const uint32_t c = b0 ? scan(cost(request_at(b0 + lane))) : cost64;
        const unsigned long long past = __ballot(before + c > it);
        if (past) {
            const int f = (int)__builtin_ctzll(past);
            b = b0 + f;
            if (f) before += (uint32_t)__builtin_amdgcn_readlane((int)c, f - 1);
            break;
        }
        before += (uint32_t)__builtin_amdgcn_readlane((int)c, 63);
        b = b0 + 64;
    }

    for (; it < it_end && b < p.B; ++b) {
        Request r = b < 64 ? request_of_lane(first64, b) : request(p, b);
        r.start = uniform(r.start);
        r.n = uniform(r.n);
        r.len = uniform(r.len);
        Span s = span(p, r);
        s.rt = uniform(s.rt);
        s.lo = uniform(s.lo);
        s.base = uniform(s.base);
        s.nt = uniform(s.nt);
        const uint32_t pairs = (uint32_t)s.rt * (uint32_t)p.KV;
        const uint32_t mine = min(it_end, before + pairs * (uint32_t)s.nt);
        while (it < mine) {
            const uint32_t pair = (it - before) / (uint32_t)s.nt;
            const int tile0 = (int)(it - before - pair * (uint32_t)s.nt);
            const int tiles = min(s.nt - tile0, (int)(mine - it));
            // (row tiles of one head side by side: they read the same keys)
            const int head = (int)(pair / (uint32_t)s.rt), row0 = (int)(pair - (uint32_t)head * (uint32_t)s.rt) * ROWS;
            const int rows = min(ROWS, s.r.n * p.g - row0);
            const int pos0 = s.r.len - s.r.n;

            // ---- the wave's tiles: tile0 + wave, + 4, ...
            const int count = (tiles - wave + WV - 1) / WV;      // (0 or less: none)
            const int last_block = max(s.r.len - 1, 0) >> 4;
            const char* kh = reinterpret_cast<const char*>(p.k + head * p.ks1);
            const char* vh = reinterpret_cast<const char*>(p.v + head * p.vs1);
            // rows' byte offsets from kh and vh: of the 16-row block that
            // lane l / 2 steps on, half l % 2 (one load of page numbers for 32 tiles)
            long long ko = 0, vo = 0;
            auto locate = [&](int key) {       // of one key: its page's and row's offsets
                const int page_slot = (int)q4::fast_div((uint32_t)key, p.div_page);
                const uint32_t page = min((uint32_t)p.table[(long long)b * p.table_stride + page_slot], (uint32_t)p.pages - 1u);
                const int row = key - page_slot * p.page_size;
                ko = page * p.ks0 * 2 + (long long)row * p.ks2;
                vo = page * p.vs0 * 2 + (long long)row * p.vs2;
            };
            auto batch = [&](int i) {
                if constexpr (PG) {
                    const int tile = tile0 + wave + WV * (i + (lane >> 1));
                    const int block = min(max((s.base + tile * KT) / 16 + (lane & 1), s.lo >> 4), last_block);
                    locate(block * 16);
                }
            };
            // tile i of the wave, into its buffer
            auto load = [&](int i, auto values_tag) {
                constexpr bool values = decltype(values_tag)::value;
                const int first = s.base + (tile0 + wave + WV * i) * KT;
                const uint32_t dst = values ? own_v : own_k;
                const char* src = values ? vh : kh;
                const int pitch = values ? p.vs2 : p.ks2;
                const long long off = values ? vo : ko;
                if constexpr (PG) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int from = 2 * (i & 31) + h;
                        const uint32_t o0 = (uint32_t)__builtin_amdgcn_readlane((int)off, from);
                        const uint32_t o1 = (uint32_t)__builtin_amdgcn_readlane((int)(off >> 32), from);
                        const char* base = src + (long long)((uint64_t)o1 << 32 | o0);
                        // rows past the last key repeat it (nothing unwritten is read)
                        const int limit = max(s.r.len - 1, 0) - 16 * min(max((first >> 4) + h, s.lo >> 4), last_block);
#pragma unroll
                        for (int e0 = 0; e0 < NI / 2; e0 += NB) {
                            uint32_t at[NB];
#pragma unroll
                            for (int e = 0; e < NB; ++e) at[e] = values ? voff[e0 + e] : koff[e0 + e];
                            if (limit < 15)
#pragma unroll
                                for (int e = 0; e < NB; ++e) {
                                    const int row = (e0 + e) * RPI + lane / CPR;
                                    at[e] -= (uint32_t)((row - min(row, limit)) * pitch);
                                }
                            dma<NB>(base, at, dst + (uint32_t)(h * NI / 2 + e0) * 1024u);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < NI; ++e) {
                        const int row = e * RPI + lane / CPR;        // of the tile
                        const int chunk = min((lane % CPR) ^ spread<D>(row), p.chunks - 1);
                        locate(min(max(first + row, s.lo), max(s.r.len - 1, 0)));
                        dma_lane(src + (values ? vo : ko) + chunk * 16, dst + e * 1024u);
                    }
                }
            };
            constexpr std::false_type KEYS;
            constexpr std::true_type VALUES;
            if (count > 0) {
                batch(0);
                load(0, KEYS);
                load(0, VALUES);
            }

            // ---- queries: lane holds row c16 of each block, values 8 quad + 32 ks ..
            u4 qf[KS];
            int klo, khi;                      // the row's visible keys
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
                    const int at = 32 * ks + 8 * quad;
                    qf[ks] = at < p.dim ? *reinterpret_cast<const u4*>(qp + at) : u4{0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 4; ++e) qf[ks][e] = (qf[ks][e] & p.q_and) ^ p.q_xor;
                }
            }
            f4 acc[DT];
            float m = kLow, l = 0.f;
#pragma unroll
            for (int d = 0; d < DT; ++d) acc[d] = f4{0.f, 0.f, 0.f, 0.f};
            // keys of a tile that every live row sees
            const int all_hi = pos0 + (int)q4::fast_div((uint32_t)row0, p.div_g);
            const int all_lo = p.window ? pos0 + (int)q4::fast_div((uint32_t)(row0 + rows - 1), p.div_g) - p.window + 1 : 0;

            const char* kb = lds_k[wave] + c16 * PITCH;
            const int kx = (quad ^ spread<D>(c16)) << 4;
            const int vrow = 4 * quad + (c16 >> 2);
            const char* vb = lds_v[wave] + vrow * PITCH + (c16 & 1) * 8;
            const int vx = (((c16 >> 1) & 1) ^ spread<D>(vrow)) << 4;

            for (int i = 0; i < count; ++i) {
                const bool more = i + 1 < count;
                const int first = s.base + (tile0 + wave + WV * i) * KT;
                __builtin_amdgcn_sched_barrier(0);
                // the keys have landed (the values' loads, issued later, may be out)
                wait_loads<NI>();
                __builtin_amdgcn_sched_barrier(0);
                f4 sc[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const u4 a = *reinterpret_cast<const u4*>(kb + h * 16 * PITCH + (kx ^ (ks << 6)));
                        if constexpr (BF) sc[h] = mfma16(bitcast<b8>(a), bitcast<b8>(qf[ks]), sc[h]);
                        else sc[h] = mfma16(bitcast<h8>(a), bitcast<h8>(qf[ks]), sc[h]);
                    }
                // (every read of the keys issued before the first product)
                __builtin_amdgcn_sched_group_barrier(0x100, 2 * KS, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (more) {
                    if (((i + 1) & 31) == 0) batch(i + 1);
                    load(i + 1, KEYS);
                }
                __builtin_amdgcn_sched_barrier(0);
                // ---- softmax: lane holds keys first + 16 h + 4 quad + e of row c16
                sc[0] *= p.scale;
                sc[1] *= p.scale;
                const bool edge = first + KT - 1 > all_hi || first < all_lo;
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = first + 16 * h + 4 * quad + e;
                            sc[h][e] = key >= klo && key <= khi ? sc[h][e] : -INFINITY;
                        }
                }
                float top = kLow;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[h][e]);
                const float mn = fmaxf(m, max_quarters(top) - lift<BF>(0.f));
                if (__any(mn > m)) {
                    const float a = exp2_fast(m - mn);
                    l *= a;
#pragma unroll
                    for (int d = 0; d < DT; ++d) acc[d] *= a;
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
                const u4 pt = u4{pack2<BF>(w[0], w[1]), pack2<BF>(w[2], w[3]), pack2<BF>(w[4], w[5]), pack2<BF>(w[6], w[7])};
                __builtin_amdgcn_sched_barrier(0);
                if (more) wait_loads<NI>();
                else wait_loads<0>();
                __builtin_amdgcn_sched_barrier(0);
                // ---- O^T += V^T P^T: keys in the order in which the lanes hold P^T
                auto mma = [&](u4 a, f4 c) {
                    if constexpr (BF) return mfma16(bitcast<b8>(a), bitcast<b8>(pt), c);
                    else return mfma16(bitcast<h8>(a), bitcast<h8>(pt), c);
                };
                bool apart = false;
                if (edge) {
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const char* at = vb + (vx ^ (d << 5));
                        apart |= not_finite<BF>(read_tr(at)) | not_finite<BF>(read_tr(at + 16 * PITCH));
                    }
                    apart = __any(apart);
                }
                if (!apart) {
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const char* at = vb + (vx ^ (d << 5));
                        const u2 a0 = read_tr(at), a1 = read_tr(at + 16 * PITCH);
                        acc[d] = mma(u4{a0[0], a0[1], a1[0], a1[1]}, acc[d]);
                    }
                } else {
                    // (key 16 h + 4 q + e of the tile is value 4 h + e of the lanes of quad q)
#pragma clang loop unroll(disable)
                    for (int x = 0; x < KT; ++x) {
                        const bool sees = first + x >= klo && first + x <= khi;
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            const char* at = vb + (vx ^ (d << 5));
                            const u4 a = lone(read_tr(at), read_tr(at + 16 * PITCH), x >> 4 << 2 | (x & 3), quad == (x >> 2 & 3));
                            const f4 y = mma(a, f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[d][e] += sees ? y[e] : 0.f;
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if (more) load(i + 1, VALUES);
            }
            it += (uint32_t)tiles;

            // ---- join the waves: 16 rows of fp32 take a tile's buffer
            __syncthreads();
            {
                const float ls = sum_quarters(l);
                if (quad == 0) {
                    lds_m[wave][c16] = m;
                    lds_l[wave][c16] = ls;
                }
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    *reinterpret_cast<f4*>(lds_k[wave] + c16 * (4 * D) + (((4 * d + quad) ^ c16) << 4)) = acc[d];
            }
            __syncthreads();
            constexpr int UNITS = ROWS * (D / 4), UPT = UNITS / NT;   // four values of a row each
            const bool whole = tile0 == 0 && tiles == s.nt;
            const uint32_t pair_at = before + pair * (uint32_t)s.nt;
            // (workgroups there are, whatever `starts` says)
            const int wf = min((int)(pair_at / per), p.workers - 1);
            const int wl = min((int)((pair_at + (uint32_t)s.nt - 1) / per), p.workers - 1);
            constexpr size_t SLOT = (size_t)ROWS * (D + 2);
            auto slot_of = [&](int w) {
                return make_rsrc(p.slots + (size_t)(2 * w + (w == wf ? 1 : 0)) * SLOT, (uint32_t)(SLOT * 4));
            };
            const rsrc_t own = slot_of(me);
            f4 o[UPT];
            float om[UPT], ol[UPT];
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                const int unit = u * NT + tid, row = unit / (D / 4), c = unit % (D / 4);
                float mm = lds_m[0][row];
#pragma unroll
                for (int w = 1; w < WV; ++w) mm = fmaxf(mm, lds_m[w][row]);
                float ll = 0.f;
                f4 v = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < WV; ++w) {
                    const float a = exp2_fast(lds_m[w][row] - mm);
                    const f4 x = *reinterpret_cast<const f4*>(lds_k[w] + row * (4 * D) + ((c ^ row) << 4));
                    ll += a * lds_l[w][row];
                    v += a * x;
                }
                o[u] = v;
                om[u] = mm;
                ol[u] = ll;
                if (!whole && row < rows) {
                    put16(own, (uint32_t)unit * 16u, v);
                    if (c == 0) {
                        put4(own, (uint32_t)(ROWS * D + row) * 4u, mm);
                        put4(own, (uint32_t)(ROWS * D + ROWS + row) * 4u, ll);
                    }
                }
            }
            bool finish = whole;
            if (!whole) {
                __builtin_amdgcn_s_waitcnt(0);
                __syncthreads();
                if (tid == 0)
                    s_last = __hip_atomic_fetch_add(&p.counters[wf], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                             (uint32_t)(wl - wf);
                __syncthreads();
                finish = s_last != 0;
                if (finish) {
#pragma unroll
                    for (int u = 0; u < UPT; ++u) {
                        const int unit = u * NT + tid, row = unit / (D / 4);
                        float mm = kLow, ll = 0.f;
                        f4 v = f4{0.f, 0.f, 0.f, 0.f};
                        constexpr int FB = 16;     // slots whose loads are under way together
                        for (int w0 = wf; row < rows && w0 <= wl; w0 += FB) {
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
            if (finish) {
#pragma unroll
                for (int u = 0; u < UPT; ++u) {
                    const int unit = u * NT + tid, row = unit / (D / 4), at = unit % (D / 4) * 4;
                    if (row >= rows || at >= p.dim) continue;
                    const int r = row0 + row, token = (int)q4::fast_div((uint32_t)r, p.div_g);
                    const f4 y = output_of(o[u], ol[u], over_sum(ol[u], pos0 + token));
                    store_row4<BF>(p.out + (s.r.start + token) * p.o_t + (head * p.g + r - token * p.g) * p.o_h + at, y,
                                   p.dim - at, p.store8);
                }
            }
            __syncthreads();    // the buffers are free for the next segment
        }
        before += pairs * (uint32_t)s.nt;
    }
}

template <int D>
hipError_t launch_rows(const Args& p, bool bf16, bool pg, hipStream_t stream)
{
    const dim3 grid(p.workers), block(NT);
    if (bf16 && pg) hipLaunchKernelGGL((q4_attend_rows_kernel<D, true, true>), grid, block, 0, stream, p);
    else if (bf16) hipLaunchKernelGGL((q4_attend_rows_kernel<D, true, false>), grid, block, 0, stream, p);
    else if (pg) hipLaunchKernelGGL((q4_attend_rows_kernel<D, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((q4_attend_rows_kernel<D, false, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

namespace q4 {

hipError_t launch_attend_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, hipStream_t stream)
{
    if (p.dim < 8 || p.dim > 256 || p.dim % 8 || p.workers < 1) return hipErrorInvalidValue;
    if (p.dim <= 64) return launch_rows<64>(p, bf16, pages_of_16, stream);
    if (p.dim <= 128) return launch_rows<128>(p, bf16, pages_of_16, stream);
    return launch_rows<256>(p, bf16, pages_of_16, stream);
}

}  // namespace q4
