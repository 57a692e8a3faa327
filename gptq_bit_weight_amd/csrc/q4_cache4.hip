// New tokens into a paged cache held in 4 bits, and rows of it back.
//
// q4_cache4_append_kernel<WIDE, IL, BF, Q>: keys and values of new tokens, the keys turned by their
// positions, are quantised in groups of G = 32 .. 256 neighbouring values:
//   lo, hi = least and largest value (finite ones held within +-65440)
//   m = binary16(lo), s = binary16(fp32(hi - m) / 15)
//   c = (x - m) / s rounded to the nearest of 0 .. 15, ties to even (0 where s is 0)
// and a group with a value that is not finite gets s = m = NaN. What the cache then stands for
// is s c + m (q4_cache4.h). The queries are turned in the same launch.
//
// (x - m) / s in fp32, by the reciprocal, is off by 4 2^-24 of itself at most, 4e-6: a code that it leaves in doubt, within 1e-5
// of half way between two, is decided in 64 bits (some waves in a hundred). x is of the tokens' 16-bit
// type, so x - m is exact there and the remainder x - m - n s of a guess n is too: whether it passes half a
// step. (Of bfloat16 values under 2^-29 a difference from a large m is rounded to 53 bits: one within 2^-37 of
// a tie counts as the tie.) Keys are turned in 64 bits, rounded to fp32 and to the type, and then quantised: a code is the
// definition's and does not hang on the last bits of fp32. (64-bit instructions run at the
// rate of 32-bit ones here.) Queries are turned as q4_rope_kernel turns them.
//
// Bound: memory, for many tokens that of the queries (16384 tokens of 64 heads of 128 over 8: 599 MB in 120 us, 5.0
// TB/s; keys and values alone 48 us, bound by their vector instructions); for a few the launch. A row of keys or
// values is taken by as many lanes as it has pieces of 8 values, all in one wave: a lane reads its piece
// and the piece that it is paired with (from the cache beside it), the group's extremes pass
// through the lanes, a lane writes 4 bytes of codes and the group's first the scale. A lane of queries takes both
// pieces of a pair, several at once.
//
// q4_cache4_read_kernel: the rows of given slots as binary16.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "q4_cache4.h"
#include "q4_cache4_host.h"
#include "q4_fastdiv.h"
#include "q4_ops.h"
#include "q4_turn.h"

namespace {

using namespace q4dev;
using namespace q4cache4;

constexpr int NT = 256;
constexpr int kMaxTokens = 4;     // tokens of a workgroup
constexpr int kUnits = 4;         // units of queries that a lane has in flight
// Tokens of a launch: 2^32 lanes and more (of 3 workgroups for 4 tokens) are a launch of their number modulo 2^32, without an error.
constexpr int kMostTokens = 1 << 24;
static_assert(3LL * kMostTokens / kMaxTokens * NT < 1LL << 32, "lanes of a launch");

// Keys or values of the cache: strides in bytes.
struct Plane {
    char *at, *scale;
    long long page, head, row, scale_page, scale_head, scale_row;
};

struct AppendArgs {
    const uint64_t* turns;
    float magnitude;
    int n, rot, dim;                  // rotated pairs (0: none), rotated values, values of a head
    int H, KV, T, TB;                 // heads of q; heads of k and v; tokens, tokens a workgroup
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    uint32_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    Plane kc, vc;
    int group_lanes, group_shift;     // lanes of a group, log2 of its values
    const void *positions, *slots;
    int positions64, slots64;
    int capacity, page_size;          // rows of the cache, rows of a page
    int lanes_shift;                  // log2 of a row's lanes
    int groups;                       // workgroups (of grid.x) of keys, and of values
    int units, rotated;               // units of a head of q, those of them that are turned
    q4::FastDiv div_kv, div_heads, div_units, div_ps, div_n;
};

// Two values of the tokens' type, rounded.
template <bool BF>
__device__ __forceinline__ uint32_t pack_act(float x, float y)
{
    if constexpr (BF) return pack_bf16(x, y);
    else return bitcast<uint32_t>(__builtin_convertvector(ff2{x, y}, h2));
}

// Place of pair i among a token's 64-bit cosines and sines: a lane reads eight neighbours, and 8
// of them fall on 2 banks without the gap.
__host__ __device__ constexpr int place64(int i) { return i + (i >> 3); }

// The code of a value: d = x - m against steps of s, inv = 1 / s.
__device__ __forceinline__ uint32_t code_of(double d, double s, double inv)
{
    double n = __builtin_rint(d * inv);
    const double r = 2. * __builtin_fma(-n, s, d);      // exact: what is left, twice
    const bool odd = (int)n & 1;
    if (r > s || (r == s && odd)) n += 1.;
    else if (r < -s || (r == -s && odd)) n -= 1.;
    return (uint32_t)fmin(fmax(n, 0.), 15.);
}

// The queries of tb tokens from t0, in units of one chunk (interleaved pairs, the rest of a head) or of two
// that are paired, so that a value is read once; cs: cosines and sines [tb][n]. In fp32, rounded once.
template <bool WIDE, bool IL, bool BF>
__device__ __forceinline__ void turn_queries(const AppendArgs& p, const float2* cs, int t0, int tb)
{
    constexpr int V = WIDE ? 8 : 1, CR = WIDE ? 8 : IL ? 2 : 1;      // values of a chunk that is copied, and turned
    const int step = NT * (int)gridDim.y, total = tb * p.H * p.units;
    for (int base = (int)blockIdx.y * NT + (int)threadIdx.x; base < total; base += kUnits * step) {
        u4 a[kUnits], b[kUnits];
        uint16_t* dst[kUnits];
        int at[kUnits];                // first pair in cs, or -1: a copy
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int i = base + u * step;
            if (i >= total) continue;
            const int row = (int)q4::fast_div((uint32_t)i, p.div_units), un = i - row * p.units;
            const int tt = p.TB == 1 ? 0 : (int)q4::fast_div((uint32_t)row, p.div_heads), h = row - tt * p.H;
            const bool turned = un < p.rotated;
            const int off = turned ? un * CR : p.rot + (un - p.rotated) * V;
            const uint16_t* src = p.q + (uint64_t)(uint32_t)(t0 + tt) * p.q_t + (uint64_t)(uint32_t)h * p.q_h + off;
            dst[u] = p.q_out + (uint64_t)(uint32_t)(t0 + tt) * p.o_t + (uint64_t)(uint32_t)h * p.o_h + off;
            at[u] = turned ? tt * p.n + (IL ? off / 2 : off) : -1;
            if constexpr (WIDE) {
                a[u] = *reinterpret_cast<const u4*>(src);
                if (!IL && turned) b[u] = *reinterpret_cast<const u4*>(src + p.n);
            } else {
                a[u][0] = src[0];
                if (turned) b[u][0] = src[IL ? 1 : p.n];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (base + u * step >= total) continue;
            const float2* f = cs + max(at[u], 0);
            if constexpr (WIDE) {
                if (at[u] >= 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a0 = act_to_f32<BF>((uint16_t)a[u][e]), a1 = act_to_f32<BF>((uint16_t)(a[u][e] >> 16));
                        if constexpr (IL) {
                            a[u][e] = pack_act<BF>(a0 * f[e].x - a1 * f[e].y, a1 * f[e].x + a0 * f[e].y);
                        } else {
                            const float b0 = act_to_f32<BF>((uint16_t)b[u][e]), b1 = act_to_f32<BF>((uint16_t)(b[u][e] >> 16));
                            const float2 g0 = f[2 * e], g1 = f[2 * e + 1];
                            a[u][e] = pack_act<BF>(a0 * g0.x - b0 * g0.y, a1 * g1.x - b1 * g1.y);
                            b[u][e] = pack_act<BF>(b0 * g0.x + a0 * g0.y, b1 * g1.x + a1 * g1.y);
                        }
                    }
                    if constexpr (!IL) *reinterpret_cast<u4*>(dst[u] + p.n) = b[u];
                }
                *reinterpret_cast<u4*>(dst[u]) = a[u];
            } else {
                if (at[u] >= 0) {
                    const float a0 = act_to_f32<BF>((uint16_t)a[u][0]), b0 = act_to_f32<BF>((uint16_t)b[u][0]);
                    dst[u][0] = f32_to_act<BF>(a0 * f->x - b0 * f->y);
                    dst[u][IL ? 1 : p.n] = f32_to_act<BF>(b0 * f->x + a0 * f->y);
                } else {
                    dst[u][0] = (uint16_t)a[u][0];
                }
            }
        }
    }
}

// WIDE: pieces on 16 bytes, rotated by whole ones; IL: interleaved pairs (2i, 2i + 1), else (i, i + n).
// Q: with queries. (Eight waves a SIMD without them, 48 us against 55 for 16384 tokens of 8 heads of 128; with them memory
// decides, and the registers are worth more: 146 against 152.)
template <bool WIDE, bool IL, bool BF, bool Q>
__global__ __launch_bounds__(NT, WIDE && !Q ? 8 : 1) void q4_cache4_append_kernel(AppendArgs p)
{
    extern __shared__ double2 cs64[];                                   // [TB][place64(n)]
    const int row64 = place64(p.n);
    float2* cs = reinterpret_cast<float2*>(cs64);                       // or [TB][n]
    // A workgroup has rows of keys, of values or of queries only. The three of the same tokens are neighbours, so that the
    // keys' vector instructions run beside the queries' memory traffic (16384 tokens of 64 heads of 128 over 8, each
    // call after one that fills the cache: 146 us; the queries in a launch of their own before 178, last in this one 225). Without queries all keys come first, which
    // take longest (each beside its values: 60 us against 49, as half of the XCDs have the keys then).
    const int role = Q ? (int)(blockIdx.x % 3u) : (int)(blockIdx.x >= (uint32_t)p.groups);
    const int t0 = (Q ? (int)(blockIdx.x / 3u) : (int)blockIdx.x - role * p.groups) * p.TB;
    const int tb = min(p.TB, p.T - t0);
    const bool value = role == 1, query = Q && role == 2;
    const int rows = p.KV, step = (int)gridDim.y * (NT >> p.lanes_shift), total = tb * rows;
    if (query ? (int)blockIdx.y * NT >= tb * p.H * p.units : (int)blockIdx.y * (NT >> p.lanes_shift) >= total) return;
    for (int i = threadIdx.x; !value && i < tb * p.n; i += NT) {
        const int tt = p.TB == 1 ? 0 : (int)q4::fast_div((uint32_t)i, p.div_n);
        const uint64_t f = (uint64_t)index_at(p.positions, p.positions64, t0 + tt) * p.turns[i - tt * p.n];
        if (query) {
            float2 e = turn_cos_sin(f);
            e.x *= p.magnitude;
            e.y *= p.magnitude;
            cs[i] = e;
        } else {
            double2 d = turn_cos_sin64(f);
            d.x *= (double)p.magnitude;
            d.y *= (double)p.magnitude;
            cs64[tt * row64 + place64(i - tt * p.n)] = d;
        }
    }
    __syncthreads();
    if constexpr (Q)
        if (query) {
            turn_queries<WIDE, IL, BF>(p, cs, t0, tb);
            return;
        }
    const uint16_t* from = value ? p.v + t0 * (uint64_t)p.v_t : p.k + t0 * (uint64_t)p.k_t;
    const uint32_t token = value ? p.v_t : p.k_t, per_head = value ? p.v_h : p.k_h;
    const Plane& c = value ? p.vc : p.kc;
    // A lane's piece is the same in every round, and the lanes of a row stay together. (Lanes past the row's or the
    // rows' end go along with the last piece and row, and store nothing.)
    const int piece = (int)threadIdx.x & ((1 << p.lanes_shift) - 1);
    const bool inside = 8 * piece < p.dim;
    const int at = inside ? 8 * piece : p.dim - 8;
    const bool turned = !value && at < p.rot, second = !IL && at >= p.n;    // (second half of the rotated values, WIDE)
    for (int row0 = (int)blockIdx.y * (NT >> p.lanes_shift); row0 < total; row0 += step) {
        const int my_row = row0 + ((int)threadIdx.x >> p.lanes_shift), row = min(my_row, total - 1);
        const int tt = p.TB == 1 ? 0 : (int)q4::fast_div((uint32_t)row, p.div_kv);
        const int t = t0 + tt, h = row - tt * rows;
        const uint16_t* src = from + (uint64_t)(uint32_t)tt * token + (uint64_t)(uint32_t)h * per_head;
        const long long slot = index_at(p.slots, p.slots64, t);
        u4 x;                                  // the lane's values
        if constexpr (WIDE) {
            x = *reinterpret_cast<const u4*>(src + at);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (uint32_t)src[at + 2 * e] | (uint32_t)src[at + 2 * e + 1] << 16;
        }
        if (turned) {
            float b[8];                        // what they are paired with, negative for the first of a pair
            if constexpr (WIDE) {
                u4 o = x;
                if constexpr (!IL) o = *reinterpret_cast<const u4*>(src + (second ? at - p.n : at + p.n));
                const uint32_t flip = second ? 0u : 0x80008000u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = IL ? (x[e] >> 16 | x[e] << 16) ^ 0x8000u : o[e] ^ flip;
                    b[2 * e] = act_to_f32<BF>((uint16_t)w);
                    b[2 * e + 1] = act_to_f32<BF>((uint16_t)(w >> 16));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = at + e;
                    b[e] = 0.f;
                    if (d >= p.rot) continue;
                    const bool first = IL ? !(d & 1) : d < p.n;
                    b[e] = act_to_f32<BF>((uint16_t)(src[IL ? d ^ 1 : first ? d + p.n : d - p.n] ^ (first ? 0x8000u : 0u)));
                }
            }
            auto pair_of = [&](int e) { return IL ? (at + e) >> 1 : at + e >= p.n ? at + e - p.n : at + e; };
            const int pair0 = second ? at - p.n : at;
            float y[8];
            {
                const double2* f = cs64 + tt * row64;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = act_to_f32<BF>((uint16_t)(x[e / 2] >> 16 * (e & 1)));
                    if (!WIDE && at + e >= p.rot) continue;
                    // (eight neighbours from a multiple of 8 have no gap between them)
                    const double2 w = f[WIDE && !IL ? place64(pair0) + e : place64(pair_of(e))];
                    y[e] = (float)__builtin_fma((double)y[e], w.x, (double)b[e] * w.y);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = pack_act<BF>(y[2 * e], y[2 * e + 1]);
            }
        }
        const bool on = my_row < total && inside;
        // (not branched over: the lanes of a row pass their extremes on)
        float lo = INFINITY, hi = -INFINITY, odd = 0.f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = act_to_f32<BF>((uint16_t)(x[e / 2] >> 16 * (e & 1)));
            v[e] = fminf(fmaxf(a, -kLargest), kLargest);
            lo = fminf(lo, v[e]);
            hi = fmaxf(hi, v[e]);
            odd = __builtin_fmaf(a, 0.f, odd); // NaN once a value is not finite
        }
        if (!(odd == 0.f)) hi = INFINITY;
        for (int d = 1; d < p.group_lanes; d *= 2) {
            lo = fminf(lo, __shfl_xor(lo, d));
            hi = fmaxf(hi, __shfl_xor(hi, d));
        }
        if (!on || slot < 0 || slot >= p.capacity) continue;            // (else the token is not written)
        const bool finite = hi < INFINITY;
        const uint16_t m16 = finite ? f32_to_f16_bits(lo) : (uint16_t)0x7e00;
        const float m = f16_bits_to_f32(m16);
        const uint16_t s16 = finite ? f32_to_f16_bits((hi - m) / 15.f) : (uint16_t)0x7e00;
        const float s = f16_bits_to_f32(s16), inv = __builtin_amdgcn_rcpf(s);
        uint32_t word = 0;
        float doubt = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = (v[e] - m) * inv, n = __builtin_rintf(c);
            doubt = fmaxf(doubt, fabsf(c - n));
            word |= (uint32_t)fminf(fmaxf(n, 0.f), 15.f) << 4 * e;
        }
        if (doubt > 0.49999f) {
            const double inv64 = 1. / (double)s;
            word = 0;
#pragma clang loop unroll(disable)
            for (int e = 0; e < 8; ++e) {
                float y = v[0];
#pragma unroll
                for (int z = 1; z < 8; ++z) y = z == e ? v[z] : y;
                word |= code_of((double)y - (double)m, (double)s, inv64) << 4 * e;
            }
        }
        if (!(s > 0.f)) word = 0;
        const long long page = q4::fast_div((uint32_t)slot, p.div_ps);
        const long long r = slot - page * p.page_size;
        *reinterpret_cast<uint32_t*>(c.at + page * c.page + h * c.head + r * c.row + 4 * piece) = word;
        if ((piece & (p.group_lanes - 1)) == 0)
            *reinterpret_cast<uint32_t*>(c.scale + page * c.scale_page + h * c.scale_head + r * c.scale_row + 4 * (at >> p.group_shift)) =
                (uint32_t)s16 | (uint32_t)m16 << 16;
    }
}

template <bool WIDE, bool IL, bool BF>
void launch_append(const AppendArgs& p, dim3 grid, size_t lds, hipStream_t stream)
{
    if (p.H) hipLaunchKernelGGL((q4_cache4_append_kernel<WIDE, IL, BF, true>), grid, dim3(NT), lds, stream, p);
    else hipLaunchKernelGGL((q4_cache4_append_kernel<WIDE, IL, BF, false>), grid, dim3(NT), lds, stream, p);
}

template <bool WIDE, bool IL>
void launch_append(const AppendArgs& p, dim3 grid, size_t lds, bool bf16, hipStream_t stream)
{
    bf16 ? launch_append<WIDE, IL, true>(p, grid, lds, stream) : launch_append<WIDE, IL, false>(p, grid, lds, stream);
}

struct ReadArgs {
    Plane kc, vc;
    uint16_t *k, *v;
    long long k_t, k_h, v_t, v_h;
    const void* slots;
    int slots64, T, KV, pieces, group_shift, capacity, page_size, wide;
    q4::FastDiv div_pieces, div_heads, div_ps;
};

__global__ __launch_bounds__(NT) void q4_cache4_read_kernel(ReadArgs p)
{
    const long long total = 2LL * p.T * p.KV * p.pieces;
    for (long long base = (long long)blockIdx.x * NT; base < total; base += (long long)gridDim.x * NT) {
        const long long at = base + threadIdx.x;
        if (at >= total) return;
        const uint32_t i = (uint32_t)at;
        const uint32_t row = q4::fast_div(i, p.div_pieces);
        const int piece = (int)(i - row * (uint32_t)p.pieces);
        const int t = (int)q4::fast_div(row, p.div_heads), head = (int)row - t * 2 * p.KV;
        const bool value = head >= p.KV;
        const int h = value ? head - p.KV : head;
        const long long slot = index_at(p.slots, p.slots64, t);
        u4 w = u4{0, 0, 0, 0};
        if (slot >= 0 && slot < p.capacity) {
            const long long page = q4::fast_div((uint32_t)slot, p.div_ps);
            const long long r = slot - page * p.page_size;
            const Plane& c = value ? p.vc : p.kc;
            const uint32_t code = *reinterpret_cast<const uint32_t*>(c.at + page * c.page + h * c.head + r * c.row + 4 * piece);
            const uint32_t sm = *reinterpret_cast<const uint32_t*>(c.scale + page * c.scale_page + h * c.scale_head + r * c.scale_row +
                                                                   4 * (8 * piece >> p.group_shift));
            w = own_order(values8(code, low_half(sm), high_half(sm), magic()));
        }
        uint16_t* to = (value ? p.v + t * p.v_t + h * p.v_h : p.k + t * p.k_t + h * p.k_h) + 8 * piece;
        if (p.wide) {
            *reinterpret_cast<u4*>(to) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                to[2 * e] = (uint16_t)w[e];
                to[2 * e + 1] = (uint16_t)(w[e] >> 16);
            }
        }
    }
}

bool mult8(long long a) { return a % 8 == 0; }
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int log2_of(int n)
{
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

Plane plane_of(const q4_cache4* c, bool values)
{
    const int64_t* s = values ? c->v_stride : c->k_stride;
    const int64_t* w = values ? c->v_scale_stride : c->k_scale_stride;
    return Plane{static_cast<char*>(values ? c->v : c->k), static_cast<char*>(values ? c->v_scale : c->k_scale),
                 s[0], s[1], s[2], w[0], w[1], w[2]};
}

}  // namespace

extern "C" {

q4_status q4_cache4_append(const q4_cache4* c, const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                           int64_t v_token, int64_t v_head, const void* slots, int slot_bits, int tokens,
                           const q4_rotary* r, const void* positions, int position_bits, const uint16_t* q,
                           int64_t q_token, int64_t q_head, uint16_t* q_out, int64_t out_token, int64_t out_head,
                           int heads, int bf16, hipStream_t stream)
{
    const char* who = "q4_cache4_append";
    if (q4_status st = q4::check_cache4(c, who); st != Q4_OK) return st;
    if (tokens < 0 || heads < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (tokens == 0) return Q4_OK;
    if (!k || !v || !slots) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null k, v or slots", who);
    if (slot_bits != 32 && slot_bits != 64) return q4::fail(Q4_ERR_INVALID_ARG, "%s: slots of %d bits", who, slot_bits);
    for (int64_t x : {k_token, k_head, v_token, v_head, q ? q_token : 0, q ? q_head : 0, q ? out_token : 0, q ? out_head : 0})
        if (x < 0 || x > 0x7fffffff) return q4::fail(Q4_ERR_UNSUPPORTED, "%s: tokens or heads more than 2^31 - 1 values apart", who);
    const q4::View kin = q4::head_view(k, k_token, k_head, tokens, c->kv_heads, c->dim);
    const q4::View vin = q4::head_view(v, v_token, v_head, tokens, c->kv_heads, c->dim);
    if (q4::meets_cache4(kin, c) || q4::meets_cache4(vin, c)) return q4::fail(Q4_ERR_INVALID_ARG, "%s: k or v overlap the cache", who);
    if (q4::meets_cache4(q4::flat_view(slots, (int64_t)tokens * slot_bits / 8), c) ||
        (r && positions && q4::meets_cache4(q4::flat_view(positions, (int64_t)tokens * position_bits / 8), c)))
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: slots or positions overlap the cache", who);
    AppendArgs p = {};
    bool wide = true;
    if (r) {
        if (q4_status st = q4::check_rotary(r, positions, position_bits, who); st != Q4_OK) return st;
        if (r->dim != c->dim) return q4::fail(Q4_ERR_INVALID_ARG, "%s: rotary heads of %d values, cache of %d", who, r->dim, c->dim);
        p.turns = r->turns;
        p.magnitude = r->magnitude;
        p.n = r->rot / 2;
        p.rot = r->rot;
        p.positions64 = position_bits == 64;
        wide = mult8(r->rot) && (r->interleaved || mult8(r->rot / 2));
    }
    if (q) {
        if (!r) return q4::fail(Q4_ERR_INVALID_ARG, "%s: q is given without a rotary", who);
        if (!q_out || heads < 1) return q4::fail(Q4_ERR_INVALID_ARG, "%s: q without heads or output", who);
        // (a workgroup writes its part of q_out while others read k and v)
        const q4::View to = q4::head_view(q_out, out_token, out_head, tokens, heads, c->dim);
        if (!q4::same_view(q, q_token, q_head, q_out, out_token, out_head, tokens, heads) &&
            q4::meet(to, q4::head_view(q, q_token, q_head, tokens, heads, c->dim)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps q without being the same view", who);
        if (q4::meet(to, kin) || q4::meet(to, vin)) return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps k or v", who);
        if (q4::meets_cache4(to, c) || q4::meets_cache4(q4::head_view(q, q_token, q_head, tokens, heads, c->dim), c))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q or q_out overlap the cache", who);
        if (q4::meet(to, q4::flat_view(slots, (int64_t)tokens * slot_bits / 8)) ||
            q4::meet(to, q4::flat_view(positions, (int64_t)tokens * position_bits / 8)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps slots or positions", who);
        p.H = heads;
        p.q_t = (uint32_t)q_token;
        p.q_h = (uint32_t)q_head;
        p.o_t = (uint32_t)out_token;
        p.o_h = (uint32_t)out_head;
        wide = wide && at16(q) && at16(q_out) && mult8(q_token) && mult8(q_head) && mult8(out_token) && mult8(out_head);
    }
    if (((long long)p.H + 2LL * c->kv_heads) * c->dim > (1 << 24))
        return q4::fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^24 values a token", who);
    wide = wide && at16(k) && at16(v) && mult8(k_token) && mult8(k_head) && mult8(v_token) && mult8(v_head);
    p.dim = c->dim;
    p.KV = c->kv_heads;
    p.T = tokens;
    p.k_t = (uint32_t)k_token;
    p.k_h = (uint32_t)k_head;
    p.v_t = (uint32_t)v_token;
    p.v_h = (uint32_t)v_head;
    p.kc = plane_of(c, false);
    p.vc = plane_of(c, true);
    p.group_lanes = c->group / 8;
    p.group_shift = log2_of(c->group);
    p.slots64 = slot_bits == 64;
    p.page_size = c->page_size;
    p.capacity = c->pages * c->page_size;
    p.lanes_shift = log2_of(c->dim / 8);
    // Few tokens: a workgroup for each 256 lanes of each token, so that a decode step
    // spreads over the CUs. Many: whole tokens, kMaxTokens to a workgroup.
    const bool il = r && r->interleaved;
    const int turn = wide ? 8 : il ? 2 : 1;
    p.rotated = p.rot / (il ? turn : 2 * turn);
    p.units = p.rotated + (p.dim - p.rot) / (wide ? 8 : 1);
    const int lanes = std::max(p.KV << p.lanes_shift, p.H * p.units), slices = (lanes + NT - 1) / NT;
    const bool few = (long long)p.T * slices <= 4096;
    p.TB = few ? 1 : kMaxTokens;
    p.div_kv = q4::make_fastdiv((uint32_t)p.KV);
    p.div_heads = q4::make_fastdiv((uint32_t)(p.H > 0 ? p.H : 1));
    p.div_units = q4::make_fastdiv((uint32_t)p.units);
    p.div_ps = q4::make_fastdiv((uint32_t)p.page_size);
    p.div_n = q4::make_fastdiv((uint32_t)(p.n > 0 ? p.n : 1));
    const size_t lds = (size_t)p.TB * place64(p.n) * sizeof(double2);
    for (int t = 0; t < tokens; t += std::min(tokens - t, kMostTokens)) {
        p.T = std::min(tokens - t, kMostTokens);
        p.q = q ? q + t * q_token : nullptr;
        p.q_out = q ? q_out + t * out_token : nullptr;
        p.k = k + t * k_token;
        p.v = v + t * v_token;
        p.slots = static_cast<const char*>(slots) + (int64_t)t * (slot_bits / 8);
        p.positions = r ? static_cast<const char*>(positions) + (int64_t)t * (position_bits / 8) : nullptr;
        p.groups = (p.T + p.TB - 1) / p.TB;
        const dim3 grid((p.H ? 3u : 2u) * (unsigned)p.groups, few ? slices : 1);
        if (wide) il ? launch_append<true, true>(p, grid, lds, bf16 != 0, stream) : launch_append<true, false>(p, grid, lds, bf16 != 0, stream);
        else il ? launch_append<false, true>(p, grid, lds, bf16 != 0, stream) : launch_append<false, false>(p, grid, lds, bf16 != 0, stream);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? Q4_OK : q4::fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

q4_status q4_cache4_read(const q4_cache4* c, const void* slots, int slot_bits, int tokens, uint16_t* k, int64_t k_token,
                         int64_t k_head, uint16_t* v, int64_t v_token, int64_t v_head, hipStream_t stream)
{
    const char* who = "q4_cache4_read";
    if (q4_status st = q4::check_cache4(c, who); st != Q4_OK) return st;
    if (tokens < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (tokens == 0) return Q4_OK;
    if (!k || !v || !slots) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null k, v or slots", who);
    if (slot_bits != 32 && slot_bits != 64) return q4::fail(Q4_ERR_INVALID_ARG, "%s: slots of %d bits", who, slot_bits);
    if (2LL * tokens * c->kv_heads * (c->dim / 8) >= (1LL << 31))
        return q4::fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^34 values", who);
    const q4::View to[2] = {q4::head_view(k, k_token, k_head, tokens, c->kv_heads, c->dim),
                            q4::head_view(v, v_token, v_head, tokens, c->kv_heads, c->dim)};
    if (q4::meet(to[0], to[1])) return q4::fail(Q4_ERR_INVALID_ARG, "%s: k and v overlap", who);
    for (const q4::View& x : to)
        if (q4::meets_cache4(x, c) || q4::meet(x, q4::flat_view(slots, (int64_t)tokens * slot_bits / 8)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: k or v overlap the cache or slots", who);
    ReadArgs p = {};
    p.kc = plane_of(c, false);
    p.vc = plane_of(c, true);
    p.k = k;
    p.v = v;
    p.k_t = k_token;
    p.k_h = k_head;
    p.v_t = v_token;
    p.v_h = v_head;
    p.slots = slots;
    p.slots64 = slot_bits == 64;
    p.T = tokens;
    p.KV = c->kv_heads;
    p.pieces = c->dim / 8;
    p.group_shift = log2_of(c->group);
    p.capacity = c->pages * c->page_size;
    p.page_size = c->page_size;
    p.wide = at16(k) && at16(v) && mult8(k_token) && mult8(k_head) && mult8(v_token) && mult8(v_head);
    p.div_pieces = q4::make_fastdiv((uint32_t)p.pieces);
    p.div_heads = q4::make_fastdiv((uint32_t)(2 * p.KV));
    p.div_ps = q4::make_fastdiv((uint32_t)p.page_size);
    const long long blocks = (2LL * tokens * p.KV * p.pieces + NT - 1) / NT;
    hipLaunchKernelGGL(q4_cache4_read_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(NT), 0, stream, p);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? Q4_OK : q4::fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // extern "C"
