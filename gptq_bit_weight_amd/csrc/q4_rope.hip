// Rotary positions, alone and with the write of keys and values to a paged
// cache.
//
// A rotated pair (a, b) of a head at position t becomes
//   (a cos - b sin, b cos + a sin) * magnitude,  angle = t * frequency(pair),
// the transpose (the gradient's pass) with the sign of the sine turned.
//
// Angles. At position 10^6 an angle is 10^6 radians, so a product in fp32
// would keep none of its fraction. Each pair's frequency is held as a
// fraction of a turn in 64-bit fixed point; position * frequency modulo 2^64
// is then the exact fractional turn of the tabled frequency (also for negative
// positions), off by position * 2^-65 turns at most. Its two leading bits,
// rounded, give the quadrant, and the Taylor polynomials of sine and cosine
// take the rest (at most pi / 4): their first omitted terms are 1.8e-9
// (x^11 / 11!) and 1.2e-10 (x^12 / 12!), below fp32's 6e-8. (The hardware's
// sine has no stated bound of that size.)
//
// Bound: memory. Each value is read and written once, 16 bytes a lane. A
// workgroup takes a few tokens: its first lanes compute the tokens' cosines
// and sines into LDS, then every lane moves units of one chunk (interleaved
// pairs, the unrotated rest of a head, values) or two (a half layout's pairs)
// and rotates in fp32, rounded once.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>

#include "q4_device.h"
#include "q4_fastdiv.h"
#include "q4_ops.h"
#include "q4_turn.h"

namespace {

using namespace q4dev;

constexpr int NT = 256;
constexpr int kMaxTokens = 4;     // tokens of a workgroup
constexpr int kUnits = 4;         // units a lane has in flight
// Tokens of a launch: 2^32 lanes and more are a launch of their number modulo 2^32, without an error.
constexpr int kMostTokens = 1 << 25;
static_assert((long long)kMostTokens / kMaxTokens * NT < 1LL << 32, "lanes of a launch");

struct RopeArgs {
    const uint64_t* turns;
    float magnitude;
    int n, rot, dim;              // rotated pairs, rotated values, values of a head
    int H, KV, T, TB;             // heads of q; heads of k and v; tokens, tokens a workgroup
    int transpose;
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    long long q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    uint16_t *kc, *vc;
    long long kc_s[3], vc_s[3];   // page, head, row
    const void *positions, *slots;
    int positions64, slots64;
    int capacity, page_size;      // rows of the cache, rows of a page
    int lph, rotated, lpv;        // units of a rotated head, those of them that rotate, units of a value head
    int r1, ipt;                  // units of a token's rotated heads, and all of them
    q4::FastDiv div_ipt, div_lph, div_lpv, div_ps, div_n;
};

// V values a load (8: 16 bytes, 1: what no alignment allows more for); IL:
// interleaved pairs (2i, 2i + 1), else (i, i + n).
template <int V, bool IL, bool BF>
__global__ __launch_bounds__(NT) void q4_rope_kernel(RopeArgs p)
{
    extern __shared__ float2 cs[];      // [TB][n]
    const int t0 = (int)blockIdx.x * p.TB;
    const int tb = min(p.TB, p.T - t0);
    for (int i = threadIdx.x; i < tb * p.n; i += NT) {
        const int tt = p.TB == 1 ? 0 : (int)q4::fast_div((uint32_t)i, p.div_n);
        const uint64_t pos = (uint64_t)index_at(p.positions, p.positions64, t0 + tt);
        float2 e = turn_cos_sin(pos * p.turns[i - tt * p.n]);
        e.x *= p.magnitude;
        e.y *= p.transpose ? -p.magnitude : p.magnitude;
        cs[i] = e;
    }
    __syncthreads();
    constexpr int CR = V == 8 ? 8 : IL ? 2 : 1;    // values of a rotated chunk
    constexpr int CC = V;                          // values of a copied one
    const int step = NT * (int)gridDim.y;
    const int total = tb * p.ipt;
    for (int base = (int)blockIdx.y * NT + (int)threadIdx.x; base < total; base += kUnits * step) {
        u4 a[kUnits], b[kUnits];
        uint16_t* dst[kUnits];
        int at[kUnits];       // first pair in cs, or -1: a copy; -2: nothing
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int i = base + u * step;
            at[u] = -2;
            if (i >= total) continue;
            const int tt = p.TB == 1 ? 0 : (int)q4::fast_div((uint32_t)i, p.div_ipt);
            int rest = i - tt * p.ipt;
            const int t = t0 + tt;
            const bool value = rest >= p.r1;
            if (value) rest -= p.r1;
            const int head = (int)q4::fast_div((uint32_t)rest, value ? p.div_lpv : p.div_lph);
            const int un = rest - head * (value ? p.lpv : p.lph);
            const uint16_t* src;
            if (!value && head < p.H) {
                src = p.q + t * p.q_t + head * p.q_h;
                dst[u] = p.q_out + t * p.o_t + head * p.o_h;
            } else {
                const long long slot = index_at(p.slots, p.slots64, t);
                if (slot < 0 || slot >= p.capacity) continue;     // this token is not written
                const int page = (int)q4::fast_div((uint32_t)slot, p.div_ps);
                const int row = (int)slot - page * p.page_size;
                if (value) {
                    src = p.v + t * p.v_t + head * p.v_h;
                    dst[u] = p.vc + page * p.vc_s[0] + head * p.vc_s[1] + row * p.vc_s[2];
                } else {
                    const int kh = head - p.H;
                    src = p.k + t * p.k_t + kh * p.k_h;
                    dst[u] = p.kc + page * p.kc_s[0] + kh * p.kc_s[1] + row * p.kc_s[2];
                }
            }
            int off;
            if (!value && un < p.rotated) {
                off = un * CR;
                at[u] = tt * p.n + (IL ? off / 2 : off);
            } else {
                off = value ? un * CC : p.rot + (un - p.rotated) * CC;
                at[u] = -1;
            }
            dst[u] += off;
            src += off;
            if constexpr (V == 8) {
                a[u] = *reinterpret_cast<const u4*>(src);
                if (!IL && at[u] >= 0) b[u] = *reinterpret_cast<const u4*>(src + p.n);
            } else {
                a[u][0] = src[0];
                if (at[u] >= 0) b[u][0] = src[IL ? 1 : p.n];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (at[u] == -2) continue;
            if constexpr (V == 8) {
                if (at[u] >= 0) {
                    uint32_t o[8], w[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a0 = act_to_f32<BF>((uint16_t)a[u][e]), a1 = act_to_f32<BF>((uint16_t)(a[u][e] >> 16));
                        if constexpr (IL) {
                            const float2 f = cs[at[u] + e];
                            o[2 * e] = f32_to_act<BF>(a0 * f.x - a1 * f.y);
                            o[2 * e + 1] = f32_to_act<BF>(a1 * f.x + a0 * f.y);
                        } else {
                            const float b0 = act_to_f32<BF>((uint16_t)b[u][e]), b1 = act_to_f32<BF>((uint16_t)(b[u][e] >> 16));
                            const float2 f = cs[at[u] + 2 * e], g = cs[at[u] + 2 * e + 1];
                            o[2 * e] = f32_to_act<BF>(a0 * f.x - b0 * f.y);
                            o[2 * e + 1] = f32_to_act<BF>(a1 * g.x - b1 * g.y);
                            w[2 * e] = f32_to_act<BF>(b0 * f.x + a0 * f.y);
                            w[2 * e + 1] = f32_to_act<BF>(b1 * g.x + a1 * g.y);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[u][e] = o[2 * e] | o[2 * e + 1] << 16;
                        if constexpr (!IL) b[u][e] = w[2 * e] | w[2 * e + 1] << 16;
                    }
                    if constexpr (!IL) *reinterpret_cast<u4*>(dst[u] + p.n) = b[u];
                }
                *reinterpret_cast<u4*>(dst[u]) = a[u];
            } else {
                if (at[u] >= 0) {
                    const float2 f = cs[at[u]];
                    const float a0 = act_to_f32<BF>((uint16_t)a[u][0]), b0 = act_to_f32<BF>((uint16_t)b[u][0]);
                    dst[u][0] = f32_to_act<BF>(a0 * f.x - b0 * f.y);
                    dst[u][IL ? 1 : p.n] = f32_to_act<BF>(b0 * f.x + a0 * f.y);
                } else {
                    dst[u][0] = (uint16_t)a[u][0];
                }
            }
        }
    }
}

template <int V, bool IL>
hipError_t launch_v(const RopeArgs& p, dim3 grid, size_t lds, bool bf16, hipStream_t stream)
{
    if (bf16) hipLaunchKernelGGL((q4_rope_kernel<V, IL, true>), grid, dim3(NT), lds, stream, p);
    else hipLaunchKernelGGL((q4_rope_kernel<V, IL, false>), grid, dim3(NT), lds, stream, p);
    return hipGetLastError();
}

// Launch shape. Few tokens: a workgroup for each 256 units of each token, so
// that a decode step spreads over the CUs. Many: whole tokens, kMaxTokens to a
// workgroup.
hipError_t launch(RopeArgs& p, bool interleaved, bool wide, bool bf16, hipStream_t stream)
{
    const int cr = wide ? 8 : interleaved ? 2 : 1, cc = wide ? 8 : 1;
    p.rotated = p.rot / (interleaved ? cr : 2 * cr);
    p.lph = p.rotated + (p.dim - p.rot) / cc;
    p.lpv = p.dim / cc;
    p.r1 = (p.H + p.KV) * p.lph;
    p.ipt = p.r1 + (p.v ? p.KV * p.lpv : 0);
    const int slices = (p.ipt + NT - 1) / NT;
    const bool few = (long long)p.T * slices <= 4096;
    p.TB = few ? 1 : kMaxTokens;
    p.div_ipt = q4::make_fastdiv((uint32_t)p.ipt);
    p.div_lph = q4::make_fastdiv((uint32_t)p.lph);
    p.div_lpv = q4::make_fastdiv((uint32_t)p.lpv);
    p.div_n = q4::make_fastdiv((uint32_t)(p.n > 0 ? p.n : 1));
    p.div_ps = q4::make_fastdiv((uint32_t)(p.page_size > 0 ? p.page_size : 1));
    const size_t lds = (size_t)p.TB * (p.n > 0 ? p.n : 1) * sizeof(float2);
    for (int left = p.T;;) {
        p.T = std::min(left, kMostTokens);
        const dim3 grid((p.T + p.TB - 1) / p.TB, few ? slices : 1);
        hipError_t e;
        if (wide) e = interleaved ? launch_v<8, true>(p, grid, lds, bf16, stream) : launch_v<8, false>(p, grid, lds, bf16, stream);
        else e = interleaved ? launch_v<1, true>(p, grid, lds, bf16, stream) : launch_v<1, false>(p, grid, lds, bf16, stream);
        if (e != hipSuccess || (left -= p.T) == 0) return e;
        auto on = [&](auto*& at, long long stride) { at = at ? at + p.T * stride : at; };
        on(p.q, p.q_t);
        on(p.q_out, p.o_t);
        on(p.k, p.k_t);
        on(p.v, p.v_t);
        auto on_index = [&](const void*& at, int wide) { at = at ? static_cast<const char*>(at) + (long long)p.T * (wide ? 8 : 4) : at; };
        on_index(p.positions, p.positions64);
        on_index(p.slots, p.slots64);
    }
}

bool mult8(long long a) { return a % 8 == 0; }
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every 8-value chunk of the rotation lies on 16 bytes.
bool wide_rotation(const q4_rotary* r) { return mult8(r->dim) && mult8(r->rot) && (r->interleaved || mult8(r->rot / 2)); }

void set_rotary(RopeArgs& p, const q4_rotary* r, bool transpose)
{
    p.turns = r->turns;
    p.magnitude = r->magnitude;
    p.n = r->rot / 2;
    p.rot = r->rot;
    p.transpose = transpose;
}

}  // namespace

namespace q4 {

q4_status check_rotary(const q4_rotary* r, const void* positions, int position_bits, const char* who)
{
    if (!r || !positions) return fail(Q4_ERR_INVALID_ARG, "%s: null rotary or positions", who);
    if (position_bits != 32 && position_bits != 64)
        return fail(Q4_ERR_INVALID_ARG, "%s: positions of %d bits", who, position_bits);
    int cur = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
    if (cur != r->device)
        return fail(Q4_ERR_INVALID_ARG, "%s: the rotary table was made on device %d, the current device is %d", who, r->device, cur);
    return Q4_OK;
}

}  // namespace q4

extern "C" {

q4_rotary* q4_rotary_make(int dim, int rot, int layout, int scaling, double base, double factor,
                          int original_length, double low, double high)
{
    uint64_t turns[Q4_ROTARY_MAX_DIM / 2];
    float magnitude = 1.f;
    if (q4_rotary_plan(dim, rot, scaling, base, factor, original_length, low, high, turns, &magnitude) != Q4_OK)
        return nullptr;
    if (layout != Q4_ROTARY_HALF && layout != Q4_ROTARY_INTERLEAVED) {
        q4::fail(Q4_ERR_INVALID_ARG, "q4_rotary_make: unknown layout %d", layout);
        return nullptr;
    }
    int dev = -1, cu = 0;
    if (q4::device_info(&dev, &cu) != Q4_OK) return nullptr;
    uint64_t* table = nullptr;
    hipError_t e = hipMalloc(&table, (size_t)rot / 2 * sizeof(uint64_t));
    if (e == hipSuccess) e = hipMemcpy(table, turns, (size_t)rot / 2 * sizeof(uint64_t), hipMemcpyHostToDevice);
    q4_rotary* r = e == hipSuccess ? new (std::nothrow) q4_rotary : nullptr;
    if (!r) {
        (void)hipFree(table);
        q4::fail(e == hipSuccess || e == hipErrorOutOfMemory ? Q4_ERR_OOM : Q4_ERR_HIP, "q4_rotary_make: %s",
                 e == hipSuccess ? "out of memory" : hipGetErrorString(e));
        return nullptr;
    }
    r->turns = table;
    r->magnitude = magnitude;
    r->dim = dim;
    r->rot = rot;
    r->interleaved = layout == Q4_ROTARY_INTERLEAVED;
    r->device = dev;
    return r;
}

void q4_rotary_free(q4_rotary* r)
{
    if (!r) return;
    (void)hipFree(r->turns);
    delete r;
}

q4_status q4_rotary_apply(const q4_rotary* r, const uint16_t* x, int64_t x_token, int64_t x_head, uint16_t* out,
                          int64_t out_token, int64_t out_head, const void* positions, int position_bits,
                          int tokens, int heads, int transpose, int bf16, hipStream_t stream)
{
    const char* who = "q4_rotary_apply";
    if (tokens < 0 || heads < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (tokens == 0 || heads == 0) return Q4_OK;
    if (q4_status st = q4::check_rotary(r, positions, position_bits, who); st != Q4_OK) return st;
    if (!x || !out) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    if ((long long)heads * r->dim > (1 << 24)) return q4::fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^24 values a token", who);
    const q4::View to = q4::head_view(out, out_token, out_head, tokens, heads, r->dim);
    if (!q4::same_view(x, x_token, x_head, out, out_token, out_head, tokens, heads) &&
        q4::meet(to, q4::head_view(x, x_token, x_head, tokens, heads, r->dim)))
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: out overlaps its input without being the same view", who);
    if (q4::meet(to, q4::flat_view(positions, (int64_t)tokens * position_bits / 8)))
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: out overlaps the positions", who);
    RopeArgs p = {};
    set_rotary(p, r, transpose != 0);
    p.dim = r->dim;
    p.H = heads;
    p.T = tokens;
    p.q = x;
    p.q_out = out;
    p.q_t = x_token;
    p.q_h = x_head;
    p.o_t = out_token;
    p.o_h = out_head;
    p.positions = positions;
    p.positions64 = position_bits == 64;
    const bool wide = wide_rotation(r) && at16(x) && at16(out) && mult8(x_token) && mult8(x_head) && mult8(out_token) && mult8(out_head);
    hipError_t e = launch(p, r->interleaved, wide, bf16 != 0, stream);
    return e == hipSuccess ? Q4_OK : q4::fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

q4_status q4_cache_append(const q4_cache* c, const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                          int64_t v_token, int64_t v_head, const void* slots, int slot_bits, int tokens,
                          const q4_rotary* r, const void* positions, int position_bits, const uint16_t* q,
                          int64_t q_token, int64_t q_head, uint16_t* q_out, int64_t out_token, int64_t out_head,
                          int heads, hipStream_t stream)
{
    const char* who = "q4_cache_append";
    if (q4_status st = q4::check_cache(c, who); st != Q4_OK) return st;
    if (tokens < 0 || heads < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (tokens == 0) return Q4_OK;
    if (!k || !v || !slots) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null k, v or slots", who);
    if (slot_bits != 32 && slot_bits != 64) return q4::fail(Q4_ERR_INVALID_ARG, "%s: slots of %d bits", who, slot_bits);
    RopeArgs p = {};
    bool wide = mult8(c->dim), il = false;
    if (r) {
        if (q4_status st = q4::check_rotary(r, positions, position_bits, who); st != Q4_OK) return st;
        if (r->dim != c->dim) return q4::fail(Q4_ERR_INVALID_ARG, "%s: rotary heads of %d values, cache of %d", who, r->dim, c->dim);
        set_rotary(p, r, false);
        wide = wide_rotation(r);
        il = r->interleaved;
        p.positions = positions;
        p.positions64 = position_bits == 64;
    }
    if (q) {
        if (!r) return q4::fail(Q4_ERR_INVALID_ARG, "%s: q is given without a rotary", who);
        if (!q_out || heads < 1) return q4::fail(Q4_ERR_INVALID_ARG, "%s: q without heads or output", who);
        // (a workgroup writes its part of q_out while others read k and v)
        const q4::View to = q4::head_view(q_out, out_token, out_head, tokens, heads, c->dim);
        if (!q4::same_view(q, q_token, q_head, q_out, out_token, out_head, tokens, heads) &&
            q4::meet(to, q4::head_view(q, q_token, q_head, tokens, heads, c->dim)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps q without being the same view", who);
        if (q4::meet(to, q4::head_view(k, k_token, k_head, tokens, c->kv_heads, c->dim)) ||
            q4::meet(to, q4::head_view(v, v_token, v_head, tokens, c->kv_heads, c->dim)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps k or v", who);
        if (q4::meet(to, q4::cache_view(c, false)) || q4::meet(to, q4::cache_view(c, true)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps the cache", who);
        if (q4::meet(to, q4::flat_view(slots, (int64_t)tokens * slot_bits / 8)) ||
            q4::meet(to, q4::flat_view(positions, (int64_t)tokens * position_bits / 8)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps slots or positions", who);
        p.H = heads;
        p.q = q;
        p.q_t = q_token;
        p.q_h = q_head;
        p.q_out = q_out;
        p.o_t = out_token;
        p.o_h = out_head;
        wide = wide && at16(q) && at16(q_out) && mult8(q_token) && mult8(q_head) && mult8(out_token) && mult8(out_head);
    }
    if (((long long)p.H + 2LL * c->kv_heads) * c->dim > (1 << 24))
        return q4::fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^24 values a token", who);
    p.dim = c->dim;
    p.KV = c->kv_heads;
    p.T = tokens;
    p.k = k;
    p.k_t = k_token;
    p.k_h = k_head;
    p.v = v;
    p.v_t = v_token;
    p.v_h = v_head;
    p.kc = static_cast<uint16_t*>(c->k);
    p.vc = static_cast<uint16_t*>(c->v);
    for (int i = 0; i < 3; ++i) {
        p.kc_s[i] = c->k_stride[i];
        p.vc_s[i] = c->v_stride[i];
        wide = wide && mult8(c->k_stride[i]) && mult8(c->v_stride[i]);
    }
    wide = wide && at16(k) && at16(v) && at16(c->k) && at16(c->v) && mult8(k_token) && mult8(k_head) && mult8(v_token) && mult8(v_head);
    p.slots = slots;
    p.slots64 = slot_bits == 64;
    p.page_size = c->page_size;
    p.capacity = c->pages * c->page_size;
    hipError_t e = launch(p, il, wide, c->bf16 != 0, stream);
    return e == hipSuccess ? Q4_OK : q4::fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // extern "C"
