// C ABI of attention over a paged cache: argument checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "q4_attend.h"
#include "q4_cache4_host.h"

namespace q4 {

hipError_t launch_attend_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, hipStream_t stream);

hipError_t launch_attend_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream);

hipError_t launch_attend4_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, bool wide, hipStream_t stream);

hipError_t launch_attend4_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream);

// (0: more than 2^30 bytes)
size_t attend4_halves_bytes(int requests, int kv_heads, int max_len, int dim);
hipError_t launch_attend4_halves(q4attend::Args p, int grid, bool bf16, char* scratch, hipStream_t stream);

namespace {

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// The workspace: one arrival counter a workgroup, or the list of row tiles to
// join, then the partial results. (Both leave what they used at zero, but a join's
// entries are not: they lie past the counters.)
constexpr size_t kCounterBytes = 1 << 16, kListAt = 1 << 14;
static_assert(kListAt + sizeof(q4attend::JoinList) <= kCounterBytes, "workspace");

// The few-row kernel: rows of a tile, least tiles of a workgroup (of which there
// is one a CU).
constexpr int kFewRows = 16, kFewLeast = 4;
// Of 4 bits: two workgroups of four waves a CU, so that one multiplies while the other begins or joins
// a piece; where there are no more than 1 / 16 row tiles a CU, one of eight, whose partial results are half as many
// (64 single tokens of 8 cached heads, 4600 keys on average, 93 us against 113; 1 over 131000 49 against 42).
constexpr int kFew4 = 2, kFewWide4 = 16;
size_t rows_bytes(int dim, int num_cu)
{
    return kCounterBytes + (size_t)num_cu * 2 * kFewRows * (padded_dim(dim) + 2) * sizeof(float);
}

// The many-row kernel: rows of a workgroup, workgroups that it splits a call's
// work for (one a CU: the chip holds twice as many, but splitting for those costs
// more in joining than it fills), least key tiles of one, and its partial
// results. (A request is split where a row tile has more than 1 / target of all
// tiles: at most `target` row tiles are, into at most 2 target units.)
constexpr int kTileRows = 128, kTileLeast = 8;
// Row tiles that a window keeps to this many keys are not split where there are as many
// as workgroups wanted, which saves the join's launch: 1.5 to 2.5 us a call whatever the window,
// where requests are alike (1100 to 16000 tokens, 32 heads over 8; heads of 64, window
// 1024: 75.3 us against 76.6, heads of 128: 111.0 and 113.3, heads of 256, window 256: 60.7
// and 63.0). The price is paid where one request's long row tile stands beside many short ones:
// one of 32 tokens and 40 of 28, heads of 128: window 512 21.1 us against 21.8, 1024 28.9
// and 23.0, 2048 44.3 and 24.0, so no further than 24 tiles of 64. (With fewer row tiles splitting
// is always worth more: one chunk of 40 tokens 20.0 us against 26.0.)
constexpr int kWholeKeys = 24 * 64;
int tile_target(int num_cu) { return num_cu < q4attend::kMaxJoins ? num_cu : q4attend::kMaxJoins; }
size_t tiles_bytes(int dim, int num_cu)
{
    return kCounterBytes + (size_t)2 * tile_target(num_cu) * kTileRows * (padded_dim(dim) + 2) * sizeof(float);
}

q4_status check_attend(const q4_cache* c, int heads, const char* who)
{
    if (q4_status st = check_cache(c, who); st != Q4_OK) return st;
    if (c->dim % 8 || c->dim > 256)
        return fail(Q4_ERR_UNSUPPORTED, "%s: heads of %d values (a multiple of 8, at most 256)", who, c->dim);
    if (heads < 1 || heads % c->kv_heads)
        return fail(Q4_ERR_INVALID_ARG, "%s: %d heads over %d cached heads", who, heads, c->kv_heads);
    return Q4_OK;
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

q4_status check_attend4(const q4_cache4* c, int heads, const char* who)
{
    if (q4_status st = check_cache4(c, who); st != Q4_OK) return st;
    if (heads < 1 || heads % c->kv_heads)
        return fail(Q4_ERR_INVALID_ARG, "%s: %d heads over %d cached heads", who, heads, c->kv_heads);
    return Q4_OK;
}

// Of 4 bits: keys and values are brought into binary16 first where a request has so many rows on average, so that
// enough workgroups read what was unpacked once. (Rows, keys; unpacked by every workgroup and once: 32 heads of 128
// over 8, 32768 over 8192 669 us and 569, 8192 over 8192 302 and 276, 8192 over 2048 71 and 69, 4 requests of
// 2048 over 8192 325 and 307, 8 of 1024 over 4000 175 and 179; over 32, 2048 over 2048 72 and 76, 4 of 1024 over
// 2000 159 and 175; heads of 64, 6 of 2800 in a window of 1024 95 and 92; heads of 256, 8192 over 4096 262 and 237.)
constexpr int kHalvesRows = 2560;
int max_length(int table_width, int page_size) { return (int)std::min<long long>((long long)table_width * page_size, 1 << 30); }
size_t halves_bytes(int kv_heads, int dim, int g, int tokens, int requests, int max_len)
{
    if ((long long)tokens * g < (long long)kHalvesRows * requests) return 0;
    return attend4_halves_bytes(requests, kv_heads, max_len, dim);
}

size_t workspace_bytes_of(int dim, int cu, bool four)
{
    const size_t rows = rows_bytes(dim, four ? kFew4 * cu : cu), tiles = tiles_bytes(dim, cu);
    return rows > tiles ? rows : tiles;
}

// What a call says beside its cache.
struct Call {
    const uint16_t* q;
    int64_t q_token, q_head;
    int heads, tokens;
    const int32_t *starts, *lengths, *table;
    int table_width;
    int64_t table_stride;
    int requests, window, sinks;
    float scale;
    uint16_t* out;
    int64_t out_token, out_head;
    void* workspace;
    size_t workspace_bytes;
    bool bf16, four, far;     // far: row blocks of a page must not be told by 32-bit numbers of units
};

// The call over a cache that p describes already (pages, page_size, KV, dim and where its
// memory is) and that `caches` are the views of.
q4_status attend(const char* who, q4attend::Args& p, const View* caches, int ncaches, const Call& a, hipStream_t stream)
{
    if (a.tokens < 0 || a.requests < 0 || a.window < 0 || a.sinks < 0)
        return fail(Q4_ERR_INVALID_ARG, "%s: %d tokens, %d requests, window %d, %d sinks", who, a.tokens, a.requests, a.window, a.sinks);
    if (!std::isfinite(a.scale)) return fail(Q4_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (a.tokens == 0 || a.requests == 0) return Q4_OK;
    if (!a.q || !a.starts || !a.lengths || !a.table || !a.out) return fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    if (a.table_width < 1 || a.table_stride < a.table_width || a.table_stride > 0x7fffffff)
        return fail(Q4_ERR_INVALID_ARG, "%s: a table of %d pages a request, %lld apart", who, a.table_width, (long long)a.table_stride);
    if (a.q_token < 0 || a.q_token % 8 || a.q_head < 0 || a.q_head % 8)
        return fail(Q4_ERR_UNSUPPORTED, "%s: strides of q must be multiples of 8 values", who);
    if (!at16(a.q) || (reinterpret_cast<uintptr_t>(a.out) & 1))
        return fail(Q4_ERR_UNSUPPORTED, "%s: q must be 16-byte aligned", who);
    const int g = a.heads / p.KV;
    if ((long long)a.tokens * g > (1 << 30) || (long long)a.heads * p.dim > (1 << 30))
        return fail(Q4_ERR_UNSUPPORTED, "%s: %d tokens of %d heads", who, a.tokens, a.heads);
    // (row tiles are stored while others still read)
    const View to = head_view(a.out, a.out_token, a.out_head, a.tokens, a.heads, p.dim);
    if (meet(to, head_view(a.q, a.q_token, a.q_head, a.tokens, a.heads, p.dim)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps q", who);
    for (int i = 0; i < ncaches; ++i)
        if (meet(to, caches[i])) return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps the cache", who);
    if (meet(to, flat_view(a.starts, ((int64_t)a.requests + 1) * 4)) || meet(to, flat_view(a.lengths, (int64_t)a.requests * 4)) ||
        meet(to, View{a.table, (int64_t)a.table_width * 4, {{a.requests, a.table_stride * 4}, {1, 0}, {1, 0}}}))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps starts, lengths or table", who);
    int dev = -1, cu = 0;
    if (q4_status st = device_info(&dev, &cu); st != Q4_OK) return st;

    p.q = a.q;
    p.out = a.out;
    p.starts = a.starts;
    p.lengths = a.lengths;
    p.table = a.table;
    p.q_t = a.q_token;
    p.q_h = a.q_head;
    p.o_t = a.out_token;
    p.o_h = a.out_head;
    p.T = a.tokens;
    p.B = a.requests;
    p.g = g;
    p.chunks = p.dim / 8;
    p.table_stride = (int)a.table_stride;
    p.max_len = max_length(a.table_width, p.page_size);
    // (a window that no key can lie outside is none; the kernels' 32-bit positions less a
    // window then stay in range)
    p.window = a.window >= p.max_len ? 0 : a.window;
    p.sinks = p.window ? std::min(a.sinks, p.max_len) : 0;
    // (a negative scale turns q's signs, a scale of zero clears q)
    // (finite with log2 e too: infinity times a score of 0 would be NaN)
    p.scale = a.scale == 0.f ? 1.f : std::min(std::fabs(a.scale) * 1.4426950408889634f, std::numeric_limits<float>::max());
    p.q_and = a.scale == 0.f ? 0u : ~0u;
    p.q_xor = a.scale < 0.f ? 0x80008000u : 0u;
    p.store8 = (reinterpret_cast<uintptr_t>(a.out) % 8 == 0) && a.out_token % 4 == 0 && a.out_head % 4 == 0;
    p.div_g = make_fastdiv((uint32_t)g);
    p.div_page = make_fastdiv((uint32_t)p.page_size);
    const bool pg = p.page_size % 16 == 0 && !a.far;

    // Few rows a request: the few-row kernel, above the many-row one. (64 x 8
    // rows over 4600 keys: 221 us and 237; 8 x 16 over 3000: 32 and 28; 20 x 32 over
    // 6000: 115 and 102.) By their mean, as the host knows no more: a long chunk beside
    // many single tokens costs more in one call than apart (63 single tokens and a chunk of
    // 512 over 8192 keys: 8 heads over 8, few rows, 450 us, apart 359 and 37; 32 heads over 8,
    // many rows, 546 us, apart 360 and 88.) In 4 bits the many-row kernel has its vector instructions to share
    // with the unpacking, and the border lies higher: 20 x 48 rows over 6000 keys 108 us and 125,
    // 20 x 64 125 and 121, 20 x 96 174 and 125; 16 x 64 of heads of 64 over 2000 32 and 34.
    const long long mean_rows = ((long long)a.tokens * g + a.requests - 1) / a.requests;
    const bool many = mean_rows > (a.four ? 64 : 12);
    const int tile = many ? kTileRows : kFewRows;
    const long long row_tiles = (long long)a.tokens * g / tile + a.requests;
    if (row_tiles * p.KV * (p.max_len / 32 + 2 + (a.four ? 8 : 0)) >= (1LL << 31))
        return fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^31 tiles of keys", who);
    const bool wide = a.four && (long long)a.requests * p.KV * kFewWide4 <= cu;
    p.workers = many ? tile_target(cu) : a.four && !wide ? kFew4 * cu : cu;
    p.least = many ? kTileLeast : kFewLeast;
    if (many) {
        const int keys = p.dim > 128 ? 32 : 64;
        // (a row tile's tokens see window - 1 keys before the first's own, and the sinks)
        const long long seen = p.window ? (long long)p.window + (kTileRows + g - 1) / g : p.max_len;
        const long long most = std::min(std::min<long long>(seen, p.max_len) / keys + 2 + (p.sinks + keys - 1) / keys,
                                        (long long)p.max_len / keys + 2);
        const bool enough = (long long)a.tokens * g / kTileRows * p.KV >= tile_target(cu);
        if (p.window && most * keys <= kWholeKeys && enough) p.least = (int)most;
        p.unsplit = most <= p.least;
    }
    const size_t need = many ? tiles_bytes(p.dim, cu) : rows_bytes(p.dim, p.workers);
    if (!a.workspace || a.workspace_bytes < need || !at16(a.workspace))
        return fail(Q4_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes on a 16-byte boundary (%s_workspace)", who, need,
                    a.four ? "q4_attend4" : "q4_attend");
    p.counters = static_cast<uint32_t*>(a.workspace);
    p.joins = reinterpret_cast<q4attend::JoinList*>(static_cast<char*>(a.workspace) + kListAt);
    p.slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounterBytes);
    // (most units there can be: a whole one each share of the work, a partial one each row tile and head. They are workgroups
    // of 256 lanes, and 2^32 lanes and more HIP launches modulo 2^32, without an error)
    const int units = (int)(row_tiles * p.KV + p.workers);
    if (many && units >= 1 << 24)
        return fail(Q4_ERR_UNSUPPORTED, "%s: %d units of 128 rows of a request and cached head, 2^24 and more", who, units);
    hipError_t e;
    const size_t halves = a.four && many ? halves_bytes(p.KV, p.dim, g, a.tokens, a.requests, p.max_len) : 0;
    if (halves && a.workspace_bytes >= need + halves)
        e = launch_attend4_halves(p, units, a.bf16, static_cast<char*>(a.workspace) + need, stream);
    else if (a.four) e = many ? launch_attend4_tiles(p, units, a.bf16, pg, stream) : launch_attend4_rows(p, a.bf16, pg, wide, stream);
    else e = many ? launch_attend_tiles(p, units, a.bf16, pg, stream) : launch_attend_rows(p, a.bf16, pg, stream);
    return e == hipSuccess ? Q4_OK : fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // namespace
}  // namespace q4

extern "C" {

size_t q4_attend_workspace(const q4_cache* c, int heads)
{
    int dev = -1, cu = 0;
    if (q4::check_attend(c, heads, "q4_attend_workspace") != Q4_OK || q4::device_info(&dev, &cu) != Q4_OK) return 0;
    return q4::workspace_bytes_of(c->dim, cu, false);
}

q4_status q4_attend_ex(const q4_cache* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                       const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                       int64_t table_stride, int requests, int window, int sinks, float scale, uint16_t* out, int64_t out_token,
                       int64_t out_head, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    using namespace q4;
    const char* who = "q4_attend";
    if (q4_status st = check_attend(c, heads, who); st != Q4_OK) return st;
    if (tokens > 0 && requests > 0) {
        const int64_t strides[] = {c->k_stride[0], c->k_stride[1], c->k_stride[2], c->v_stride[0], c->v_stride[1], c->v_stride[2]};
        for (int64_t s : strides)
            if (s < 0 || s % 8) return fail(Q4_ERR_UNSUPPORTED, "%s: strides of the cache must be multiples of 8 values", who);
        if (!at16(c->k) || !at16(c->v)) return fail(Q4_ERR_UNSUPPORTED, "%s: the cache must be 16-byte aligned", who);
        if (c->k_stride[2] > (1 << 25) || c->v_stride[2] > (1 << 25))
            return fail(Q4_ERR_UNSUPPORTED, "%s: rows of a page more than 2^25 values apart", who);
    }
    q4attend::Args p = {};
    p.k = static_cast<const uint16_t*>(c->k);
    p.v = static_cast<const uint16_t*>(c->v);
    p.ks0 = c->k_stride[0];
    p.ks1 = c->k_stride[1];
    p.ks2 = (int)c->k_stride[2] * 2;
    p.vs0 = c->v_stride[0];
    p.vs1 = c->v_stride[1];
    p.vs2 = (int)c->v_stride[2] * 2;
    p.KV = c->kv_heads;
    p.dim = c->dim;
    p.pages = c->pages;
    p.page_size = c->page_size;
    const View caches[] = {cache_view(c, false), cache_view(c, true)};
    return attend(who, p, caches, 2, Call{q, q_token, q_head, heads, tokens, starts, lengths, table, table_width, table_stride, requests,
                                          window, sinks, scale, out, out_token, out_head, workspace, workspace_bytes, c->bf16 != 0, false, false}, stream);
}

q4_status q4_attend(const q4_cache* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                    const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                    int64_t table_stride, int requests, int window, float scale, uint16_t* out, int64_t out_token,
                    int64_t out_head, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return q4_attend_ex(c, q, q_token, q_head, heads, tokens, starts, lengths, table, table_width, table_stride, requests, window, 0,
                        scale, out, out_token, out_head, workspace, workspace_bytes, stream);
}

size_t q4_attend4_workspace(const q4_cache4* c, int heads)
{
    int dev = -1, cu = 0;
    if (q4::check_attend4(c, heads, "q4_attend4_workspace") != Q4_OK || q4::device_info(&dev, &cu) != Q4_OK) return 0;
    return q4::workspace_bytes_of(c->dim, cu, true);
}

size_t q4_attend4_workspace_for(const q4_cache4* c, int heads, int tokens, int requests, int table_width)
{
    const size_t least = q4_attend4_workspace(c, heads);
    if (!least || tokens < 1 || requests < 1 || table_width < 1) return least;
    int dev = -1, cu = 0;
    if (q4::device_info(&dev, &cu) != Q4_OK) return 0;
    const size_t halves = q4::halves_bytes(c->kv_heads, c->dim, heads / c->kv_heads, tokens, requests, q4::max_length(table_width, c->page_size));
    return std::max(least, halves ? q4::tiles_bytes(c->dim, cu) + halves : 0);
}

q4_status q4_attend4(const q4_cache4* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                     const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                     int64_t table_stride, int requests, int window, int sinks, float scale, uint16_t* out, int64_t out_token,
                     int64_t out_head, void* workspace, size_t workspace_bytes, int bf16, hipStream_t stream)
{
    using namespace q4;
    const char* who = "q4_attend4";
    if (q4_status st = check_attend4(c, heads, who); st != Q4_OK) return st;
    q4attend::Args p = {};
    auto side = [&](bool values) {
        const int64_t *s = values ? c->v_stride : c->k_stride, *w = values ? c->v_scale_stride : c->k_scale_stride;
        return q4attend::Side{static_cast<const char*>(values ? c->v : c->k), static_cast<const char*>(values ? c->v_scale : c->k_scale),
                              s[0], s[1], w[0], w[1], (int)s[2], (int)w[2]};
    };
    p.k4 = side(false);
    p.v4 = side(true);
    for (p.group_shift = 5; 1 << p.group_shift < c->group;) ++p.group_shift;
    p.KV = c->kv_heads;
    p.dim = c->dim;
    p.pages = c->pages;
    p.page_size = c->page_size;
    // (many rows: 32 bits count the codes' 16 bytes and the scales' 4)
    bool far = false;
    for (int v = 0; v < 2; ++v) {
        const int64_t *s = v ? c->v_stride : c->k_stride, *w = v ? c->v_scale_stride : c->k_scale_stride;
        far = far || (double)c->pages * (double)s[0] + (double)c->page_size * (double)s[2] >= 0x1p36 ||
              (double)c->pages * (double)w[0] + (double)c->page_size * (double)w[2] >= 0x1p34;
    }
    const View caches[] = {cache4_view(c, false, false), cache4_view(c, true, false), cache4_view(c, false, true), cache4_view(c, true, true)};
    return attend(who, p, caches, 4, Call{q, q_token, q_head, heads, tokens, starts, lengths, table, table_width, table_stride, requests,
                                          window, sinks, scale, out, out_token, out_head, workspace, workspace_bytes, bf16 != 0, true, far}, stream);
}

}  // extern "C"
