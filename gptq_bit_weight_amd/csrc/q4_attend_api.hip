// C ABI of attention over a paged cache: argument checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "q4_attend.h"

namespace q4 {

hipError_t launch_attend_rows(const q4attend::Args& p, bool bf16, bool pages_of_16, hipStream_t stream);

hipError_t launch_attend_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream);

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

}  // namespace
}  // namespace q4

extern "C" {

size_t q4_attend_workspace(const q4_cache* c, int heads)
{
    int dev = -1, cu = 0;
    if (q4::check_attend(c, heads, "q4_attend_workspace") != Q4_OK || q4::device_info(&dev, &cu) != Q4_OK) return 0;
    const size_t rows = q4::rows_bytes(c->dim, cu), tiles = q4::tiles_bytes(c->dim, cu);
    return rows > tiles ? rows : tiles;
}

q4_status q4_attend(const q4_cache* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                    const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                    int64_t table_stride, int requests, int window, float scale, uint16_t* out, int64_t out_token,
                    int64_t out_head, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    using namespace q4;
    const char* who = "q4_attend";
    if (q4_status st = check_attend(c, heads, who); st != Q4_OK) return st;
    if (tokens < 0 || requests < 0 || window < 0)
        return fail(Q4_ERR_INVALID_ARG, "%s: %d tokens, %d requests, window %d", who, tokens, requests, window);
    if (!std::isfinite(scale)) return fail(Q4_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (tokens == 0 || requests == 0) return Q4_OK;
    if (!q || !starts || !lengths || !table || !out) return fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    if (table_width < 1 || table_stride < table_width || table_stride > 0x7fffffff)
        return fail(Q4_ERR_INVALID_ARG, "%s: a table of %d pages a request, %lld apart", who, table_width, (long long)table_stride);
    const int64_t strides[] = {q_token, q_head, c->k_stride[0], c->k_stride[1], c->k_stride[2], c->v_stride[0], c->v_stride[1], c->v_stride[2]};
    for (int64_t s : strides)
        if (s < 0 || s % 8) return fail(Q4_ERR_UNSUPPORTED, "%s: strides of q and the cache must be multiples of 8 values", who);
    if (!at16(q) || !at16(c->k) || !at16(c->v) || (reinterpret_cast<uintptr_t>(out) & 1))
        return fail(Q4_ERR_UNSUPPORTED, "%s: q and the cache must be 16-byte aligned", who);
    if (c->k_stride[2] > (1 << 25) || c->v_stride[2] > (1 << 25))
        return fail(Q4_ERR_UNSUPPORTED, "%s: rows of a page more than 2^25 values apart", who);
    const int g = heads / c->kv_heads;
    if ((long long)tokens * g > (1 << 30) || (long long)heads * c->dim > (1 << 30))
        return fail(Q4_ERR_UNSUPPORTED, "%s: %d tokens of %d heads", who, tokens, heads);
    // (row tiles are stored while others still read)
    const View to = head_view(out, out_token, out_head, tokens, heads, c->dim);
    if (meet(to, head_view(q, q_token, q_head, tokens, heads, c->dim))) return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps q", who);
    if (meet(to, cache_view(c, false)) || meet(to, cache_view(c, true)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps the cache", who);
    if (meet(to, flat_view(starts, ((int64_t)requests + 1) * 4)) || meet(to, flat_view(lengths, (int64_t)requests * 4)) ||
        meet(to, View{table, (int64_t)table_width * 4, {{requests, table_stride * 4}, {1, 0}, {1, 0}}}))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps starts, lengths or table", who);
    int dev = -1, cu = 0;
    if (q4_status st = device_info(&dev, &cu); st != Q4_OK) return st;

    q4attend::Args p = {};
    p.q = q;
    p.out = out;
    p.k = static_cast<const uint16_t*>(c->k);
    p.v = static_cast<const uint16_t*>(c->v);
    p.starts = starts;
    p.lengths = lengths;
    p.table = table;
    p.q_t = q_token;
    p.q_h = q_head;
    p.o_t = out_token;
    p.o_h = out_head;
    p.ks0 = c->k_stride[0];
    p.ks1 = c->k_stride[1];
    p.ks2 = (int)c->k_stride[2] * 2;
    p.vs0 = c->v_stride[0];
    p.vs1 = c->v_stride[1];
    p.vs2 = (int)c->v_stride[2] * 2;
    p.T = tokens;
    p.B = requests;
    p.KV = c->kv_heads;
    p.g = g;
    p.dim = c->dim;
    p.chunks = c->dim / 8;
    p.pages = c->pages;
    p.page_size = c->page_size;
    p.table_stride = (int)table_stride;
    const long long rows = (long long)table_width * c->page_size;
    p.max_len = (int)(rows < (1 << 30) ? rows : (1 << 30));
    // (a window that no key can lie outside is none; the kernels' 32-bit positions less a
    // window then stay in range)
    if (window >= p.max_len) window = 0;
    p.window = window;
    // (a negative scale turns q's signs, a scale of zero clears q)
    p.scale = scale == 0.f ? 1.f : std::fabs(scale) * 1.4426950408889634f;
    p.q_and = scale == 0.f ? 0u : ~0u;
    p.q_xor = scale < 0.f ? 0x80008000u : 0u;
    p.store8 = (reinterpret_cast<uintptr_t>(out) % 8 == 0) && out_token % 4 == 0 && out_head % 4 == 0;
    p.div_g = make_fastdiv((uint32_t)g);
    p.div_page = make_fastdiv((uint32_t)c->page_size);
    const bool bf16 = c->bf16 != 0, pg = c->page_size % 16 == 0;

    // Few rows a request: the few-row kernel, above the many-row one. (64 x 8
    // rows over 4600 keys: 221 us and 237; 8 x 16 over 3000: 32 and 28; 20 x 32 over
    // 6000: 115 and 102.) By their mean, as the host knows no more: a long chunk beside
    // many single tokens costs more in one call than apart (63 single tokens and a chunk of
    // 512 over 8192 keys: 8 heads over 8, few rows, 450 us, apart 359 and 37; 32 heads over 8,
    // many rows, 546 us, apart 360 and 88).
    const long long mean_rows = ((long long)tokens * g + requests - 1) / requests;
    const bool many = mean_rows > 12;
    const int tile = many ? kTileRows : kFewRows;
    const long long row_tiles = (long long)tokens * g / tile + requests;
    if (row_tiles * c->kv_heads * (p.max_len / 32 + 2) >= (1LL << 31))
        return fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^31 tiles of keys", who);
    p.workers = many ? tile_target(cu) : cu;
    p.least = many ? kTileLeast : kFewLeast;
    if (many) {
        const int keys = c->dim > 128 ? 32 : 64;
        // (a row tile's tokens see window - 1 keys before the first's own)
        const long long seen = window ? (long long)window + (kTileRows + g - 1) / g : p.max_len;
        const long long most = std::min<long long>(seen, p.max_len) / keys + 2;
        const bool enough = (long long)tokens * g / kTileRows * c->kv_heads >= tile_target(cu);
        if (window && most * keys <= kWholeKeys && enough) p.least = (int)most;
        p.unsplit = most <= p.least;
    }
    const size_t need = many ? tiles_bytes(c->dim, cu) : rows_bytes(c->dim, cu);
    if (!workspace || workspace_bytes < need || !at16(workspace))
        return fail(Q4_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes on a 16-byte boundary (q4_attend_workspace)", who, need);
    p.counters = static_cast<uint32_t*>(workspace);
    p.joins = reinterpret_cast<q4attend::JoinList*>(static_cast<char*>(workspace) + kListAt);
    p.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
    // (most units there can be: a whole one each share of the work, a partial one each row tile and head)
    hipError_t e = many ? launch_attend_tiles(p, (int)(row_tiles * c->kv_heads + p.workers), bf16, pg, stream)
                        : launch_attend_rows(p, bf16, pg, stream);
    return e == hipSuccess ? Q4_OK : fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // extern "C"
