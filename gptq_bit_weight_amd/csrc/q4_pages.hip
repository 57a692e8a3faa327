// The pages of a cache: copies of them, and which request's tokens they hold
// (allotted, forked, freed and compacted without the host knowing any of it).
//
// Bound. Copies: memory, twice the pages' bytes. The bookkeeping: the launch and a
// few latencies. It needs an order (the lowest free page goes first, requests are
// served in theirs), so one workgroup plans, with prefix sums over its 1024 lanes, and
// what can go in parallel (page copies, table rows) is a second launch that reads the plan.
//
// A copy goes by pieces of 16 KiB, each read whole before it is written: 64 bytes a lane
// under way, 128 KiB a CU. Stores pass the caches by (nobody reads a page next): 940 pages
// of 256 KiB in 80 us, 6.1 TB/s read and written, against 99 with ordinary stores.
#include <hip/hip_runtime.h>

#include "q4_device.h"
#include "q4_fastdiv.h"
#include "q4_ops.h"
#include "q4_turn.h"

namespace {

using namespace q4dev;

// ---------------------------------------------------------------- copies ---

constexpr int CT = 256, kEach = 4;        // lanes of a workgroup, elements of a lane in a piece

// A plane's part of a page: `count` elements of `width` bytes in runs of `run` that
// lie contiguously, `rows` of them a head.
struct CopyPlane {
    char* at;
    long long page, head, row;
    int width, count, pieces, whole;      // whole: one run
    q4::FastDiv div_run, div_rows;
    int run, rows;
};

struct CopyArgs {
    CopyPlane plane[4];
    int planes, pieces, pages, n;
    q4::FastDiv div_pieces;
    const void *src, *dst;
    int src64, dst64;
    const int* count;                     // pairs there are, on the device (NULL: n)
};

template <class T>
__device__ __forceinline__ void copy_piece(const CopyPlane& c, const char* from, char* to, int first)
{
    const int i0 = first + (int)threadIdx.x;
    T v[kEach];
    if (c.whole && first + kEach * CT <= c.count) {
        const T* a = reinterpret_cast<const T*>(from) + i0;
        T* b = reinterpret_cast<T*>(to) + i0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) v[e] = a[e * CT];
#pragma unroll
        for (int e = 0; e < kEach; ++e) __builtin_nontemporal_store(v[e], b + e * CT);
        return;
    }
    long long off[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = min(i0 + e * CT, c.count - 1);
        const int run = (int)q4::fast_div((uint32_t)i, c.div_run), head = (int)q4::fast_div((uint32_t)run, c.div_rows);
        off[e] = head * c.head + (run - head * c.rows) * c.row + (long long)(i - run * c.run) * (int)sizeof(T);
        v[e] = *reinterpret_cast<const T*>(from + off[e]);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        if (i0 + e * CT < c.count) *reinterpret_cast<T*>(to + off[e]) = v[e];
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Piece `piece` of page s to page d. (The planes are read from the kernel's arguments, of which
// CopyArgs is the first, where they lie: a parameter that is indexed is copied to memory of each lane's own.)
__device__ __forceinline__ void copy_piece_of(int s, int d, int piece)
{
    auto p = (const __attribute__((address_space(4))) CopyArgs*)__builtin_amdgcn_kernarg_segment_ptr();
    int x = 0;
    while (piece >= p->plane[x].pieces) piece -= p->plane[x++].pieces;
    const CopyPlane& c = *(const CopyPlane*)&p->plane[x];
    const char* from = c.at + s * c.page;
    char* to = c.at + d * c.page;
    const int first = piece * CT * kEach;
    if (c.width == 16) copy_piece<u4>(c, from, to, first);
    else if (c.width == 4) copy_piece<uint32_t>(c, from, to, first);
    else if (c.width == 2) copy_piece<uint16_t>(c, from, to, first);
    else copy_piece<uint8_t>(c, from, to, first);
}

__device__ __forceinline__ void copy_pages(const CopyArgs& p, int n)
{
    // (the host keeps n pieces below 2^31)
    const uint32_t total = (uint32_t)uniform(n) * (uint32_t)p.pieces;
    for (uint32_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int pair = (int)q4::fast_div(w, p.div_pieces);
        const long long s = index_at(p.src, p.src64, pair), d = index_at(p.dst, p.dst64, pair);
        if (s < 0 || s >= p.pages || d < 0 || d >= p.pages || s == d) continue;
        copy_piece_of(uniform((int)s), uniform((int)d), (int)w - pair * p.pieces);
    }
}

__global__ __launch_bounds__(CT) void q4_copy_pages_kernel(CopyArgs p) { copy_pages(p, p.n); }

// ----------------------------------------------------------- bookkeeping ---

constexpr int PT = 1024;                  // lanes of the planning workgroup
constexpr int kHeader = 16;               // ints of the workspace before its lists

struct Books {
    int *table, *lengths, *counts, *work, *list_a, *list_b;
    int R, W, P, ps;
    q4::FastDiv div_ps;
};

__device__ __forceinline__ int pages_of(const Books& b, int length) { return (int)q4::fast_div((uint32_t)(length + b.ps - 1), b.div_ps); }
// A request's length, and the entries that it holds, whatever the arrays say.
__device__ __forceinline__ int length_of(const Books& b, int r) { return min(max(b.lengths[r], 0), b.W * b.ps); }

// Sum over the workgroup's lanes before this one, and of all; every lane calls it.
__device__ __forceinline__ int sum_before(int v, int* lds, int& all)
{
    const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < PT / 64; ++w) {
        const int x = lds[w];
        before += w < wave ? x : 0;
        all += x;
    }
    __syncthreads();
    return before + s - v;
}

// The lowest free pages, up to `want` of them, in list_b; returns how many there are.
__device__ int free_pages(const Books& b, int want, int* lds)
{
    int found = 0;
    for (int p0 = 0; p0 < b.P && found < want; p0 += 4 * PT) {
        int c[4], mine = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = p0 + 4 * (int)threadIdx.x + e;
            c[e] = p < b.P ? b.counts[p] : 1;
            mine += c[e] <= 0;
        }
        int all;
        int at = found + sum_before(mine, lds, all);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c[e] <= 0) {
                if (at < want) b.list_b[at] = p0 + 4 * (int)threadIdx.x + e;
                ++at;
            }
        found += all;
    }
    __syncthreads();
    return min(found, want);
}

// Allots pages for the new tokens of every request, and says where they go. Tokens and
// pages of a request with many are the whole workgroup's work, few the lane's.
constexpr int kFew = 4;

__global__ __launch_bounds__(PT) void q4_pages_extend_kernel(Books b, const int* starts, int T, int* slots)
{
    __shared__ int lds[PT / 64], many[PT], s_many;
    for (int t = threadIdx.x; t < T; t += PT) slots[t] = -1;
    auto tokens_of = [&](int r, int& start) {
        start = min(max(starts[r], 0), T);
        return min(max(starts[r + 1] - start, 0), T - start);
    };
    // pages that each request needs, counted before its own (-1: more than its table holds)
    int total = 0;
    for (int r0 = 0; r0 < b.R; r0 += PT) {
        const int r = r0 + (int)threadIdx.x;
        int need = 0;
        bool fits = true;
        if (r < b.R) {
            int start;
            const int n = tokens_of(r, start), len = length_of(b, r);
            fits = n <= b.W * b.ps - len;
            if (fits) need = pages_of(b, len + n) - pages_of(b, len);
        }
        int all;
        const int at = total + sum_before(need, lds, all);
        if (r < b.R) b.list_a[r] = fits ? at : -1;
        total += all;
    }
    const int have = free_pages(b, min(total, b.P), lds);
    for (int r0 = 0; r0 < b.R; r0 += PT) {
        const int r = r0 + (int)threadIdx.x;
        if (threadIdx.x == 0) s_many = 0;
        __syncthreads();
        auto give = [&](int r, int lane, int lanes, bool tokens) {
            int start;
            const int n = tokens_of(r, start), len = length_of(b, r), at = b.list_a[r], first = pages_of(b, len);
            int* row = b.table + (long long)r * b.W;
            if (!tokens) {
                for (int e = lane; e < pages_of(b, len + n) - first; e += lanes) {
                    const int page = b.list_b[at + e];
                    row[first + e] = page;
                    b.counts[page] = 1;
                }
            } else {
                for (int i = lane; i < n; i += lanes) {
                    const int e = (int)q4::fast_div((uint32_t)(len + i), b.div_ps), page = row[e];
                    if (page >= 0 && page < b.P) slots[start + i] = page * b.ps + (len + i - e * b.ps);
                }
            }
            return len + n;
        };
        bool mine = false;
        if (r < b.R) {
            int start;
            const int n = tokens_of(r, start), len = length_of(b, r), at = b.list_a[r];
            const int need = at < 0 ? 0 : pages_of(b, len + n) - pages_of(b, len);      // (-1: len + n may not fit in an int)
            // (who needs no page does not wait for those who find none)
            const bool served = n > 0 && at >= 0 && (need == 0 || at + need <= have);
            if (served && n > kFew) many[atomicAdd(&s_many, 1)] = r;
            else if (served) {
                give(r, 0, 1, false);
                give(r, 0, 1, true);
                mine = true;
            }
            if (mine) b.lengths[r] = len + n;
        }
        __syncthreads();
        const int count = s_many;
        for (int x = 0; x < count; ++x) {
            give(many[x], (int)threadIdx.x, PT, false);
            __syncthreads();
            const int len = give(many[x], (int)threadIdx.x, PT, true);
            __syncthreads();
            if (threadIdx.x == 0) b.lengths[many[x]] = len;
        }
        __syncthreads();
    }
}

// Which pairs of a fork can be done (done[i]), and the page that the parent's last one,
// where it is not full, is copied to (to[i]; -1: none is needed, -2: the parent holds nothing).
// list_a: the first pair that names a request as its child.
__global__ __launch_bounds__(PT) void q4_pages_fork_kernel(Books b, const void* parents, int parents64, const void* children,
                                                           int children64, int n, int* done, int* to)
{
    __shared__ int lds[PT / 64];
    for (int r = threadIdx.x; r < b.R; r += PT)
        __hip_atomic_store(&b.list_a[r], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    auto pair = [&](int i, int& par, int& chi) {
        const long long x = i < n ? index_at(parents, parents64, i) : -1, y = i < n ? index_at(children, children64, i) : -1;
        par = (int)x;
        chi = (int)y;
        return x >= 0 && x < b.R && y >= 0 && y < b.R;
    };
    int par, chi;
    for (int i = threadIdx.x; i < n; i += PT)
        if (pair(i, par, chi)) atomicMin(&b.list_a[chi], i);
    __threadfence_block();
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += PT) {
        const int i = i0 + (int)threadIdx.x;
        bool fine = pair(i, par, chi);
        int len = 0;
        if (fine) {
            fine = __hip_atomic_load(&b.list_a[chi], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == i && b.lengths[chi] == 0;
            len = length_of(b, par);
        }
        const bool tail = fine && len - (int)q4::fast_div((uint32_t)len, b.div_ps) * b.ps != 0;
        int all;
        const int at = total + sum_before(tail, lds, all);
        total += all;
        if (i < n) {
            done[i] = fine;
            to[i] = tail ? at : len ? -1 : -2;
        }
    }
    const int have = free_pages(b, min(total, b.P), lds);
    for (int i = threadIdx.x; i < n; i += PT) {
        const int at = to[i];
        if (at < 0) continue;
        const bool served = at < have;
        done[i] = served;
        to[i] = served ? b.list_b[at] : -1;
    }
}

// The plan's page copies and table rows. The page copied is the parent's last.
__global__ __launch_bounds__(CT) void q4_pages_fork_copy_kernel(CopyArgs p, Books b, const void* parents, int parents64,
                                                                const void* children, int children64, int n, const int* done, const int* to)
{
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        if (!done[i] || to[i] == -2) continue;
        // (a parent that holds tokens is no pair's child: nobody writes its row or length here)
        const int par = (int)index_at(parents, parents64, i), chi = (int)index_at(children, children64, i);
        const int len = length_of(b, par), need = pages_of(b, len), last = to[i] >= 0 ? need - 1 : -1;
        for (int e = threadIdx.x; e < need; e += CT) {
            const int page = b.table[(long long)par * b.W + e];
            b.table[(long long)chi * b.W + e] = e == last ? to[i] : page;
            if (e == last) b.counts[to[i]] = 1;
            else if (page >= 0 && page < b.P) atomicAdd(&b.counts[page], 1);
        }
        if (threadIdx.x == 0) b.lengths[chi] = len;
    }
    const uint32_t total = (uint32_t)n * (uint32_t)p.pieces;
    for (uint32_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int i = (int)q4::fast_div(w, p.div_pieces);
        if (!done[i] || to[i] < 0) continue;
        const int par = (int)index_at(parents, parents64, i);
        const int s = b.table[(long long)par * b.W + pages_of(b, length_of(b, par)) - 1];
        if (s < 0 || s >= b.P) continue;
        copy_piece_of(uniform(s), uniform(to[i]), (int)w - i * p.pieces);
    }
}

// Gives back the pages of requests. (Named twice, one of the two finds the length.)
__global__ __launch_bounds__(CT) void q4_pages_free_kernel(Books b, const void* requests, int wide, int n)
{
    __shared__ int s_len;
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const long long r = index_at(requests, wide, i);
        if (r < 0 || r >= b.R) continue;
        if (threadIdx.x == 0) s_len = min(max(atomicExch(&b.lengths[r], 0), 0), b.W * b.ps);
        __syncthreads();
        const int need = pages_of(b, s_len);
        for (int e = threadIdx.x; e < need; e += CT) {
            const int page = b.table[r * b.W + e];
            if (page >= 0 && page < b.P) atomicSub(&b.counts[page], 1);
            b.table[r * b.W + e] = -1;
        }
        __syncthreads();
    }
}

// Gives back the pages that a token after the last one sees nothing of.
__global__ __launch_bounds__(CT) void q4_pages_trim_kernel(Books b, int window, int sinks)
{
    for (int r = blockIdx.x; r < b.R; r += gridDim.x) {
        const int len = length_of(b, r);
        // keys below `past` lie behind the window
        const int past = (int)max((long long)len - window + 1, 0LL);
        const int from = (int)(((long long)sinks + b.ps - 1) / b.ps), end = min((int)q4::fast_div((uint32_t)past, b.div_ps), b.W);
        for (int e = from + (int)threadIdx.x; e < end; e += CT) {
            const int page = b.table[(long long)r * b.W + e];
            if (page >= 0 && page < b.P) atomicSub(&b.counts[page], 1);
            b.table[(long long)r * b.W + e] = -1;
        }
    }
}

// The moves that leave the pages in use at the front: with U of them, the k-th one from page U on
// goes to the k-th free page below U. to[p]: where page p is afterwards (-1: it was free).
__global__ __launch_bounds__(PT) void q4_pages_compact_kernel(Books b, int* to)
{
    __shared__ int lds[PT / 64];
    int used = 0;
    for (int p = threadIdx.x; p < b.P; p += PT) used += b.counts[p] > 0;
    int U, all;
    sum_before(used, lds, U);
    int holes = 0, moved = 0;
    for (int p0 = 0; p0 < U; p0 += PT) {
        const int p = p0 + (int)threadIdx.x;
        const bool hole = p < U && b.counts[p] <= 0;
        const int at = holes + sum_before(hole, lds, all);
        if (hole) b.list_b[at] = p;
        if (p < U) to[p] = hole ? -1 : p;
        holes += all;
    }
    __syncthreads();
    for (int p0 = U; p0 < b.P; p0 += PT) {
        const int p = p0 + (int)threadIdx.x;
        const int count = p < b.P ? b.counts[p] : 0;
        const int at = moved + sum_before(count > 0, lds, all);
        if (count > 0) {
            const int hole = b.list_b[at];
            b.list_a[at] = p;
            to[p] = hole;
            b.counts[hole] = count;
            b.counts[p] = 0;
        } else if (p < b.P) {
            to[p] = -1;
        }
        moved += all;
    }
    if (threadIdx.x == 0) b.work[0] = moved;
}

__global__ __launch_bounds__(CT) void q4_pages_move_kernel(CopyArgs p, Books b, const int* to)
{
    const int threads = (int)gridDim.x * CT;
    const long long entries = (long long)b.R * b.W;
    for (long long i = (long long)blockIdx.x * CT + threadIdx.x; i < entries; i += threads) {
        const int r = (int)(i / b.W), e = (int)(i - (long long)r * b.W);
        if (e >= pages_of(b, length_of(b, r))) continue;
        const int page = b.table[i];
        if (page >= 0 && page < b.P) b.table[i] = to[page];
    }
    copy_pages(p, b.work[0]);
}

// ------------------------------------------------------------------ host ---

constexpr int kCopyGrid = 2048;

q4_status check_pool(const q4_pool* c, const char* who)
{
    if (!c || c->planes < 1 || c->planes > 4 || c->pages < 1) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null or empty pool", who);
    for (int i = 0; i < c->planes; ++i) {
        const q4_plane& x = c->plane[i];
        if (!x.at || x.heads < 1 || x.rows < 1 || x.bytes < 1 || x.page < 0 || x.head < 0 || x.row < 0)
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: plane %d: %d heads of %d rows of %d bytes", who, i, x.heads, x.rows, x.bytes);
        // (a lane's elements lie up to a piece past the last one: their numbers fit in an int)
        if ((long long)x.heads * x.rows > (1 << 30) / x.bytes)
            return q4::fail(Q4_ERR_UNSUPPORTED, "%s: plane %d: pages of more than 2^30 bytes", who, i);
    }
    return Q4_OK;
}

CopyArgs copy_args(const q4_pool* c)
{
    CopyArgs p = {};
    p.planes = c->planes;
    p.pages = c->pages;
    for (int i = 0; i < c->planes; ++i) {
        const q4_plane& x = c->plane[i];
        long long run = x.bytes, rows = x.rows, heads = x.heads, row = x.row, head = x.head;
        // (dimensions that run on into each other are one)
        if (row == run || rows == 1) {
            run *= rows;
            rows = 1;
            row = 0;
            if (head == run || heads == 1) {
                run *= heads;
                heads = 1;
                head = 0;
            }
        }
        auto whole = [&](long long w) {
            return run % w == 0 && (rows == 1 || row % w == 0) && (heads == 1 || head % w == 0) && x.page % w == 0 &&
                   reinterpret_cast<uintptr_t>(x.at) % (uintptr_t)w == 0;
        };
        CopyPlane& d = p.plane[i];
        d.at = static_cast<char*>(x.at);
        d.page = x.page;
        d.head = head;
        d.row = row;
        d.width = whole(16) ? 16 : whole(4) ? 4 : whole(2) ? 2 : 1;
        d.run = (int)(run / d.width);
        d.rows = (int)rows;
        d.count = (int)(run / d.width * rows * heads);
        d.whole = rows == 1 && heads == 1;
        d.div_run = q4::make_fastdiv((uint32_t)d.run);
        d.div_rows = q4::make_fastdiv((uint32_t)d.rows);
        d.pieces = (d.count + CT * kEach - 1) / (CT * kEach);
        p.pieces += d.pieces;
    }
    p.div_pieces = q4::make_fastdiv((uint32_t)p.pieces);
    return p;
}

q4::View plane_view(const q4_pool* c, int i)
{
    const q4_plane& x = c->plane[i];
    return q4::View{x.at, x.bytes, {{c->pages, x.page}, {x.heads, x.head}, {x.rows, x.row}}};
}

q4_status check_pages(const q4_pages* b, const char* who)
{
    if (!b || !b->table || !b->lengths || !b->counts || !b->work) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    if (b->requests < 1 || b->width < 1 || b->pages < 1 || b->page_size < 1)
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: %d requests of %d pages, %d pages of %d rows", who, b->requests, b->width, b->pages, b->page_size);
    if ((long long)b->requests * b->width > (1 << 30) || (long long)b->width * b->page_size > (1 << 30) ||
        (long long)b->pages * b->page_size > 0x7fffffffLL)
        return q4::fail(Q4_ERR_UNSUPPORTED, "%s: %d requests of %d pages, %d pages of %d rows", who, b->requests, b->width, b->pages, b->page_size);
    return Q4_OK;
}

// The books' arrays, all of which calls write (work as the scratch).
constexpr int kArrays = 4;
q4::View array_view(const q4_pages* b, int i)
{
    switch (i) {
    case 0: return q4::flat_view(b->table, (int64_t)b->requests * b->width * 4);
    case 1: return q4::flat_view(b->lengths, (int64_t)b->requests * 4);
    case 2: return q4::flat_view(b->counts, (int64_t)b->pages * 4);
    default: return q4::flat_view(b->work, (int64_t)q4_pages_workspace(b->requests, b->pages));
    }
}

// The books lie apart from each other and from the cache (which calls with a pool write).
q4_status check_apart(const q4_pages* b, const q4_pool* pool, const char* who)
{
    for (int i = 0; i < kArrays; ++i) {
        const q4::View v = array_view(b, i);
        for (int j = 0; j < i; ++j)
            if (q4::meet(v, array_view(b, j))) return q4::fail(Q4_ERR_INVALID_ARG, "%s: table, lengths, counts and work overlap", who);
        for (int j = 0; pool && j < pool->planes; ++j)
            if (q4::meet(v, plane_view(pool, j))) return q4::fail(Q4_ERR_INVALID_ARG, "%s: the books overlap the cache", who);
    }
    return Q4_OK;
}

// An index or an output lies apart from the books, the cache and `other`.
q4_status check_apart(const q4::View& v, const char* what, const q4_pages* b, const q4_pool* pool, const q4::View* other, const char* who)
{
    for (int i = 0; i < kArrays; ++i)
        if (q4::meet(v, array_view(b, i))) return q4::fail(Q4_ERR_INVALID_ARG, "%s: %s overlaps the books", who, what);
    for (int i = 0; pool && i < pool->planes; ++i)
        if (q4::meet(v, plane_view(pool, i))) return q4::fail(Q4_ERR_INVALID_ARG, "%s: %s overlaps the cache", who, what);
    return other && q4::meet(v, *other) ? q4::fail(Q4_ERR_INVALID_ARG, "%s: %s overlaps the output", who, what) : Q4_OK;
}

q4::View index_view(const void* p, int bits, int n) { return q4::flat_view(p, (int64_t)n * bits / 8); }

Books books_of(const q4_pages* x)
{
    Books b = {};
    b.table = x->table;
    b.lengths = x->lengths;
    b.counts = x->counts;
    b.work = x->work;
    b.R = x->requests;
    b.W = x->width;
    b.P = x->pages;
    b.ps = x->page_size;
    b.list_a = x->work + kHeader;
    b.list_b = b.list_a + (b.R > b.P ? b.R : b.P);
    b.div_ps = q4::make_fastdiv((uint32_t)b.ps);
    return b;
}

q4_status check_index(const void* p, int bits, int n, const char* who)
{
    if (bits != 32 && bits != 64) return q4::fail(Q4_ERR_INVALID_ARG, "%s: indexes of %d bits", who, bits);
    if (n > (1 << 30)) return q4::fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^30 indexes", who);
    return n > 0 && !p ? q4::fail(Q4_ERR_INVALID_ARG, "%s: null indexes", who) : Q4_OK;
}

q4_status pieces_fit(const CopyArgs& p, long long n, const char* who)
{
    if (n * p.pieces >= (1LL << 31)) return q4::fail(Q4_ERR_UNSUPPORTED, "%s: %lld pages of %d pieces of 16 KiB", who, n, p.pieces);
    return Q4_OK;
}

q4_status launched(const char* who)
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? Q4_OK : q4::fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // namespace

extern "C" {

q4_status q4_copy_pages(const q4_pool* pool, const void* src, int src_bits, const void* dst, int dst_bits, int n, hipStream_t stream)
{
    const char* who = "q4_copy_pages";
    if (q4_status st = check_pool(pool, who); st != Q4_OK) return st;
    if (n < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (q4_status st = check_index(src, src_bits, n, who); st != Q4_OK) return st;
    if (q4_status st = check_index(dst, dst_bits, n, who); st != Q4_OK) return st;
    if (n == 0) return Q4_OK;
    for (int i = 0; i < pool->planes; ++i)
        if (q4::meet(plane_view(pool, i), q4::flat_view(src, (int64_t)n * src_bits / 8)) ||
            q4::meet(plane_view(pool, i), q4::flat_view(dst, (int64_t)n * dst_bits / 8)))
            return q4::fail(Q4_ERR_INVALID_ARG, "%s: the indexes overlap the cache", who);
    CopyArgs p = copy_args(pool);
    if (q4_status st = pieces_fit(p, n, who); st != Q4_OK) return st;
    p.n = n;
    p.src = src;
    p.dst = dst;
    p.src64 = src_bits == 64;
    p.dst64 = dst_bits == 64;
    const long long units = (long long)n * p.pieces;
    hipLaunchKernelGGL(q4_copy_pages_kernel, dim3((unsigned)(units < kCopyGrid ? units : kCopyGrid)), dim3(CT), 0, stream, p);
    return launched(who);
}

size_t q4_pages_workspace(int requests, int pages)
{
    if (requests < 1 || pages < 1) return 0;
    return (kHeader + 2 * (size_t)(requests > pages ? requests : pages)) * sizeof(int32_t);
}

q4_status q4_pages_extend(const q4_pages* pages, const int32_t* starts, int tokens, int32_t* slots, hipStream_t stream)
{
    const char* who = "q4_pages_extend";
    if (q4_status st = check_pages(pages, who); st != Q4_OK) return st;
    if (tokens < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (tokens == 0) return Q4_OK;
    if (tokens > (1 << 30)) return q4::fail(Q4_ERR_UNSUPPORTED, "%s: %d tokens", who, tokens);
    if (!starts || !slots) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    const q4::View to = q4::flat_view(slots, (int64_t)tokens * 4), from = q4::flat_view(starts, ((int64_t)pages->requests + 1) * 4);
    if (q4_status st = check_apart(pages, nullptr, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(to, "slots", pages, nullptr, nullptr, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(from, "starts", pages, nullptr, &to, who); st != Q4_OK) return st;
    hipLaunchKernelGGL(q4_pages_extend_kernel, dim3(1), dim3(PT), 0, stream, books_of(pages), starts, tokens, slots);
    return launched(who);
}

q4_status q4_pages_fork(const q4_pages* pages, const q4_pool* pool, const void* parents, int parent_bits, const void* children,
                        int child_bits, int n, int32_t* done, hipStream_t stream)
{
    const char* who = "q4_pages_fork";
    if (q4_status st = check_pages(pages, who); st != Q4_OK) return st;
    if (q4_status st = check_pool(pool, who); st != Q4_OK) return st;
    if (pool->pages != pages->pages) return q4::fail(Q4_ERR_INVALID_ARG, "%s: %d pages, the pool has %d", who, pages->pages, pool->pages);
    if (n < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (q4_status st = check_index(parents, parent_bits, n, who); st != Q4_OK) return st;
    if (q4_status st = check_index(children, child_bits, n, who); st != Q4_OK) return st;
    if (n == 0) return Q4_OK;
    if (!done) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    const q4::View to = q4::flat_view(done, (int64_t)n * 8);
    if (q4_status st = check_apart(pages, pool, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(to, "done", pages, pool, nullptr, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(index_view(parents, parent_bits, n), "parents", pages, pool, &to, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(index_view(children, child_bits, n), "children", pages, pool, &to, who); st != Q4_OK) return st;
    const CopyArgs p = copy_args(pool);
    if (q4_status st = pieces_fit(p, n, who); st != Q4_OK) return st;
    const Books b = books_of(pages);
    hipLaunchKernelGGL(q4_pages_fork_kernel, dim3(1), dim3(PT), 0, stream, b, parents, parent_bits == 64, children, child_bits == 64, n,
                       done, done + n);
    if (q4_status st = launched(who); st != Q4_OK) return st;
    const long long units = (long long)n * p.pieces;
    hipLaunchKernelGGL(q4_pages_fork_copy_kernel, dim3((unsigned)(units < kCopyGrid ? units : kCopyGrid)), dim3(CT), 0, stream, p, b,
                       parents, parent_bits == 64, children, child_bits == 64, n, done, done + n);
    return launched(who);
}

q4_status q4_pages_free(const q4_pages* pages, const void* requests, int bits, int n, hipStream_t stream)
{
    const char* who = "q4_pages_free";
    if (q4_status st = check_pages(pages, who); st != Q4_OK) return st;
    if (n < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: negative size", who);
    if (q4_status st = check_index(requests, bits, n, who); st != Q4_OK) return st;
    if (n == 0) return Q4_OK;
    if (q4_status st = check_apart(pages, nullptr, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(index_view(requests, bits, n), "requests", pages, nullptr, nullptr, who); st != Q4_OK) return st;
    hipLaunchKernelGGL(q4_pages_free_kernel, dim3(n < kCopyGrid ? n : kCopyGrid), dim3(CT), 0, stream, books_of(pages), requests, bits == 64, n);
    return launched(who);
}

q4_status q4_pages_trim(const q4_pages* pages, int window, int sinks, hipStream_t stream)
{
    const char* who = "q4_pages_trim";
    if (q4_status st = check_pages(pages, who); st != Q4_OK) return st;
    if (window < 1 || sinks < 0) return q4::fail(Q4_ERR_INVALID_ARG, "%s: window %d, %d sinks", who, window, sinks);
    if (q4_status st = check_apart(pages, nullptr, who); st != Q4_OK) return st;
    hipLaunchKernelGGL(q4_pages_trim_kernel, dim3(pages->requests < kCopyGrid ? pages->requests : kCopyGrid), dim3(CT), 0, stream,
                       books_of(pages), window, sinks);
    return launched(who);
}

q4_status q4_pages_compact(const q4_pages* pages, const q4_pool* pool, int32_t* to, hipStream_t stream)
{
    const char* who = "q4_pages_compact";
    if (q4_status st = check_pages(pages, who); st != Q4_OK) return st;
    if (q4_status st = check_pool(pool, who); st != Q4_OK) return st;
    if (pool->pages != pages->pages) return q4::fail(Q4_ERR_INVALID_ARG, "%s: %d pages, the pool has %d", who, pages->pages, pool->pages);
    if (!to) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null pointer", who);
    if (q4_status st = check_apart(pages, pool, who); st != Q4_OK) return st;
    if (q4_status st = check_apart(q4::flat_view(to, (int64_t)pages->pages * 4), "to", pages, pool, nullptr, who); st != Q4_OK) return st;
    CopyArgs p = copy_args(pool);
    if (q4_status st = pieces_fit(p, pool->pages, who); st != Q4_OK) return st;
    const Books b = books_of(pages);
    p.src = b.list_a;
    p.dst = b.list_b;
    hipLaunchKernelGGL(q4_pages_compact_kernel, dim3(1), dim3(PT), 0, stream, b, to);
    if (q4_status st = launched(who); st != Q4_OK) return st;
    const long long units = (long long)pool->pages / 2 * p.pieces + 1, entries = ((long long)b.R * b.W + CT - 1) / CT;
    const long long grid = units > entries ? units : entries;
    hipLaunchKernelGGL(q4_pages_move_kernel, dim3((unsigned)(grid < kCopyGrid ? grid : kCopyGrid)), dim3(CT), 0, stream, p, b, to);
    return launched(who);
}

}  // extern "C"
