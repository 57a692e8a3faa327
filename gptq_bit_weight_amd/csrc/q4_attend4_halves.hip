// Attention over a cache held in 4 bits for chunks so long that its keys and values are brought
// into binary16 once, in the call's workspace, and not by every workgroup: 128 rows' workgroups each
// unpack all that they see.
//
// q4_attend4_unpack_kernel: the rows that the call's tokens see, request by request, as a
// cache of binary16 with one page a request. Bound: memory, dim / 2 + 4 dim / group bytes read
// and 2 dim written a row, and the latencies of one small launch: lengths, table, codes (8192 keys and values of 8
// heads of 128, 10 MB to 34: 16 us; 64 rows a workgroup 19, 32 rows 21).
#include "q4_attend_tiles_kernel.h"

#include "q4_ops.h"

namespace q4 {

hipError_t launch_attend_tiles(const q4attend::Args& p, int grid, bool bf16, bool pages_of_16, hipStream_t stream);

}  // namespace q4

namespace {

using namespace q4cache4;

constexpr int UT = 256, UR = 128, kEach = 4;   // lanes of a workgroup, its rows, pieces that a lane has under way

struct Unpack {
    uint16_t* to;                  // keys [request][head][rows][dim], then values
    int* table;                    // [request]: the request's page
    int rows, blocks, pieces;      // rows of a page, workgroups' parts of it, pieces of 8 values of a row
    q4::FastDiv div_pieces;
};

__global__ __launch_bounds__(UT) void q4_attend4_unpack_kernel(Args p, Unpack u)
{
    int at = (int)blockIdx.x;
    const int block = at % u.blocks;
    at /= u.blocks;
    const int side = at % (2 * p.KV), b = at / (2 * p.KV), head = side >> 1;
    const bool values = side & 1;
    if (block == 0 && side == 0 && threadIdx.x == 0) u.table[b] = b;
    const Request r = request(p, b);
    if (r.n == 0) return;
    // (the blocks of 16 rows that the kernel reads: the sinks', and from the first visible key's on. What no
    // token sees in them holds that key's row: its own page may be another request's, or none)
    const int row0 = UR * block, last = max(r.len - 1, 0);
    const int lo = p.window ? min(max(r.len - r.n - p.window + 1, 0), last) : 0;
    const int sink_rows = (p.sinks + 15) & ~15, window_row0 = lo & ~15;
    if (row0 > last || (row0 + UR <= window_row0 && row0 >= sink_rows)) return;
    const Side& c = values ? p.v4 : p.k4;
    uint16_t* to = u.to + (((values ? (long long)p.B : 0) + b) * p.KV + head) * ((long long)u.rows * p.dim);
    const int total = UR * u.pieces;
    for (int base = (int)threadIdx.x; base < total; base += kEach * UT) {
        uint32_t code[kEach], scale[kEach];
        int row[kEach], piece[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = min(base + e * UT, total - 1);
            const int x = (int)q4::fast_div((uint32_t)i, u.div_pieces);
            piece[e] = i - x * u.pieces;
            row[e] = row0 + x;
            const int key = min(row[e] < p.sinks ? row[e] : max(row[e], lo), last), slot = (int)q4::fast_div((uint32_t)key, p.div_page);
            const long long page = min((uint32_t)p.table[(long long)b * p.table_stride + slot], (uint32_t)p.pages - 1u);
            const long long in = key - slot * p.page_size;
            code[e] = *reinterpret_cast<const uint32_t*>(c.at + head * c.head + page * c.page + in * c.row + 4 * piece[e]);
            scale[e] = *reinterpret_cast<const uint32_t*>(c.scale + head * c.scale_head + page * c.scale_page + in * c.scale_row +
                                                          4 * (8 * piece[e] >> p.group_shift));
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (base + e * UT < total && row[e] <= last && (row[e] < sink_rows || row[e] >= window_row0))
                *reinterpret_cast<u4*>(to + (long long)row[e] * p.dim + 8 * piece[e]) =
                    own_order(values8(code[e], low_half(scale[e]), high_half(scale[e]), magic()));
    }
}

constexpr size_t table_bytes(int requests) { return ((size_t)requests * sizeof(int) + 15) / 16 * 16; }
long long rows_of(int max_len) { return ((long long)max_len + UR - 1) / UR * UR; }

}  // namespace

namespace q4 {

size_t attend4_halves_bytes(int requests, int kv_heads, int max_len, int dim)
{
    const double bytes = 4. * requests * kv_heads * (double)rows_of(max_len) * dim;
    if (bytes > (double)(1 << 30) || (double)requests * rows_of(max_len) > 0x7fffffff) return 0;
    return table_bytes(requests) + (size_t)bytes;
}

hipError_t launch_attend4_halves(q4attend::Args p, int grid, bool bf16, char* scratch, hipStream_t stream)
{
    if (p.dim < 32 || p.dim > 256 || p.dim % 32 || grid < 1 || p.workers < 1) return hipErrorInvalidValue;
    Unpack u = {};
    u.table = reinterpret_cast<int*>(scratch);
    u.to = reinterpret_cast<uint16_t*>(scratch + table_bytes(p.B));
    u.rows = (int)rows_of(p.max_len);
    u.blocks = u.rows / UR;
    u.pieces = p.dim / 8;
    u.div_pieces = make_fastdiv((uint32_t)u.pieces);
    hipLaunchKernelGGL(q4_attend4_unpack_kernel, dim3((unsigned)(u.blocks * 2 * p.KV * p.B)), dim3(UT), 0, stream, p, u);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const long long head = (long long)u.rows * p.dim;
    p.k = u.to;
    p.v = u.to + p.B * p.KV * head;
    p.ks0 = p.vs0 = p.KV * head;
    p.ks1 = p.vs1 = head;
    p.ks2 = p.vs2 = p.dim * 2;
    p.table = u.table;
    p.table_stride = 1;
    p.page_size = u.rows;
    p.pages = p.B;
    p.div_page = make_fastdiv((uint32_t)u.rows);
    if (!bf16) return launch_attend_tiles(p, grid, false, true, stream);
    if (p.sinks) {
        if (p.dim <= 64) return launch_halves<64, true>(p, grid, stream);
        if (p.dim <= 128) return launch_halves<128, true>(p, grid, stream);
        return launch_halves<256, true>(p, grid, stream);
    }
    if (p.dim <= 64) return launch_halves<64, false>(p, grid, stream);
    if (p.dim <= 128) return launch_halves<128, false>(p, grid, stream);
    return launch_halves<256, false>(p, grid, stream);
}

}  // namespace q4
