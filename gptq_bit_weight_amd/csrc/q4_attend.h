// Shared parts of the kernels that attend over a paged cache.
//
// A request has `n` new tokens, the last of its `len` cached ones: token i of
// them sits at position len - n + i and sees the keys up to its own, at most
// `window` of them when a window is set. The heads of a group share their keys
// and values, so a tile's rows are the pairs (token, head of the group) of one
// request and one cached head, token-major.
//
// Both kernels compute transposed products, S^T = K Q^T and O^T = V^T P^T: a
// lane of the matrix instructions then holds one row (a token and head) and
// some of its keys, so the softmax needs no exchange but the row maximum's
// among the few lanes of a row, and P^T leaves the first product's result
// registers in the order in which the second product takes them, without
// passing through memory. V^T comes from the row-major V tile in LDS by
// transposing reads (ds_read_b64_tr_b16: sixteen lanes read four rows of
// sixteen values and receive four values of one column each).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "q4_device.h"
#include "q4_fastdiv.h"
#include "q4_ops.h"

namespace q4attend {

using namespace q4dev;

// Row tiles whose keys were split: where their rows and partial results are.
struct Join {
    int start, row0, rows, head, slot, parts, pos0;
};
constexpr int kMaxJoins = 1024;         // (at most one for each workgroup that work is split for)
constexpr int kJoinGroups = 32;
struct JoinList {
    uint32_t count, done, pad[30];
    struct { uint32_t done, pad[31]; } group[kJoinGroups];
    Join item[kMaxJoins];
};

// Keys or values of a cache held in 4 bits: codes and scales, strides in bytes.
struct Side {
    const char *at, *scale;
    long long page, head, scale_page, scale_head;
    int row, scale_row;
};

struct Args {
    const uint16_t* q;
    uint16_t* out;
    const uint16_t *k, *v;
    const int *starts, *lengths, *table;
    long long q_t, q_h, o_t, o_h;          // token and head strides, values
    long long ks0, ks1, vs0, vs1;          // page and head strides, values
    int ks2, vs2;                          // row strides, bytes
    int T, B, KV, g;                       // tokens, requests, cached heads, heads of a group
    int dim, chunks;                       // values of a head and its 16-byte pieces
    int pages, page_size, table_stride, max_len, window;
    float scale;                           // on the scores, times log2 e; positive
    uint32_t q_and, q_xor;                 // on two of q's values: a scale of 0 clears them, a negative one turns them
    int store8;                            // 8-byte stores reach every output row
    float* slots;                          // partial results
    uint32_t* counters;                    // few rows: arrivals
    JoinList* joins;                       // many rows
    int workers, least;                    // workgroups, and least tiles of one
    int unsplit;                           // many rows: no row tile has more than `least` tiles
    q4::FastDiv div_g, div_page;           // by heads of a group; by rows of a page (or 16-row blocks of one)
    // (last, as not all kernels read them)
    int sinks;                             // none without a window
    Side k4, v4;                           // 4 bits, in place of k, v and their strides
    int group_shift;                       // log2 of the values that share a scale
};

constexpr float kLow = -3.4028234663852886e38f;   // running maximum of a row that has seen no key (the lowest finite value, lifted or not)

// A row's running maximum is held less this many powers of two, so that the weights
// of binary16 lie in the upper part of its range: unlifted, those below 2^-25 of the
// largest vanish when they are rounded for the second product and stay in the sum
// (12000 keys of weight 2^-25.5 beside one of 1 are 2^-12 of the result). Up to 2^15 goes in;
// `slack` is the log2 of what a weight may already pass 1 by. (bfloat16 has fp32's range.)
template <bool BF>
constexpr float lift(float slack) { return BF ? 0.f : 15.f - slack; }

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s4v lds_s4;

// 16 bytes a lane from memory straight into LDS: lane l's land at dst + 16 l,
// the next load's 1 KiB further on (dst is wave-uniform, as is the base).
// Written in assembly, with no register result, because the compiler cannot
// tell which LDS a transposing read touches and would wait for every load under
// way before each; the kernels count them out with wait_loads. (s_nop: five
// wait states between a vector instruction's write of the base's SGPRs and its
// use, one after a write of m0.)
template <int N>
__device__ __forceinline__ void dma(const char* base, const uint32_t (&off)[N], uint32_t dst)
{
    static_assert(N == 1 || N == 2 || N == 4, "loads of one block");
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    if constexpr (N == 1)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off[0]), "s"(b), "s"(dst) : "memory");
    else if constexpr (N == 2)
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %2\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     ::"v"(off[0]), "v"(off[1]), "s"(b), "s"(dst) : "memory", "scc");
    else
        asm volatile("s_mov_b32 m0, %5\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %4\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %4\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %4\n\t"
                     "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %4"
                     ::"v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(b), "s"(dst) : "memory", "scc");
}

// 4 bytes a lane from memory straight into LDS: lane l's land at dst + 4 l.
__device__ __forceinline__ void dma_words(const char* base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(reinterpret_cast<uint64_t>(base)), "s"(dst) : "memory");
}
__device__ __forceinline__ void dma_words_lane(const char* src, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory");
}

// A weight of zero does not keep a value that is not finite out of a sum. Where a
// tile of keys is not wholly visible to a tile's rows, the kernels therefore look
// for such values, and multiply key by key if there are any: `lone` leaves one of
// a fragment's eight keys, whose products only rows that see it take.
template <bool BF>
__device__ __forceinline__ bool not_finite(u2 v)
{
    constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
    bool r = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) r |= ((v[i] & E) == E) | ((v[i] >> 16 & E) == E);
    return r;
}
__device__ __forceinline__ u4 lone(u2 a0, u2 a1, int key, bool mine)
{
    u4 a = u4{a0[0], a0[1], a1[0], a1[1]};
    const uint32_t keep = key & 1 ? 0xffff0000u : 0xffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = mine && i == key >> 1 ? a[i] & keep : 0u;
    return a;
}

// A head's row lies in LDS as 16-byte chunks, chunk c of row r at place
// c ^ spread<D>(r) of the row: 16 rows' chunk c (a product's operand read) and the
// 32-byte pieces of 8 or 16 rows (a transposing read) then fall on all banks evenly.
template <int D>
__device__ __forceinline__ int spread(int row)
{
    if constexpr (D == 64) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    else return ((row & 3) << 2) | ((row >> 2) & 3);
}

__device__ __forceinline__ u2 read_tr(const char* p)
{
    return bitcast<u2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p));
}

// What this wave has read from LDS is in registers, what it wrote is there.
__device__ __forceinline__ void wait_lds()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (BF) return pack_bf16(a, b);
    else return bitcast<uint32_t>(__builtin_convertvector(ff2{a, b}, h2));
}

// Maximum over the lanes l, l ^ 32 (and l ^ 16).
__device__ __forceinline__ float max_halves(float v)
{
    const uint32_t u = bitcast<uint32_t>(v);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(bitcast<float>((uint32_t)r[0]), bitcast<float>((uint32_t)r[1]));
}
__device__ __forceinline__ float max_quarters(float v)
{
    const float h = max_halves(v);
    const uint32_t u = bitcast<uint32_t>(h);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(bitcast<float>((uint32_t)r[0]), bitcast<float>((uint32_t)r[1]));
}
__device__ __forceinline__ float sum_halves(float v)
{
    const uint32_t u = bitcast<uint32_t>(v);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return bitcast<float>((uint32_t)r[0]) + bitcast<float>((uint32_t)r[1]);
}
__device__ __forceinline__ float sum_quarters(float v)
{
    const float h = sum_halves(v);
    const uint32_t u = bitcast<uint32_t>(h);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return bitcast<float>((uint32_t)r[0]) + bitcast<float>((uint32_t)r[1]);
}

// A request's tokens and lengths, held inside what the arguments' sizes allow
// whatever the arrays say: no access leaves q, the output or the table.
struct Request {
    int start, n, len;
};
__device__ __forceinline__ Request request(const Args& p, int b)
{
    Request r;
    r.start = min(max(p.starts[b], 0), p.T);
    r.n = min(max(p.starts[b + 1] - r.start, 0), p.T - r.start);
    r.len = min(max(p.lengths[b], 0), p.max_len);
    return r;
}

// The same of lane `b`'s request.
__device__ __forceinline__ Request request_of_lane(const Request& r, int b)
{
    return Request{__builtin_amdgcn_readlane(r.start, b), __builtin_amdgcn_readlane(r.n, b), __builtin_amdgcn_readlane(r.len, b)};
}

// What a row's sums are multiplied by for its output. A sum of zero: a row that sees no
// key (its position is negative) gives zeros; one that does has scores of -inf
// only, which have no softmax.
__device__ __forceinline__ float over_sum(float sum, int pos)
{
    return sum != 0.f ? 1.f / sum : pos < 0 ? 0.f : __builtin_nanf("");
}
__device__ __forceinline__ f4 output_of(f4 v, float sum, float inv)
{
    // (what a row that sees no key has summed may not be finite)
    return sum == 0.f ? f4{inv, inv, inv, inv} : v * inv;
}

// The kernel's arguments (Args is its only one), read anew where this stands: what
// rare parts of a loop take from them does not stay in registers across it.
__device__ __forceinline__ const Args& args_again()
{
    auto p = (const __attribute__((address_space(4))) Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Args*)p;
}
// A value whose uses are not computed ahead of here.
__device__ __forceinline__ int here(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// Four values of an output row.
template <bool BF>
__device__ __forceinline__ void store_row4(uint16_t* o, f4 v, int left, int store8)
{
    if (store8 && left >= 4) {
        *reinterpret_cast<u2*>(o) = u2{pack2<BF>(v[0], v[1]), pack2<BF>(v[2], v[3])};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) o[e] = f32_to_act<BF>(v[e]);
    }
}

}  // namespace q4attend
