// The adapters' bank and the first of a call's two products, c A x.
//
// Few rows (the skinny kernel's M): a workgroup for each (row, value of rank),
// whose four waves share K. It reads rank * K values a row and is bound by them;
// nothing is sorted, since each row reads its own adapter whatever the others do.
//
// Many rows: the rows of one adapter are multiplied together. Each workgroup
// counts the index (the same counting sort in all, in place of a launch of its own;
// with nothing multiplied the launch takes 4 us for 77 rows, 7 for 2048) and takes 32 rows of one adapter, 32 or 64 of
// its values and a share of K. Bound: what one CU can fetch, about 45 GB/s where the
// rows come from beyond its XCD's L2, so the shares of K spread a tile over CUs until
// each has a workgroup; x and A stream through a ring of LDS stages, 64 of
// K each, filled by direct loads of whole 128-byte lines, and the last workgroup of a
// tile to arrive adds the shares in order (K = 4096: 77 rows of 12 adapters of rank 32
// 9.0 us, 2048 rows of 8 of rank 64 20.3 us; one workgroup a tile, operands straight from
// memory: 13.4 and 33). The workgroups also leave the order of the rows for the
// product's launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <memory>
#include <mutex>
#include <new>
#include <vector>

#include "q4_adapters.h"
#include "q4_ops.h"

namespace {

using namespace q4dev;

constexpr int kMaxSlots = 4096;
constexpr int kMaxRank = 1024;

// ---- bank -------------------------------------------------------------------
// A [parts][r][K] -> slot's [parts][rank][K], B [N][r] -> slot's [N / 32][rp / 8][32][8],
// zeros past r and N; null A clears the slot.
__global__ void q4_adapter_reset_kernel(float* scale, int* wild, float c)
{
    *scale = c;
    *wild = 0;
}

template <bool BF>
__global__ void q4_adapter_load_kernel(const uint16_t* A, const uint16_t* B, uint16_t* dA, uint16_t* dB, int* wild, int parts,
                                       int r, int rank, int rp, int K, int N)
{
    const long long na = (long long)parts * rank * K, nb = (N + 31) / 32 * 32ll * rp, step = (long long)gridDim.x * blockDim.x;
    const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    for (long long i = id; i < na; i += step) {
        const long long row = i / K;
        const int p = (int)(row / rank), j = (int)(row % rank);
        dA[i] = A && j < r ? A[((long long)p * r + j) * K + i % K] : (uint16_t)0;
    }
    for (long long i = id; i < nb; i += step) {
        const long long n = i / (32 * rp) * 32 + i / 8 % 32;
        const int j = (int)(i % (32 * rp) / kChunk * 8 + i % 8);
        const uint16_t v = A && n < N && j < r ? B[n * r + j] : (uint16_t)0;
        constexpr uint16_t E = BF ? 0x7f80 : 0x7c00;
        if ((v & E) == E) *wild = 1;       // (any of them)
        dB[i] = v;
    }
}

// ---- few rows ---------------------------------------------------------------
constexpr int DW = 4;      // waves of a workgroup

template <bool BF>
__global__ __launch_bounds__(64 * DW) void q4_adapter_few_kernel(const uint16_t* x, const int* index, const uint16_t* A,
                                                                 const float* scale, float* t, int K, int slots,
                                                                 int rank, int rp, int parts)
{
    __shared__ float part_sum[DW];
    const int m = blockIdx.y, w = blockIdx.x, p = w / rp, j = w - p * rp;
    const int s = index[m];
    if ((unsigned)s >= (unsigned)slots) return;     // (its t is not read)
    const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const bool live = j < rank;
    const uint16_t* xr = x + (size_t)m * K;
    const uint16_t* ar = A + (((size_t)s * parts + p) * rank + (live ? j : 0)) * K;
    float y = 0.f;
    constexpr int U = 4;       // loads of each operand under way
    for (int k0 = 8 * (int)threadIdx.x; live && k0 < K; k0 += U * 512 * DW) {
        u4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * 512 * DW;
            a[u] = k < K ? *reinterpret_cast<const u4*>(ar + k) : u4{0, 0, 0, 0};
            b[u] = k < K ? *reinterpret_cast<const u4*>(xr + k) : u4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y = __builtin_fmaf(act_to_f32<BF>((uint16_t)a[u][e]), act_to_f32<BF>((uint16_t)b[u][e]), y);
                y = __builtin_fmaf(act_to_f32<BF>((uint16_t)(a[u][e] >> 16)), act_to_f32<BF>((uint16_t)(b[u][e] >> 16)), y);
            }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) y += __shfl_xor(y, d);
    if (lane == 0) part_sum[wave] = y;
    __syncthreads();
    if (threadIdx.x == 0) {
        float z = part_sum[0];
#pragma unroll
        for (int v = 1; v < DW; ++v) z += part_sum[v];
        t[((size_t)m * parts + p) * rp + j] = live ? z * scale[s] : 0.f;
    }
}

// ---- many rows --------------------------------------------------------------
constexpr int MW = 4, MT = 64 * MW;    // waves, threads
constexpr int MR = 32;                 // rows of a workgroup
constexpr int RPT = 8;                 // rows of the index that a thread looks at together
constexpr int KC = 64;                 // values of K of a stage: a 16-value step for each wave
constexpr int NS = 6;                  // stages
constexpr int kMaxShares = 8;          // of K
constexpr int kManyGroups = 256;       // workgroups that shares are made for (one a CU; 512: 21.4 us against 20.5
                                       // at 2048 rows, whose sums are then twice as many)

struct ManyArgs {
    const uint16_t* x;
    const int* index;
    const uint16_t* A;
    const float* scale;
    const int* wild;
    AdapterRow* rows;
    uint16_t *hi, *lo;
    float* partial;                    // [tile][columns' block][share][MR][64]
    uint32_t* arrived;                 // [tile][columns' block], zero between calls
    float* up;                         // binary16: [stretch][up_pitch]
    int M, K, slots, rank, rp, parts;
    int per_part, up_pitch;            // columns' blocks of a part (0: of the whole width)
};

// binary16 reaches from 2^-24 to 2^16. c A x whose largest value of a stretch lies outside
// these bounds is stored over a power of two near it, so that the pair of values is never
// off by more than 2^-16 of the largest (2^-25 of 2^-9).
constexpr float kReachLow = 0x1p-9f, kReachHigh = 0x1p15f;

template <bool BF, int NB>
__global__ __launch_bounds__(MT, 2) void q4_adapter_many_kernel(ManyArgs p)
{
    constexpr int MC = 32 * NB;                  // values of a workgroup
    constexpr int STAGE = (MR + MC) * KC * 2;    // bytes
    constexpr int LPW = (MR + MC) / 8 / MW;      // direct loads of a wave a stage, 8 rows each
    extern __shared__ int count[];               // [slots + 1]: rows of each adapter; of none
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE];
    __shared__ int wave_n[RPT * MW], tile_row[MR];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bins = p.slots + 1;
    // The index is gone through twice, RPT rows a thread at a time; the first
    // RPT MT of them stay in registers.
    auto bins_of = [&](int i0, int (&s)[RPT]) {
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
            const int i = i0 + u * MT + tid;
            s[u] = i < p.M ? p.index[i] : 0;
        }
#pragma unroll
        for (int u = 0; u < RPT; ++u)
            s[u] = i0 + u * MT + tid >= p.M ? -1 : (unsigned)s[u] < (unsigned)p.slots ? s[u] : p.slots;
    };
    int bin0[RPT];
    bins_of(0, bin0);
    for (int i = tid; i < bins; i += MT) count[i] = 0;
    __syncthreads();
    auto add = [&](int i0, const int (&bin)[RPT]) {
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
            if (i0 + u * MT >= p.M) continue;
            // one addition for each run of equal neighbours
            const int s = bin[u], before = __shfl_up(s, 1);
            const bool head = lane == 0 || s != before;
            const unsigned long long heads = __ballot(head);
            if (head && s >= 0) {
                const unsigned long long after = lane == 63 ? 0 : heads >> (lane + 1) << (lane + 1);
                atomicAdd(&count[s], (after ? (int)__builtin_ctzll(after) : 64) - lane);
            }
        }
    };
    add(0, bin0);
    for (int i0 = RPT * MT; i0 < p.M; i0 += RPT * MT) {
        int bin[RPT];
        bins_of(i0, bin);
        add(i0, bin);
    }
    __syncthreads();
    // ---- this workgroup's tile: of all bins' tiles of MR rows, the blockIdx.x-th
    // (in every wave, which needs no barrier)
    int slot = -1, first = 0, pos = 0, n_rows = 0;
    {
        int tiles = 0, at = 0;
        for (int b0 = 0; b0 < bins; b0 += 64) {
            const int n = b0 + lane < bins ? count[b0 + lane] : 0;
            int t = (n + MR - 1) / MR, r = n;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int to = __shfl_up(t, d), ro = __shfl_up(r, d);
                if (lane >= d) t += to, r += ro;
            }
            const unsigned long long past = __ballot(tiles + t > (int)blockIdx.x);
            if (past) {
                const int f = (int)__builtin_ctzll(past);
                const int mine = __builtin_amdgcn_readlane(n, f);
                slot = b0 + f;
                first = ((int)blockIdx.x - (tiles + __builtin_amdgcn_readlane(t, f) - (mine + MR - 1) / MR)) * MR;
                pos = at + __builtin_amdgcn_readlane(r, f) - mine + first;
                n_rows = min(MR, mine - first);
                break;
            }
            tiles += __builtin_amdgcn_readlane(t, 63);
            at += __builtin_amdgcn_readlane(r, 63);
        }
    }
    if (slot < 0) return;
    const bool none = slot == p.slots;           // rows without an adapter: only their order
    if (none && (blockIdx.y || blockIdx.z)) return;
    // (asked for here, used much later)
    const float scale = none ? 0.f : p.scale[slot];
    const int wild = none ? 0 : p.wild[slot];
    // ---- its rows: those of the bin ranked first .. first + MR - 1
    int seen = 0;
    auto pick = [&](int i0, const int (&bin)[RPT]) {
        unsigned long long b[RPT];
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
            b[u] = __ballot(bin[u] == slot);
            if (lane == 0) wave_n[u * MW + wave] = (int)__builtin_popcountll(b[u]);
        }
        __syncthreads();
        int before = seen;
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
            if (i0 + u * MT >= p.M) continue;
            int rank = before;
#pragma unroll
            for (int w = 0; w < MW; ++w) {
                if (w < wave) rank += wave_n[u * MW + w];
                before += wave_n[u * MW + w];
            }
            rank += (int)__builtin_popcountll(b[u] & ((1ull << lane) - 1)) - first;
            if (bin[u] == slot && rank >= 0 && rank < MR) tile_row[rank] = i0 + u * MT + tid;
        }
        seen = before;
        __syncthreads();
    };
    pick(0, bin0);
    for (int i0 = RPT * MT; i0 < p.M && seen < first + n_rows; i0 += RPT * MT) {
        int bin[RPT];
        bins_of(i0, bin);
        pick(i0, bin);
    }
    if (blockIdx.y == 0 && blockIdx.z == 0 && tid < n_rows)
        p.rows[pos + tid] = AdapterRow{tile_row[tid], none ? -1 : slot, wild, 0};
    if (none) return;
    // ---- a stage is 128 bytes of each row of x and of A; its 16-byte chunk c lies at
    // place c ^ row % 8, which spreads a product's operand over the banks
    // (a stretch of one part each, or 64 values of the whole width)
    const int width = p.parts * p.rp, of_part = p.per_part ? (int)blockIdx.y / p.per_part : 0;
    const int col0 = p.per_part ? of_part * p.rp + ((int)blockIdx.y - of_part * p.per_part) * kStretch : (int)blockIdx.y * MC;
    const int cols = p.per_part ? (of_part + 1) * p.rp : width;
    const int l32 = lane & 31, lhi = lane >> 5;
    // the 8 values of one row that a thread finishes, where they are in their part, and the
    // block's columns of their stretch
    // (binary16: a row's are neighbours, who look for its largest together)
    const int row = BF ? tid % MR : tid / 8, c8 = (BF ? tid / MR : tid % 8) * 8, w0 = col0 + c8;
    static_assert(MT / MR == 8, "64 columns of a row over 8 threads");
    const int part = p.per_part ? of_part : w0 / p.rp, at_rank = w0 - part * p.rp;
    const int from = p.per_part ? 0 : c8 - at_rank, to = p.per_part ? MC : from + p.rp;
    const char* src[LPW];
    const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
        const int row = 8 * (wave + MW * i) + (lane >> 3);
        const int w = min(col0 + max(row - MR, 0), width - 1), part = w / p.rp, j = min(w - part * p.rp, p.rank - 1);
        const uint16_t* r = row < MR ? p.x + (size_t)tile_row[min(row, n_rows - 1)] * p.K
                                     : p.A + (((size_t)slot * p.parts + part) * p.rank + j) * p.K;
        src[i] = reinterpret_cast<const char*>(r);
    }
    const uint32_t base = lds_address(lds) + (uint32_t)wave * 1024u;
    const int shares = (int)gridDim.z, chunks = (p.K + KC - 1) / KC;
    const int c0 = chunks * (int)blockIdx.z / shares, c1 = chunks * ((int)blockIdx.z + 1) / shares;
    auto load = [&](int c, int stage) {
        // (past K, whose multiple is 32, the first half repeats; it is not multiplied)
        const int at = c * KC + chunk * 8 < p.K ? chunk : chunk & 3;
#pragma unroll
        for (int i = 0; i < LPW; ++i) dma_lane(src[i] + ((size_t)c * KC * 2 + at * 16), base + (uint32_t)(stage * STAGE + i * MW * 1024));
    };
    f16x acc[NB];
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[h][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) load(min(c0 + i, c1 - 1), i);
    int stage = 0;
    const char* operand = lds + l32 * (KC * 2) + (((2 * wave + lhi) ^ (l32 & 7)) << 4);
    for (int c = c0; c < c1; ++c) {
        // this stage has landed, in every wave, and the one before is read
        wait_loads<(NS - 2) * LPW>();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        load(min(c + NS - 1, c1 - 1), stage == 0 ? NS - 1 : stage - 1);
        __builtin_amdgcn_sched_barrier(0);
        if (c * KC + 16 * wave < p.K) {
            const u4 a = *reinterpret_cast<const u4*>(operand + stage * STAGE);
#pragma unroll
            for (int h = 0; h < NB; ++h) {
                const u4 b = *reinterpret_cast<const u4*>(operand + stage * STAGE + (MR + 32 * h) * (KC * 2));
                if constexpr (BF) acc[h] = mfma32(bitcast<b8>(a), bitcast<b8>(b), acc[h]);
                else acc[h] = mfma32(bitcast<h8>(a), bitcast<h8>(b), acc[h]);
            }
        }
        stage = stage + 1 == NS ? 0 : stage + 1;
    }
    wait_loads<0>();      // (the repeated last ones, before their stage is written)
    __syncthreads();
    // ---- the waves' sums: a thread takes 8 values of one row
    constexpr int PITCH = MC + 4;
    float(*red)[MR][PITCH] = reinterpret_cast<float(*)[MR][PITCH]>(lds);
    static_assert(sizeof(float) * MW * MR * PITCH <= sizeof(lds), "sums in the stages");
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e) red[wave][8 * (e >> 2) + 4 * lhi + (e & 3)][32 * h + l32] = acc[h][e];
    __syncthreads();
    const bool mine = c8 < MC && row < n_rows && w0 < cols;
    f4 z[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
    if (mine)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] = *reinterpret_cast<const f4*>(&red[0][row][c8 + 4 * h]);
#pragma unroll
            for (int v = 1; v < MW; ++v) z[h] += *reinterpret_cast<const f4*>(&red[v][row][c8 + 4 * h]);
        }
    // ---- the shares of K, in order, by the last to arrive
    if (shares > 1) {
        const int block = (int)blockIdx.x * (int)gridDim.y + (int)blockIdx.y;
        const rsrc_t r = make_rsrc(p.partial + (size_t)block * shares * (MR * 64), (uint32_t)shares * (MR * 64 * 4));
        const uint32_t at = (uint32_t)tid * 32u;
        if (mine)
#pragma unroll
            for (int h = 0; h < 2; ++h) put16(r, (uint32_t)blockIdx.z * (MR * 64 * 4) + at + 16u * h, z[h]);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(&p.arrived[block], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(shares - 1);
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) __hip_atomic_store(&p.arrived[block], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        f4 o[kMaxShares][2];
#pragma unroll
        for (int s = 0; s < kMaxShares; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) o[s][h] = take16(r, (uint32_t)min(s, shares - 1) * (MR * 64 * 4) + at + 16u * h);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] = o[0][h];
#pragma unroll
            for (int s = 1; s < kMaxShares; ++s)
                if (s < shares) z[h] += o[s][h];
        }
    }
    // (values past the rank meet zeros of B: they must be finite)
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = mine && at_rank + e < p.rank ? z[e >> 2][e & 3] * scale : 0.f;
    float down = 1.f;
    if constexpr (!BF) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_isfinite(t[e]) ? fabsf(t[e]) : 0.f);
        // (of this part's: a block of the whole width has several)
        const float own = top;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl(own, (lane & ~7) + i);
            top = fmaxf(top, 8 * i >= from && 8 * i < to ? other : 0.f);
        }
        float up = 1.f;
        if (top != 0.f && (top < kReachLow || top > kReachHigh)) {
            const int exponent = min(max((int)(bitcast<uint32_t>(top) >> 23), 27), 253);
            up = bitcast<float>((uint32_t)exponent << 23);
            down = bitcast<float>((uint32_t)(254 - exponent) << 23);
        }
        if (mine && c8 == from) p.up[(size_t)(p.per_part ? (int)blockIdx.y : part) * p.up_pitch + pos + row] = up;
    }
    if (!mine) return;
    u4 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = t[e] * down;
        const uint16_t r = f32_to_act<BF>(y);
        // what the rounding leaves; nothing of a value beyond the type's range
        const float rest = y - act_to_f32<BF>(r);
        const uint16_t u = f32_to_act<BF>(__builtin_isfinite(rest) ? rest : 0.f);
        hi[e >> 1] = e & 1 ? hi[e >> 1] | (uint32_t)r << 16 : r;
        lo[e >> 1] = e & 1 ? lo[e >> 1] | (uint32_t)u << 16 : u;
    }
    const int at = pos + row;
    const size_t o = ((size_t)(at >> 5) * width + w0) * 32 + (at & 31) * 8;
    *reinterpret_cast<u4*>(p.hi + o) = hi;
    *reinterpret_cast<u4*>(p.lo + o) = lo;
}

}  // namespace

struct q4_adapters {
    int slots = 0, rank = 0, rp = 0, parts = 0, K = 0, N = 0, device = -1;
    std::vector<int> part_n;           // columns of each part
    bool bf16 = false;
    uint16_t *A = nullptr, *B = nullptr;
    float* scale = nullptr;
    int* wild = nullptr;               // whether a slot's B has values that are not finite
    uint8_t* part8 = nullptr;
    float* t = nullptr;                // few rows: [Q4_GEMV_MAX_M][parts * rp]
    std::mutex mutex;
    char* shares = nullptr;            // many rows' workspace: shares of K, and (many) what goes by rows,
    char* many = nullptr;              // of which it holds many_rows
    int many_rows = 0;
    std::vector<char*> retired;        // outgrown ones, freed with the bank
};

namespace q4 {

namespace {

// Values of a slot's B.
size_t b_values(const q4_adapters* a) { return ((size_t)a->N + 31) / 32 * 32 * a->rp; }

// (a count for each tile whose K is shared, and their sums)
constexpr size_t kArrivedBytes = kManyGroups * sizeof(uint32_t), kPartialBytes = (size_t)kManyGroups * MR * 64 * sizeof(float);

struct ManySpace {
    AdapterRow* rows;
    uint16_t *hi, *lo;
    float* up;
    size_t bytes;
};

// Stretches of a bank; blocks of columns that c A x of many rows is made in: the whole
// width where it has 64 values at most, else 64 at a time, of binary16 a stretch.
int stretches(const q4_adapters* a) { return a->parts * ((a->rp + kStretch - 1) / kStretch); }
bool whole_width(const q4_adapters* a) { return a->parts * a->rp <= kStretch; }
int column_blocks(const q4_adapters* a)
{
    return whole_width(a) ? 1 : a->bf16 ? (a->parts * a->rp + kStretch - 1) / kStretch : stretches(a);
}

// What goes by rows of a bank's many-row workspace. The rows are whole output tiles.
constexpr int kRowStep = 256;
ManySpace many_space(const q4_adapters* a, char* base, int rows)
{
    const size_t m = (size_t)rows, width = (size_t)a->parts * a->rp;
    ManySpace s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    s.rows = reinterpret_cast<AdapterRow*>(take(m * sizeof(AdapterRow)));
    s.hi = reinterpret_cast<uint16_t*>(take(m * width * 2));
    s.lo = reinterpret_cast<uint16_t*>(take(m * width * 2));
    s.up = reinterpret_cast<float*>(take(a->bf16 ? 0 : m * stretches(a) * sizeof(float)));
    s.bytes = at;
    return s;
}

q4_status load_slot(q4_adapters* a, int slot, const uint16_t* A, const uint16_t* B, int rank, float c,
                    hipStream_t stream, const char* who)
{
    if (!a) return fail(Q4_ERR_INVALID_ARG, "%s: null bank", who);
    if (slot < 0 || slot >= a->slots) return fail(Q4_ERR_INVALID_ARG, "%s: slot %d outside [0, %d)", who, slot, a->slots);
    int cur = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
    if (cur != a->device) return fail(Q4_ERR_INVALID_ARG, "%s: the bank is on device %d, the current device is %d", who, a->device, cur);
    const size_t sa = (size_t)a->parts * a->rank * a->K, sb = b_values(a);
    const int grid = (int)std::min<size_t>((std::max(sa, sb) + 255) / 256, 4096);
    const std::lock_guard<std::mutex> lock(a->mutex);      // (two launches)
    hipLaunchKernelGGL(q4_adapter_reset_kernel, dim3(1), dim3(1), 0, stream, a->scale + slot, a->wild + slot, c);
    hipLaunchKernelGGL((a->bf16 ? q4_adapter_load_kernel<true> : q4_adapter_load_kernel<false>), dim3(grid), dim3(256), 0, stream, A, B,
                       a->A + slot * sa, a->B + slot * sb, a->wild + slot, a->parts, rank, a->rank, a->rp, a->K, a->N);
    e = hipGetLastError();
    return e == hipSuccess ? Q4_OK : fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // namespace

q4_status adapters_check(const q4_adapters* a, const q4_matrix* h, const int* index, bool bf16, const char* who)
{
    if (!a || !index) return fail(Q4_ERR_INVALID_ARG, "%s: null bank or index", who);
    if (a->K != h->K || a->N != h->N || a->device != h->device || a->part_n != h->part_n)
        return fail(Q4_ERR_INVALID_ARG, "%s: the bank was made for another matrix", who);
    if (a->bf16 != bf16)
        return fail(Q4_ERR_INVALID_ARG, "%s: the bank holds %s, the activations are %s", who, a->bf16 ? "bfloat16" : "float16",
                    bf16 ? "bfloat16" : "float16");
    return Q4_OK;
}

// Held over all of a call's launches: they hand c A x over in the bank's workspace, and
// two host threads may use one stream.
std::unique_lock<std::mutex> adapters_lock(q4_adapters* a) { return std::unique_lock<std::mutex>(a->mutex); }

// Grow a bank's workspace to hold M rows before anything of a call is launched.
q4_status adapters_reserve(q4_adapters* a, int M, hipStream_t stream)
{
    const char* who = "q4_matmul_adapters";
    if (a->many_rows >= M) return Q4_OK;
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(stream, &cap);
    if (e != hipSuccess) return fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
    if (cap != hipStreamCaptureStatusNone)
        return fail(Q4_ERR_INVALID_ARG, "%s: the bank's workspace must grow to M=%d under stream capture; make one "
                    "uncaptured call with this M (or larger) first", who, M);
    auto failed = [&](hipError_t e) { return fail(e == hipErrorOutOfMemory ? Q4_ERR_OOM : Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e)); };
    if (!a->shares) {
        char* shares = nullptr;
        if ((e = hipMalloc(&shares, kArrivedBytes + kPartialBytes)) != hipSuccess) return failed(e);
        if ((e = hipMemsetAsync(shares, 0, kArrivedBytes, stream)) != hipSuccess) {
            (void)hipFree(shares);
            return failed(e);
        }
        a->shares = shares;
    }
    // (twice the last at least, so that those outgrown hold no more together than the
    // present one; as much as is needed where there is no room for that)
    const long long need = ((long long)M + kRowStep - 1) / kRowStep * kRowStep;
    long long rows = std::min<long long>(std::max(need, 2LL * a->many_rows), INT_MAX / kRowStep * kRowStep);
    char* fresh = nullptr;
    e = hipMalloc(&fresh, many_space(a, nullptr, (int)rows).bytes);
    if (e == hipErrorOutOfMemory && rows > need) {
        (void)hipGetLastError();
        rows = need;
        e = hipMalloc(&fresh, many_space(a, nullptr, (int)rows).bytes);
    }
    if (e != hipSuccess) return failed(e);
    // (earlier launches, and graphs, may still use the outgrown one)
    try {
        if (a->many) a->retired.push_back(a->many);
    } catch (const std::bad_alloc&) {
        (void)hipFree(fresh);
        return fail(Q4_ERR_OOM, "%s: out of memory", who);
    }
    a->many = fresh;
    a->many_rows = (int)rows;
    return Q4_OK;
}

// c A x for the rows of a call, and the arguments of the product's launch.
q4_status adapters_prepare(q4_adapters* a, const uint16_t* x, const int* index, int M, bool few,
                           q4dev::AdapterArgs* args, hipStream_t stream)
{
    const char* who = "q4_matmul_adapters";
    *args = {};
    args->B = a->B;
    args->part8 = a->part8;
    args->slots = a->slots;
    args->b_slot = b_values(a);
    args->rp = a->rp;
    args->width = a->parts * a->rp;
    args->index = index;
    hipError_t e;
    if (few) {
        args->t = a->t;
        const dim3 grid(args->width, M), block(64 * DW);
        if (a->bf16)
            hipLaunchKernelGGL((q4_adapter_few_kernel<true>), grid, block, 0, stream, x, index, a->A, a->scale, a->t, a->K, a->slots, a->rank, a->rp, a->parts);
        else
            hipLaunchKernelGGL((q4_adapter_few_kernel<false>), grid, block, 0, stream, x, index, a->A, a->scale, a->t, a->K, a->slots, a->rank, a->rp, a->parts);
        e = hipGetLastError();
        return e == hipSuccess ? Q4_OK : fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
    }
    const int held = a->many_rows;
    char* base = a->many;
    const ManySpace s = many_space(a, base, held);
    args->rows = s.rows;
    args->hi = s.hi;
    args->lo = s.lo;
    args->up = s.up;
    args->up_pitch = held;
    ManyArgs p;
    p.x = x;
    p.index = index;
    p.A = a->A;
    p.scale = a->scale;
    p.wild = a->wild;
    p.rows = s.rows;
    p.hi = s.hi;
    p.lo = s.lo;
    p.M = M;
    p.K = a->K;
    p.slots = a->slots;
    p.rank = a->rank;
    p.rp = a->rp;
    p.parts = a->parts;
    p.arrived = reinterpret_cast<uint32_t*>(a->shares);
    p.partial = reinterpret_cast<float*>(a->shares + kArrivedBytes);
    // tiles: a whole one each MR rows, and a partial one each bin with rows; K is
    // shared out while there are fewer workgroups than CUs, in shares of 256
    // values and more
    const bool narrow = args->width <= 32;
    const int tiles = M / MR + std::min(a->slots + 1, M), blocks = column_blocks(a);
    p.up = s.up;
    p.up_pitch = held;
    p.per_part = a->bf16 || whole_width(a) ? 0 : blocks / a->parts;
    const int shares = (int)std::clamp<long long>(kManyGroups / ((long long)tiles * blocks), 1, std::min(kMaxShares, std::max(a->K / 256, 1)));
    const dim3 grid(tiles, blocks, shares), block(MT);
    const size_t lds = (size_t)(a->slots + 1) * sizeof(int);
    auto launch = [&](auto bf, auto nb) {
        hipLaunchKernelGGL((q4_adapter_many_kernel<decltype(bf)::value, decltype(nb)::value>), grid, block, lds, stream, p);
    };
    using std::integral_constant;
    if (a->bf16 && narrow) launch(integral_constant<bool, true>{}, integral_constant<int, 1>{});
    else if (a->bf16) launch(integral_constant<bool, true>{}, integral_constant<int, 2>{});
    else if (narrow) launch(integral_constant<bool, false>{}, integral_constant<int, 1>{});
    else launch(integral_constant<bool, false>{}, integral_constant<int, 2>{});
    e = hipGetLastError();
    return e == hipSuccess ? Q4_OK : fail(Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
}

}  // namespace q4

extern "C" {

q4_status q4_check_adapters(int slots, int rank)
{
    if (slots < 1 || rank < 1)
        return q4::fail(Q4_ERR_INVALID_ARG, "q4_adapters_make: %d slots of rank %d", slots, rank);
    if (slots > kMaxSlots || rank > kMaxRank)
        return q4::fail(Q4_ERR_UNSUPPORTED, "q4_adapters_make: %d slots of rank %d (at most %d of %d)", slots, rank, kMaxSlots, kMaxRank);
    return Q4_OK;
}

q4_adapters* q4_adapters_make(const q4_matrix* h, int slots, int rank, int bf16)
{
    const char* who = "q4_adapters_make";
    if (!h) {
        q4::fail(Q4_ERR_INVALID_ARG, "%s: null handle", who);
        return nullptr;
    }
    if (q4_check_adapters(slots, rank) != Q4_OK) return nullptr;
    int cur = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess || cur != h->device) {
        q4::fail(e != hipSuccess ? Q4_ERR_HIP : Q4_ERR_INVALID_ARG, "%s: the handle was made on device %d, the current device is %d", who, h->device, cur);
        return nullptr;
    }
    q4_adapters* a = new (std::nothrow) q4_adapters;
    if (!a) {
        q4::fail(Q4_ERR_OOM, "%s: out of memory", who);
        return nullptr;
    }
    try {
        a->part_n = h->part_n;
    } catch (const std::bad_alloc&) {
        delete a;
        q4::fail(Q4_ERR_OOM, "%s: out of memory", who);
        return nullptr;
    }
    a->slots = slots;
    a->rank = rank;
    a->rp = (rank + 7) / 8 * 8;
    a->parts = (int)h->part_n.size();
    a->K = h->K;
    a->N = h->N;
    a->device = h->device;
    a->bf16 = bf16 != 0;
    const size_t na = (size_t)slots * a->parts * rank * a->K * 2, nb = (size_t)slots * q4::b_values(a) * 2;
    e = hipMalloc(&a->A, na);
    if (e == hipSuccess) e = hipMalloc(&a->B, nb);
    if (e == hipSuccess) e = hipMalloc(&a->scale, (size_t)slots * 4);
    if (e == hipSuccess) e = hipMalloc(&a->wild, (size_t)slots * 4);
    if (e == hipSuccess) e = hipMalloc(&a->t, (size_t)q4::kGemvMaxM * a->parts * a->rp * 4);
    if (e == hipSuccess && a->parts > 1) e = hipMalloc(&a->part8, (size_t)a->N / 8);
    if (e == hipSuccess) e = hipMemset(a->A, 0, na);
    if (e == hipSuccess) e = hipMemset(a->B, 0, nb);
    if (e == hipSuccess) e = hipMemset(a->scale, 0, (size_t)slots * 4);
    if (e == hipSuccess) e = hipMemset(a->wild, 0, (size_t)slots * 4);
    if (e == hipSuccess && a->parts > 1) {
        std::unique_ptr<uint8_t[]> part(new (std::nothrow) uint8_t[(size_t)a->N / 8]);
        if (!part) {
            e = hipErrorOutOfMemory;
        } else {
            size_t at = 0;
            for (int i = 0; i < a->parts; ++i)
                for (int n = 0; n < h->part_n[i]; n += 8) part[at++] = (uint8_t)i;
            e = hipMemcpy(a->part8, part.get(), (size_t)a->N / 8, hipMemcpyHostToDevice);
        }
    }
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        q4_adapters_free(a);
        q4::fail(e == hipErrorOutOfMemory ? Q4_ERR_OOM : Q4_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
        return nullptr;
    }
    return a;
}

void q4_adapters_free(q4_adapters* a)
{
    if (!a) return;
    (void)hipFree(a->A);
    (void)hipFree(a->B);
    (void)hipFree(a->scale);
    (void)hipFree(a->wild);
    (void)hipFree(a->t);
    (void)hipFree(a->part8);
    (void)hipFree(a->shares);
    (void)hipFree(a->many);
    for (char* p : a->retired) (void)hipFree(p);
    delete a;
}

q4_status q4_adapters_load(q4_adapters* a, int slot, const uint16_t* A, const uint16_t* B, int rank, float c, hipStream_t stream)
{
    const char* who = "q4_adapters_load";
    if (!A || !B) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null A or B", who);
    if (a && (rank < 1 || rank > a->rank)) return q4::fail(Q4_ERR_INVALID_ARG, "%s: rank %d outside [1, %d]", who, rank, a->rank);
    return q4::load_slot(a, slot, A, B, rank, c, stream, who);
}

q4_status q4_adapters_clear(q4_adapters* a, int slot, hipStream_t stream)
{
    return q4::load_slot(a, slot, nullptr, nullptr, 0, 0.f, stream, "q4_adapters_clear");
}

}  // extern "C"
