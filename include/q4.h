/*
 * q4.h -- C ABI of libq4: the fused GPTQ 4-bit dequantize-and-multiply on
 * AMD Instinct MI355X (gfx950).
 *
 *   y[m,n] = sum_k x[m,k] * W[k,n],  W[k,n] = s[g(k),n] * (q[k,n] - z[g(k),n])
 *
 * The packed 4-bit weights are read from device memory and unpacked and
 * dequantized in registers; no dequantized weight matrix is ever written to
 * memory ("GPTQ's 'Exllama Kernel Not Installed' Warning", section "What the
 * fallback actually does"). The interface follows the handle + matmul pair of
 * "Implementation: Predibase Lorax GPTQ Exllama V1" (Description: a handle is
 * made once from qweight, qzeros, scales and an optional g_idx; the matmul
 * takes a 2-D activation and produces (batch, width)).
 *
 * Conventions for every entry point:
 *  - All tensor pointers passed to q4_make / q4_matmul* / q4_dequant_dump are
 *    DEVICE pointers on the current HIP device, to dense row-major data. A
 *    handle is used on the device it was made on: q4_matmul* and
 *    q4_dequant_dump return Q4_ERR_INVALID_ARG when another device is
 *    current.
 *  - fp16 data is passed as uint16_t bit patterns (IEEE binary16).
 *  - A failing call returns NULL or a non-zero q4_status, enqueues nothing and
 *    leaves every output untouched; q4_last_error() then holds the reason
 *    (thread-local, valid until the next failing call on that thread).
 *  - There is no silent fallback: when a case is not implemented on the GPU
 *    the call fails with Q4_ERR_UNSUPPORTED.
 *  - Calls that take a stream enqueue work on it and return without waiting;
 *    faults inside a kernel surface at the caller's next synchronization.
 *
 * Tensor formats (GPTQ checkpoint layout; "GPTQ's 'Exllama Kernel Not
 * Installed' Warning", section "Why the kernel is missing": 32-bit words
 * carrying 4-bit codes, a scale and a zero point for each group; I/O
 * contract table of the Lorax page: qweight/qzeros int32, scales fp16, g_idx
 * int32 or absent, bits = 4):
 *  - qweight int32 [K/8][N]: word (r, n) holds the codes of input rows
 *    k = 8r .. 8r+7 of column n, the code of k = 8r+i in bits 4i .. 4i+3.
 *  - qzeros  int32 [ceil(K/G)][N/8]: word (g, c) holds the zero points of
 *    columns n = 8c .. 8c+7 of group g, in the same nibble order. The stored
 *    nibble is the zero point itself (no offset).
 *  - scales  fp16  [ceil(K/G)][N].
 *  - g_idx   int32 [K] or NULL: group of input row k. NULL means g(k) = k / G.
 *  - x fp16 [M][K], out fp16 [M][N], bias fp16 [N].
 */
#ifndef Q4_H
#define Q4_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct q4_matrix q4_matrix;   /* opaque handle, immutable after q4_make */

typedef enum {
    Q4_OK = 0,
    Q4_ERR_INVALID_ARG = 1,   /* null pointer, bad shape or value            */
    Q4_ERR_UNSUPPORTED = 2,   /* valid input the GPU path does not implement */
    Q4_ERR_DEVICE = 3,        /* current device is not gfx950                */
    Q4_ERR_HIP = 4,           /* a HIP runtime call failed                   */
    Q4_ERR_OOM = 5            /* device allocation failed                    */
} q4_status;

/* Kernel identifiers returned by q4_path_for / accepted by q4_dequant_dump. */
enum {
    Q4_PATH_NONE = 0,   /* M == 0: nothing is launched                            */
    Q4_PATH_GEMV = 1,   /* bandwidth-bound skinny kernel, 1 <= M <= Q4_GEMV_MAX_M */
    Q4_PATH_MFMA = 2    /* LDS-staged MFMA GEMM for larger M                      */
};

/* Most rows the skinny kernel takes: q4_matmul runs it for 1 <= M <= 32 and
 * the MFMA GEMM above (q4_path_for tells which). */
#define Q4_GEMV_MAX_M 32
/* Most workgroups one streaming-GEMM launch may be given (q4_matmul_ex). */
#define Q4_GEMM_MAX_WORKERS 1024

/*
 * q4_make -- build a handle from GPTQ tensors (Lorax page, Description: the
 * handle is made once from the packed weights, zero points, scales and an
 * optional group index, and act-order is recognised from a g_idx that is not
 * the identity grouping).
 *
 * Arguments: device pointers qweight and scales (required), qzeros (NULL for
 * a symmetric layer stored without zeros: every zero point is then
 * 2^(bits-1) = 8, as GPTQModel wiki "Inference Backends", section "Packing,
 * conversion, and runtime initialization", row "Missing zeros" synthesizes
 * it), g_idx (optional, NULL allowed); K, N > 0 with K % 32 == 0 and
 * N % 8 == 0;
 * groupsize in {32, 64, 128, 256} with K % groupsize == 0, or -1 for one
 * group spanning K (then K % 32 == 0 still applies).
 *
 * Act-order: a g_idx equal to k / groupsize for every k is trivial and is
 * dropped (same result bit for bit as NULL). Otherwise the rows are reordered
 * by one stable argsort of g_idx (GPTQModel wiki "Inference Backends",
 * section "Runtime cache lifetime"); the sorted g_idx must equal
 * k / groupsize (every group exactly groupsize rows), else
 * Q4_ERR_UNSUPPORTED. g_idx values outside [0, K/groupsize) give
 * Q4_ERR_INVALID_ARG.
 *
 * Ownership: the inputs are read (the call synchronizes the device) and
 * copied into handle-owned device memory in private layouts: the packed
 * weights at the same size (K rounded up to a multiple of 128 rows), and
 * each group's scale and zero point as one 32-bit word per column (the
 * checkpoint's scale and packed zero tensors are not kept). The caller
 * keeps and may free or change its tensors afterwards; such changes do not
 * reach the handle (make a new one). The handle also owns the skinny
 * kernel's split-K workspace, sized for the largest splits x M its launch
 * plan takes at any M <= Q4_GEMV_MAX_M (none when the plan never splits K,
 * as for 4096-wide and wider layers on 256 CUs). It never holds a
 * dequantized K x N matrix. Temporary device buffers for the checkpoint's
 * group parameters are allocated and freed during the call.
 *
 * Returns NULL on error (q4_last_status / q4_last_error tell why).
 */
q4_matrix* q4_make(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                   const int32_t* g_idx, int K, int N, int groupsize);

/*
 * q4_make_bits -- q4_make for 4- or 8-bit codes (bits = 4 or 8). GPTQModel
 * wiki "Inference Backends": GPTQ kernels declare 4- and 8-bit weights
 * (backend catalogue) and the native 8-bit GPTQ path keeps the same
 * checkpoint tensors (section "Runtime cache lifetime"). With bits = 8 a word
 * holds four codes packed the same way (code i in bits 8i .. 8i + 7):
 * qweight [K/4][N] (row k = 4r + i in byte i of word (r, n)), qzeros
 * [K/groupsize][N/4] (column n = 4c + j in byte j of word (g, c)); a NULL
 * qzeros means the symmetric zero point 2^(8-1) = 128. bits = 4 is q4_make.
 * Every other argument, the ownership and the errors are as in q4_make
 * (Q4_ERR_UNSUPPORTED for other bit widths). The matmul calls are the same;
 * 8-bit handles take at most two skinny-kernel column tiles and GEMM
 * variant 0 or 3 only.
 */
q4_matrix* q4_make_bits(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                        const int32_t* g_idx, int K, int N, int groupsize, int bits);

/*
 * q4_matmul -- out[M][N] = fp16(x[M][K] @ W) (Lorax page, Description: x @ q4
 * producing (batch, width)). Accumulation is in fp32 (GPTQModel wiki,
 * hardware table, ExLlama v2 row: FP32 accumulation, FP16 scales); the only
 * rounding to fp16 is the final cast (round to nearest even).
 *
 * x and out are caller-owned device buffers and must not overlap. M == 0 is
 * a no-op returning Q4_OK. M < 0, NULL pointers or a NULL handle give
 * Q4_ERR_INVALID_ARG. M <= Q4_GEMV_MAX_M runs the skinny kernel, larger M the
 * MFMA GEMM (q4_path_for tells which). Sizes beyond the kernels' 32-bit
 * offsets give Q4_ERR_UNSUPPORTED: M * K * 2 or M * N above 2^31 - 1, or
 * more than 2^30 GEMM (output tile, 64-row k-step) pairs (about
 * M * K * N / 2^19).
 *
 * Concurrency: the handle's workspace is shared by its calls, so calls on one
 * handle must be ordered on one stream (or synchronized); different handles
 * are independent. The GEMM's stream-K partial sums (tiles whose K range is
 * split between two workgroups) go to a workspace per (device, stream) that
 * the library allocates on the first call on that stream that needs it
 * (2 x 128 KiB + 4 bytes per workgroup: 128 MiB for 512 workgroups) and
 * keeps until the process ends; calls on one stream share it in order. A
 * captured call keeps the workspace of the stream it was captured on, while
 * a graph replays on whatever stream launches it: graphs holding GEMM calls
 * captured on one stream (torch captures every graph on one shared side
 * stream unless told otherwise) must not be replayed concurrently with each
 * other or with uncaptured GEMM calls on that stream, or they race on its
 * partial sums and arrival counters (wrong outputs, no error). Replays in
 * stream order, one after the other, are safe.
 *
 * Act-order (non-trivial g_idx): the weights are stored in sorted-group
 * order, so the product needs the activations x[:, perm] (the Lorax GPTQ
 * Exllama V1 page, Description: a temporary buffer reorders the activations
 * in the act-order case). Without K splits and for M <= 2, the skinny kernel
 * builds them in LDS itself when they fit (q4_gemv_gather); otherwise, and
 * for the GEMM, a separate kernel first writes x[:, perm] to the handle's
 * workspace.
 *
 * Graph capture: a call may be captured into a HIP graph and replayed; it
 * enqueues kernels only (no memset or copy nodes; the skinny kernel's split-K
 * counters, and the GEMM's stream-K counters, are reset by the kernels). A
 * GEMM call captured on a stream that has no stream-K workspace yet runs one
 * workgroup per output tile instead (the same result up to fp32 rounding).
 * An act-order handle grows its activation workspace on the first call with
 * a larger M that needs the separate permute, which cannot happen under
 * capture: such a call returns Q4_ERR_INVALID_ARG, so make one uncaptured
 * call with the largest M first. Outgrown workspaces are not freed before
 * the handle (act-order buffer) or the process (stream-K buffers), so graphs
 * captured earlier stay valid.
 */
q4_status q4_matmul(const q4_matrix* h, const uint16_t* x, uint16_t* out, int M,
                    hipStream_t stream);

/*
 * q4_matmul_bias -- as q4_matmul, plus bias[n] added to the fp32 accumulator
 * before the single cast to fp16 (GPTQModel wiki, section "Numeric epilogues
 * and input gradients": the bias is summed in FP32 with the product, and the
 * result is rounded once at the end). bias may be NULL (then identical to
 * q4_matmul).
 */
q4_status q4_matmul_bias(const q4_matrix* h, const uint16_t* x, const uint16_t* bias,
                         uint16_t* out, int M, hipStream_t stream);

/*
 * q4_matmul_ex -- q4_matmul_bias with explicit kernel choice, for tests and
 * tuning. path = 0 (automatic, as q4_matmul), Q4_PATH_GEMV (needs
 * 1 <= M <= Q4_GEMV_MAX_M) or Q4_PATH_MFMA (any M >= 1).
 *   skinny kernel: variant = 16-column MFMA tiles per wave, 0 (planned), 1, 2
 *                  or 4; splits = K splits across workgroups, 0 (planned) or
 *                  1..16;
 *   GEMM:          variant = the tile width: 0 or 3 (planned,
 *                  q4_plan_gemm_waves), 4 (128 columns, four waves) or 8
 *                  (256 columns, eight waves; M > 512 only); splits =
 *                  workgroups: 0 (planned, q4_plan_gemm for the planned
 *                  width; for an explicit width, the plan at that width),
 *                  1 (one per output tile: 256 or 64 rows by the width) or
 *                  2..Q4_GEMM_MAX_WORKERS (the tiles' 64-row k-steps shared
 *                  evenly, stream-K; a count above the number of (tile,
 *                  k-step) pairs is reduced to it; under stream capture only
 *                  once the stream has a workspace that large, else
 *                  Q4_ERR_INVALID_ARG).
 * Anything else is Q4_ERR_INVALID_ARG. Results differ between paths,
 * tile widths and split counts only by fp32 rounding. An explicit skinny-kernel
 * split count above the largest the plan takes for the handle grows its
 * split-K workspace, which cannot happen under stream capture
 * (Q4_ERR_INVALID_ARG there: make one uncaptured call with that count first).
 */
q4_status q4_matmul_ex(const q4_matrix* h, const uint16_t* x, const uint16_t* bias,
                       uint16_t* out, int M, int path, int variant, int splits,
                       hipStream_t stream);

/* Bytes of the per-GPU scratch array q4_matmul_static works in (64 MiB). */
#define Q4_STATIC_SCRATCH_BYTES (64u << 20)

/*
 * q4_matmul_static -- q4_matmul_bias for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc. It allocates nothing (no hipMalloc, hipFree or allocating
 * library call): every workspace the call needs (the skinny kernel's split-K
 * partial sums and arrival counters, an act-order layer's permuted
 * activations, the GEMM's stream-K partial sums and counters) lives in one
 * static array of Q4_STATIC_SCRATCH_BYTES per GPU. The array is set up when
 * the first handle is made on a GPU (q4_make looks up its device address, at
 * which point the HIP runtime places it in device memory, and clears its
 * counters) and is kept until the process ends.
 *
 * Arguments, result, numerics and errors as q4_matmul_bias (fp16 x, bias,
 * out). The launch plan is q4_matmul_bias's, except that the skinny kernel's
 * K splits are halved, and the GEMM's stream-K workgroups reduced, until
 * their partial sums fit the array (results then differ from q4_matmul_bias
 * only by fp32 rounding; with the plans of the 7B and 70B layers they are the
 * same bits). An act-order call that needs the separate permute (M > 2, or K
 * split) stores x[:, perm] in the array too: M * K * 2 bytes must fit in
 * Q4_STATIC_SCRATCH_BYTES - 64 KiB, else Q4_ERR_UNSUPPORTED with nothing
 * enqueued.
 *
 * Concurrency: every q4_matmul_static call on a GPU shares that GPU's array,
 * which keeps the last call's contents, so calls that overlap in time on one
 * GPU (other streams, concurrent graph replays) race and give wrong results
 * without an error; order them on one stream. Every call leaves the arrival
 * counters at zero.
 */
q4_status q4_matmul_static(const q4_matrix* h, const uint16_t* x, const uint16_t* bias,
                           uint16_t* out, int M, hipStream_t stream);

/*
 * q4_matmul_bf16 -- q4_matmul_bias with bfloat16 activations, bias and output
 * (GPTQModel wiki "Inference Backends", hardware table, ExLlama v2 row: the
 * activation dtype -- FP16, BF16 or FP32 -- is kept, with FP16 scales and
 * FP32 accumulation). x is bfloat16 [M][K], bias bfloat16 [N] or NULL, out
 * bfloat16 [M][N]; the handle (fp16 scales) is the same as for fp16 calls.
 * Accumulation is fp32 and the only rounding of the result is the final
 * round-to-nearest-even cast to bfloat16. The skinny kernel applies the
 * exact weights s * (q - z) (as the fp16 path); the GEMM multiplies the
 * weights rounded once to bfloat16, RNE_bf16(s * (q - z)), since its matrix
 * operands are bfloat16. Same arguments, ownership, errors, concurrency and
 * graph-capture rules as q4_matmul.
 */
q4_status q4_matmul_bf16(const q4_matrix* h, const uint16_t* x, const uint16_t* bias,
                         uint16_t* out, int M, hipStream_t stream);

/*
 * q4_matmul_ex_bf16 -- q4_matmul_bf16 with an explicit kernel, as
 * q4_matmul_ex; the GEMM takes variant 0 or 3 only (other variants:
 * Q4_ERR_UNSUPPORTED).
 */
q4_status q4_matmul_ex_bf16(const q4_matrix* h, const uint16_t* x, const uint16_t* bias,
                            uint16_t* out, int M, int path, int variant, int splits,
                            hipStream_t stream);

/* q4_free -- release a handle and every device buffer it owns (NULL is
 * allowed). The caller must have synchronized every stream that used it. The
 * pages have no counterpart: their handle lives as long as the module holding
 * it; a C ABI needs an explicit end of life. */
void q4_free(q4_matrix* h);

/*
 * q4_last_status / q4_last_error -- the status and the reason of the last
 * failing call on this thread (Q4_OK and "" before any failure). Every
 * failure is returned, never replaced by a slower route: an explicitly
 * requested backend whose checks fail raises rather than silently running
 * another one, and the rejection keeps its specific reason (GPTQModel wiki
 * "Inference Backends", section "Loading and selecting a backend", and the
 * device-validation paragraph of "Hardware, dependency, and format
 * requirements"). The message is thread-local and stays valid until the next
 * failing call on the same thread.
 */
q4_status q4_last_status(void);
const char* q4_last_error(void);
/*
 * q4_make_cat -- one handle over the column concatenation of `parts` layers
 * (1 <= parts <= 64) that take the same input: QKV or gate/up projection
 * fusion (GPTQModel wiki "Inference Backends", section "How AUTO selection
 * works": eligible QKV or gate/up calls are combined into one after backend
 * selection). One q4_matmul then computes all parts with one launch.
 *
 * Arguments: arrays of `parts` device pointers qweight[i] [K/8][N[i]],
 * qzeros[i] [K/groupsize][N[i]/8], scales[i] [K/groupsize][N[i]] (layouts as
 * in q4_make; qzeros[i] NULL, or qzeros itself NULL, for symmetric parts);
 * N[i] > 0 and a multiple of 8 (host array); one g_idx shared by every part
 * (NULL allowed), K and groupsize as in q4_make.
 *
 * The handle behaves as one layer with N = sum N[i] columns: output column
 * off_i + n (off_i = N[0] + ... + N[i-1]) is column n of part i, and a bias
 * passed to q4_matmul_bias is the concatenation of the parts' biases. Each
 * column's result is the one a handle of its own part gives (same kernel,
 * same order of accumulation when the plan takes the same K splits).
 * Ownership and errors as q4_make; every part's arguments are checked.
 */
q4_matrix* q4_make_cat(int parts, const int32_t* const* qweight, const int32_t* const* qzeros,
                       const uint16_t* const* scales, const int32_t* g_idx, int K, const int* N,
                       int groupsize);

/* q4_make_cat_bits -- q4_make_cat for 4- or 8-bit parts (all parts the
 * same width; layouts as in q4_make_bits). */
q4_matrix* q4_make_cat_bits(int parts, const int32_t* const* qweight, const int32_t* const* qzeros,
                            const uint16_t* const* scales, const int32_t* g_idx, int K, const int* N,
                            int groupsize, int bits);

/*
 * q4_path_for -- the kernel q4_matmul would launch for this M (Q4_PATH_*),
 * or -1 for a NULL handle or M < 0. Lets a caller check which kernel runs
 * ("GPTQ's 'Exllama Kernel Not Installed' Warning": check which kernel runs
 * rather than relying on the absence of a warning).
 */
int q4_path_for(const q4_matrix* h, int M);

/*
 * q4_dequant_dump -- debug: run the unpack + dequantize code of kernel `path`
 * (the dequantized values a kernel computes, dumped in a debug mode so that
 * the in-register unpack and dequantization of "GPTQ's 'Exllama Kernel Not
 * Installed' Warning", section "What the fallback actually does", can be
 * compared bit for bit with the plain definition s * (q - z)):
 * kernel Q4_PATH_GEMV or Q4_PATH_MFMA, over the whole handle, writes the fp16
 * values that kernel feeds its multiply-accumulate to w[K][N] (device
 * buffer, caller-owned, original k order). Each value is
 * round-to-nearest-even of s * (q - z). Not on the hot path.
 */
q4_status q4_dequant_dump(const q4_matrix* h, int path, uint16_t* w, hipStream_t stream);

/*
 * q4_dequant_dump_bf16 -- as q4_dequant_dump (same purpose and source) for
 * the bfloat16 kernels: w is
 * bfloat16 [K][N]. Q4_PATH_GEMV: the skinny kernel's q - z in bfloat16 times
 * the fp32 scale, rounded once to bfloat16; Q4_PATH_MFMA: the bfloat16
 * weights the GEMM feeds its MFMA. Each value is round-to-nearest-even of
 * s * (q - z) to bfloat16.
 */
q4_status q4_dequant_dump_bf16(const q4_matrix* h, int path, uint16_t* w, hipStream_t stream);

/*
 * q4_gemv_gather -- 1 when, for this act-order handle, M and K splits
 * (0: the automatic plan), the skinny kernel builds x[:, perm] in LDS itself,
 * 0 when q4_matmul runs the separate permute kernel first (and for handles
 * without act-order). -1 for a NULL handle, M outside [1, Q4_GEMV_MAX_M] or
 * splits outside [0, 16].
 */
int q4_gemv_gather(const q4_matrix* h, int M, int splits);

/* Handle geometry: K, N, groupsize (after -1 -> K), act-order flag (1 when a
 * non-trivial g_idx was given). Returns 0, or -1 for a NULL handle. */
int q4_handle_info(const q4_matrix* h, int* K, int* N, int* groupsize, int* act_order);

/* The handle's code width (4 or 8), or -1 for a NULL handle. */
int q4_handle_bits(const q4_matrix* h);

/*
 * q4_read_probe -- measurement helper, not part of the product: enqueue one
 * kernel on `stream` that reads `bytes` of device memory at buf with the
 * skinny kernel's kind of load (16 bytes a lane, non-temporal) and no other
 * work, so that timing it gives the achievable read rate of one launch of
 * that size. Decode steps whose bytes are mostly weights run at the speed of
 * memory, not arithmetic ("GPTQ's 'Exllama Kernel Not Installed' Warning",
 * section "What the fallback actually does"); this is the ceiling the fused
 * kernel's effective bandwidth is compared with. buf: device pointer, 16-byte aligned; bytes: a positive
 * multiple of 16384; sink: device buffer of 256 uint32_t, written only when
 * the folded data match a fixed constant (the caller ignores it). Returns
 * Q4_ERR_INVALID_ARG for bad arguments (nothing enqueued), Q4_ERR_HIP if the
 * launch fails.
 */
q4_status q4_read_probe(const void* buf, size_t bytes, uint32_t* sink, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Host-only planning helpers (no HIP calls; usable without a GPU).
 * ---------------------------------------------------------------------- */

/*
 * q4_check_shape -- the argument checks q4_make applies to (K, N, groupsize),
 * without touching memory. Returns Q4_OK, Q4_ERR_INVALID_ARG or
 * Q4_ERR_UNSUPPORTED (message in q4_last_error).
 */
q4_status q4_check_shape(int K, int N, int groupsize);

/* q4_check_shape for q4_make_bits (bits = 4 or 8; other widths give
 * Q4_ERR_UNSUPPORTED). */
q4_status q4_check_shape_bits(int K, int N, int groupsize, int bits);

/*
 * q4_plan_actorder -- host act-order plan for a host copy of g_idx[K]:
 * perm[k'] = stable argsort of g_idx (ties by increasing k), *trivial = 1
 * when g_idx[k] == k / groupsize for all k (perm is then the identity).
 * Returns Q4_ERR_INVALID_ARG for out-of-range values and Q4_ERR_UNSUPPORTED
 * when the sorted groups are not exactly groupsize rows each.
 */
q4_status q4_plan_actorder(const int32_t* g_idx_host, int K, int groupsize, int32_t* perm,
                           int* trivial);

/*
 * q4_plan_gemm -- the streaming GEMM's planned workgroup count for an
 * M x N output with K rows on a chip of num_cu compute units (<= 0: 256), at
 * the planned tile width for 4-bit weights (q4_plan_gemm_waves; an 8-bit
 * handle plans as for four waves). Output tiles are 64 x 128
 * when M <= 512, else 256 x 128 (four waves) or 256 x 256 (eight waves).
 * Four waves: one workgroup per tile when the tiles fill whole rounds of two
 * per CU (to within a tenth) or make at least 1.5 such rounds; otherwise the
 * tiles' 64-row k-steps are shared evenly (stream-K): with 64-row tiles by
 * 2 num_cu workgroups when each gets at least 32 k-steps, by num_cu when
 * each gets at least 16, else by one per 16 k-steps (at least one per tile);
 * with 256-row tiles by min(2 num_cu, max(2 tiles, num_cu)). Eight waves
 * (one workgroup per CU): one per tile when the tiles fill whole rounds of
 * num_cu to within a tenth, else num_cu. Never more than there are (tile,
 * k-step) pairs.
 * Host-only; -1 for M, N or K < 1.
 */
int q4_plan_gemm(int M, int N, int K, int num_cu);

/*
 * q4_plan_gemm_waves -- the streaming GEMM's planned tile width, in waves of
 * 32 columns: 8 (256-column tiles) for M > 512 when the 256 x 256 tiles are
 * at least num_cu, or at least num_cu / 2 with at least 64 (tile, 64-row
 * k-step) pairs per CU, or any number with at least 128 pairs per CU; else
 * 4 (128-column tiles). For 4-bit weights: 8-bit handles always take 4.
 * Host-only; -1 for M, N or K < 1.
 */
int q4_plan_gemm_waves(int M, int N, int K, int num_cu);

/*
 * q4_plan_gemv -- the skinny kernel's launch plan for (M, K, N, groupsize) on
 * a chip of num_cu compute units (<= 0: 256): 16-column tiles per wave
 * (*col_tiles: 1, 2 or 4) and K splits across workgroups (*splits: 1..16).
 * Host-only. Q4_ERR_INVALID_ARG for M outside [1, Q4_GEMV_MAX_M] or null
 * outputs; the q4_check_shape status for an unsupported shape.
 */
q4_status q4_plan_gemv(int M, int K, int N, int groupsize, int num_cu, int* col_tiles,
                       int* splits);

/*
 * q4_plan_gemv_gather -- host-only form of q4_gemv_gather's rule: 1 when
 * splits == 1, M <= 2, K padded to whole 128-row blocks is at most 12288
 * rows and M of those rows, each padded by 8 halfs, fit 20480 halfs (40 KiB
 * of LDS); else 0. -1 for M outside [1, Q4_GEMV_MAX_M], K < 1 or splits outside
 * [1, 16].
 */
int q4_plan_gemv_gather(int M, int K, int splits);

/* ------------------------------------------------------------------------
 * Operators around the product: rotary positions, a paged cache of keys and
 * values. All take 16-bit data: binary16 or (bf16 != 0) bfloat16 patterns.
 * Token and head strides count values; the values of a head are dense.
 * ---------------------------------------------------------------------- */

typedef struct q4_rotary q4_rotary;   /* opaque, immutable after q4_rotary_make */

#define Q4_ROTARY_MAX_DIM 512
enum { Q4_ROTARY_HALF = 0, Q4_ROTARY_INTERLEAVED = 1 };
enum { Q4_ROTARY_NONE = 0, Q4_ROTARY_LINEAR = 1, Q4_ROTARY_BASE = 2, Q4_ROTARY_BY_PARTS = 3 };

/*
 * q4_rotary_make -- rotary positions for heads of `dim` values (at most
 * Q4_ROTARY_MAX_DIM) whose first `rot` (even, 2 .. dim) are rotated. With
 * n = rot / 2, pair i is values (i, i + n) (Q4_ROTARY_HALF) or (2i, 2i + 1)
 * (Q4_ROTARY_INTERLEAVED) and turns by w_i radians a position:
 *   NONE      w_i = base^(-i / n)
 *   LINEAR    w_i = base^(-i / n) / factor
 *   BASE      the same as NONE with base * factor^(rot / (rot - 2))
 *   BY_PARTS  w_i keep_i + w_i / factor (1 - keep_i), w_i as for NONE, where
 *             keep_i = clamp((original_length w_i / 2 pi - low) / (high - low), 0, 1):
 *             pairs that turn at least `high` times within the original length
 *             keep their frequency, those below `low` turns are stretched;
 *             the result is multiplied by 0.1 ln(factor) + 1.
 * factor >= 1, base > 1. The table lives on the current device, on which the
 * handle is then used. Returns NULL on error (q4_last_status/q4_last_error).
 */
q4_rotary* q4_rotary_make(int dim, int rot, int layout, int scaling, double base, double factor,
                          int original_length, double low, double high);
/* q4_rotary_free -- release it (NULL allowed); the caller has synchronized
 * every stream that used it. */
void q4_rotary_free(q4_rotary* r);

/*
 * q4_rotary_plan -- host-only: the checks of q4_rotary_make and its table,
 * turns[rot / 2] = w_i / (2 pi) * 2^64 rounded, and the factor on the result.
 */
q4_status q4_rotary_plan(int dim, int rot, int scaling, double base, double factor, int original_length,
                         double low, double high, uint64_t* turns, float* magnitude);

/*
 * q4_rotary_apply -- out[t][h] = rotation by positions[t] of x[t][h], or with
 * `transpose` its transpose (the gradient of the input from the gradient of
 * the output). Positions are device integers of 32 or 64 bits, negative ones
 * allowed; the angle is exact modulo a turn (64-bit fixed point). fp32, one
 * rounding. out may be x itself (same strides), else they must not overlap (nor
 * out and the positions): Q4_ERR_INVALID_ARG.
 */
q4_status q4_rotary_apply(const q4_rotary* r, const uint16_t* x, int64_t x_token, int64_t x_head, uint16_t* out,
                          int64_t out_token, int64_t out_head, const void* positions, int position_bits,
                          int tokens, int heads, int transpose, int bf16, hipStream_t stream);

/*
 * A paged cache: `pages` pages of `page_size` rows for each of `kv_heads`
 * heads. Row r of head h of page p lies at k + p k_stride[0] + h k_stride[1]
 * + r k_stride[2] (in values, non-negative), `dim` dense values; v likewise.
 * Device memory is the caller's.
 */
typedef struct {
    void* k;
    void* v;
    int64_t k_stride[3];
    int64_t v_stride[3];
    int pages, kv_heads, page_size, dim, bf16;
} q4_cache;

/*
 * q4_cache_append -- write `tokens` tokens to the cache: token t's keys
 * (rotated by positions[t] when `rotary` is given, copied when it is NULL)
 * and its values go to row slots[t] % page_size of page slots[t] / page_size.
 * A token whose slot is negative or not below pages * page_size is not
 * written. Slots must differ: a row is written in pieces, so two tokens with one slot
 * may leave pieces of both, and the keys of one with the values of the other. k and v
 * may be rows of the cache only if each goes to where it is. With q, its `heads`
 * heads are rotated too, into q_out (which may be q itself), for every token; q_out
 * must not overlap anything else of the call (Q4_ERR_INVALID_ARG).
 */
q4_status q4_cache_append(const q4_cache* c, const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                          int64_t v_token, int64_t v_head, const void* slots, int slot_bits, int tokens,
                          const q4_rotary* rotary, const void* positions, int position_bits, const uint16_t* q,
                          int64_t q_token, int64_t q_head, uint16_t* q_out, int64_t out_token, int64_t out_head,
                          int heads, hipStream_t stream);

/* Bytes of workspace q4_attend needs for this cache and number of heads on
 * the current device, whatever the call's other sizes; 0 on error
 * (q4_last_error). */
size_t q4_attend_workspace(const q4_cache* c, int heads);

/*
 * q4_attend -- attention of new tokens over the cache. q holds `tokens` new
 * tokens of `requests` requests one after the other: request b's are tokens
 * starts[b] .. starts[b + 1] - 1 (starts: requests + 1 values, from 0 to
 * tokens), the last of its lengths[b] cached ones (their own keys and values
 * are in the cache already). Key j of request b is row j % page_size of page
 * table[b table_stride + j / page_size]. `heads` is a multiple of the cached
 * heads; head h reads cached head h / (heads / kv_heads). Token i, at position
 * p, sees keys j <= p, with window > 0 only p - window < j:
 *   out[i][h] = sum_j softmax_j(scale q[i][h] . k[j]) v[j]
 * and zeros where it sees none (NaN where every score is -inf). fp32 scores, softmax and sums; the weights
 * are rounded to the data's type for the second product.
 *
 * Only rows that some token of the tile sees are read, and of the table only
 * the entries of pages that hold them. Entries outside [0, pages), lengths above
 * table_width * page_size and starts outside the tokens do not lead outside
 * the tensors, but the result then has no meaning. Keys and values that are not
 * finite reach the tokens that see them and no others.
 *
 * dim is a multiple of 8, at most 256; strides of q and the cache are
 * multiples of 8 values, their base 16-byte aligned. `workspace` is device
 * memory of at least q4_attend_workspace bytes whose first 64 KiB are zero before
 * its first use (each call leaves them fit for the next); calls that share it must not overlap
 * in time. out must not overlap an input (Q4_ERR_INVALID_ARG). A call of 2^24 units and more of 128 rows
 * (token, head of a group) of one request and cached head is refused (Q4_ERR_UNSUPPORTED). Host and device never
 * synchronize; the call may be captured.
 */
q4_status q4_attend(const q4_cache* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                    const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                    int64_t table_stride, int requests, int window, float scale, uint16_t* out, int64_t out_token,
                    int64_t out_head, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * q4_attend_ex -- q4_attend with sinks: with window > 0 a token at position p
 * sees key j <= p if p - window < j or j < sinks: the first `sinks` keys of
 * every request stay visible. (Without a window they are visible anyway.) Of
 * the table only the entries of pages that hold a visible key are read, so
 * those between the sinks and the window may name no page.
 */
q4_status q4_attend_ex(const q4_cache* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                       const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                       int64_t table_stride, int requests, int window, int sinks, float scale, uint16_t* out,
                       int64_t out_token, int64_t out_head, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/*
 * A paged cache held in 4 bits. Row r of head h of page p is dim / 2 bytes of
 * codes at k + p k_stride[0] + h k_stride[1] + r k_stride[2] (value 2 i in the low
 * half of byte i, 2 i + 1 in its high half) and, at k_scale + p k_scale_stride[0]
 * + ..., for each group of `group` neighbouring values a binary16 pair: the step s
 * and the least value m. Strides count bytes. Code c stands for the binary16
 * value RNE(s c + m). v likewise. dim is a multiple of 32, at most 256; group is
 * 32, 64, 128 or 256 and divides dim; code strides are multiples of 16 bytes (base
 * 16-byte aligned), scale strides of 4; rows lie at most 2^26 bytes apart.
 * Device memory is the caller's.
 */
typedef struct {
    void* k;
    void* v;
    void* k_scale;
    void* v_scale;
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t k_scale_stride[3];
    int64_t v_scale_stride[3];
    int pages, kv_heads, page_size, dim, group;
} q4_cache4;

/* The checks of a cache held in 4 bits that need no device, and, what the calls themselves do not
 * look at, that codes and scales do not overlap each other. */
q4_status q4_check_cache4(const q4_cache4* c);

/*
 * q4_cache4_append -- q4_cache_append into a cache held in 4 bits; k, v and q are
 * binary16 or (bf16 != 0) bfloat16. A key is turned (in 64 bits, rounded to fp32 and
 * then to that type) and quantised, a value is quantised, by groups:
 *   lo, hi = the group's least and largest value, held within +-65440
 *   m = binary16(lo), s = binary16(fp32(hi - m) / 15)
 *   code = (x - m) / s rounded to the nearest of 0 .. 15, ties to even; 0 where s is 0.
 * A group with a value that is not finite gets s = m = NaN: it stands for NaN as a
 * whole. q is turned as q4_rotary_apply does. Tokens and heads lie at most 2^31 - 1 values
 * apart. k, v, q, q_out, slots and positions must not
 * overlap the cache (Q4_ERR_INVALID_ARG).
 */
q4_status q4_cache4_append(const q4_cache4* c, const uint16_t* k, int64_t k_token, int64_t k_head, const uint16_t* v,
                           int64_t v_token, int64_t v_head, const void* slots, int slot_bits, int tokens,
                           const q4_rotary* rotary, const void* positions, int position_bits, const uint16_t* q,
                           int64_t q_token, int64_t q_head, uint16_t* q_out, int64_t out_token, int64_t out_head,
                           int heads, int bf16, hipStream_t stream);

/*
 * q4_cache4_read -- the keys and values that rows slots[t] stand for, in binary16;
 * zeros for a slot outside the cache. k and v must not overlap each other, the cache or
 * the slots.
 */
q4_status q4_cache4_read(const q4_cache4* c, const void* slots, int slot_bits, int tokens, uint16_t* k, int64_t k_token,
                         int64_t k_head, uint16_t* v, int64_t v_token, int64_t v_head, hipStream_t stream);

/*
 * q4_attend4 -- q4_attend_ex over the values that a cache held in 4 bits stands for;
 * q and out are binary16 or (bf16 != 0) bfloat16. Both products take those
 * binary16 values as they are; queries of bfloat16 are brought into binary16 by a power
 * of two a row (values below 2^-31 of the row's largest lose bits), and the weights are
 * rounded to binary16 whatever the type. A group whose codes 0 or 15 stand for a value that is
 * not finite (q4_cache4_append makes none but NaN as a whole) may count as NaN as a
 * whole. The workspace is as for q4_attend.
 */
size_t q4_attend4_workspace(const q4_cache4* c, int heads);

/* The workspace with which a call of these sizes is fastest (any from q4_attend4_workspace on will
 * do), at least that of q4_attend4_workspace: chunks of some thousand rows (tokens times heads of a group) a request on average
 * and more bring the keys and values into binary16 there first, if they take no more than 2^30
 * bytes (2 dim a row and side, of requests * table_width pages). */
size_t q4_attend4_workspace_for(const q4_cache4* c, int heads, int tokens, int requests, int table_width);
q4_status q4_attend4(const q4_cache4* c, const uint16_t* q, int64_t q_token, int64_t q_head, int heads, int tokens,
                     const int32_t* starts, const int32_t* lengths, const int32_t* table, int table_width,
                     int64_t table_stride, int requests, int window, int sinks, float scale, uint16_t* out,
                     int64_t out_token, int64_t out_head, void* workspace, size_t workspace_bytes, int bf16,
                     hipStream_t stream);

/* ------------------------------------------------------------------------
 * The pages of a cache, of either kind.
 * ---------------------------------------------------------------------- */

/*
 * One tensor of a cache: of each page `heads` heads of `rows` rows of `bytes` dense
 * bytes, row r of head h of page p at `at` + p page + h head + r row (strides in bytes,
 * non-negative), 2^30 of them a page at most. A pool is the one to four tensors of a cache.
 */
typedef struct {
    void* at;
    int64_t page, head, row;
    int heads, rows, bytes;
} q4_plane;
typedef struct {
    q4_plane plane[4];
    int planes, pages;
} q4_pool;

/*
 * q4_copy_pages -- page dst[i] becomes a copy of page src[i], in all tensors of the
 * pool, for i < n. src and dst are device integers of 32 or 64 bits; a pair with one outside
 * [0, pages) is left out. The pages of dst must differ from each other and from those of src
 * (a mixture may be left); indexes must not overlap the cache.
 */
q4_status q4_copy_pages(const q4_pool* pool, const void* src, int src_bits, const void* dst, int dst_bits, int n,
                        hipStream_t stream);

/*
 * Which pages hold which request's tokens, as dense device arrays of the caller's. Request r
 * has lengths[r] tokens, in pages table[r width + i] for i < ceil(lengths[r] /
 * page_size) (an entry outside [0, pages) names none). counts[p] is the number of
 * those entries that name page p; a page whose count is not positive is free. work is
 * scratch of q4_pages_workspace(requests, pages) bytes; calls that share the arrays are ordered
 * on one stream. Nothing waits for the device, every call may be captured, and results do
 * not depend on the order in which anything runs. The arrays, a call's indexes and its output must
 * not overlap each other or the cache (Q4_ERR_INVALID_ARG; indexes may overlap indexes).
 */
typedef struct {
    int32_t* table;
    int32_t* lengths;
    int32_t* counts;
    int32_t* work;
    int requests, width, pages, page_size;
} q4_pages;

size_t q4_pages_workspace(int requests, int pages);

/*
 * q4_pages_extend -- room for new tokens: request r gets starts[r + 1] - starts[r] more
 * (starts: requests + 1 values from 0 to `tokens`, as in q4_attend), the lowest free pages for
 * them where its last one does not suffice, in the order of the requests, and slots[t] is where
 * token t goes (as q4_cache_append takes it). A request whose table row is too short gets
 * nothing; one that the free pages do not suffice for gets nothing either, nor does any after it
 * that needs some: lengths stay, slots are -1. (One that needs none is served. Tokens without a slot are not
 * in the cache: the caller leaves them out of what follows, q4_attend would take them for its last ones.)
 */
q4_status q4_pages_extend(const q4_pages* pages, const int32_t* starts, int tokens, int32_t* slots, hipStream_t stream);

/*
 * q4_pages_fork -- for i < n, request children[i] becomes a copy of request parents[i]: its
 * pages are the same ones but the last, which is copied to the lowest free page where it is not
 * full, so that both go on in their own. done[i] is 1, or 0 for a pair with an index outside
 * [0, requests), a child that holds tokens or that an earlier pair names, and one for which no
 * free page is left. All pairs see the requests as they were before the call. done has room
 * for 2 n values (the second n are scratch). pool describes the cache, pool->pages = pages.
 */
q4_status q4_pages_fork(const q4_pages* pages, const q4_pool* pool, const void* parents, int parent_bits, const void* children,
                        int child_bits, int n, int32_t* done, hipStream_t stream);

/*
 * q4_pages_free -- gives back the pages of n requests (one named twice is freed once): their
 * lengths are 0 and their entries -1.
 */
q4_status q4_pages_free(const q4_pages* pages, const void* requests, int bits, int n, hipStream_t stream);

/*
 * q4_pages_trim -- gives back the pages that no token after the present ones sees anything of,
 * with a window >= 1 and sinks as in q4_attend_ex; their entries are -1. (Tokens that are in the
 * cache but have not been attended for yet still need theirs: trim after that.)
 */
q4_status q4_pages_trim(const q4_pages* pages, int window, int sinks, hipStream_t stream);

/*
 * q4_pages_compact -- moves pages so that the U in use are pages 0 .. U - 1: the k-th one in use
 * from page U on goes to the k-th free page below it. Tables and counts follow; to[p] is
 * where page p went, -1 for one that was free.
 */
q4_status q4_pages_compact(const q4_pages* pages, const q4_pool* pool, int32_t* to, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Adapters of many requests beside one quantized product.
 * ---------------------------------------------------------------------- */

typedef struct q4_adapters q4_adapters;   /* opaque bank of slots */

/* The argument checks of q4_adapters_make that need no device: 1 .. 4096
 * slots, rank 1 .. 1024. */
q4_status q4_check_adapters(int slots, int rank);

/*
 * q4_adapters_make -- a bank of `slots` adapters of rank at most `rank` for
 * handle h, in binary16 or (bf16 != 0) bfloat16, on h's device (the current
 * one). Every slot is empty (adds nothing). The bank holds slots * (parts * rank *
 * K + N rounded up to 32 * rank rounded up to 8) values and the workspace of its calls:
 * once M passes Q4_GEMV_MAX_M, 2 MiB and, a row, 16 bytes and 4 for each part and value of
 * rank (rounded up to 8; in binary16 4 more for each part and 64 of rank). Rows come in 256s and at least double as M grows; what is
 * outgrown stays until the bank is freed, which is at most as much again. It does not
 * keep h. NULL on error.
 */
q4_adapters* q4_adapters_make(const q4_matrix* h, int slots, int rank, int bf16);
/* q4_adapters_free -- NULL allowed; the caller has synchronized its streams. */
void q4_adapters_free(q4_adapters* a);

/*
 * q4_adapters_load -- copy an adapter of `rank` (at most the bank's) into a slot,
 * in `stream`'s order: A [parts][rank][K] (a part for each layer the handle
 * concatenates, K in the checkpoint's order), B [N][rank], factor c.
 * q4_adapters_clear empties a slot.
 */
q4_status q4_adapters_load(q4_adapters* a, int slot, const uint16_t* A, const uint16_t* B, int rank, float c,
                           hipStream_t stream);
q4_status q4_adapters_clear(q4_adapters* a, int slot, hipStream_t stream);

/*
 * q4_matmul_adapters -- q4_matmul_bias / q4_matmul_bf16 with the adapters of
 * the rows' requests:
 *   out[m][n] = (x[m] W)[n] + bias[n] + sum_j B[n][j] (c sum_k A[p][j][k] x[m][k])
 * with A, B, c of slot index[m] and p the part of column n; an index outside
 * [0, slots) (-1) adds nothing. index is int32 [M] on the device. fp32 sums, one
 * rounding of the result. Up to Q4_GEMV_MAX_M rows c A x is kept in fp32; above, as
 * two values of the activations' type (its rounding and the rest): off by 2^-16 of itself
 * in bfloat16, in binary16 by 2^-22 of itself or 2^-16 of the largest of 64 values of its
 * row and part (which a power of two brings into the type's reach). Rows of other adapters,
 * or of none, are not touched by one's values that are not finite.
 *
 * Errors, graph capture and concurrency as q4_matmul, for the handle and the bank alike: a
 * bank's workspace for M > Q4_GEMV_MAX_M grows on the first call with a larger
 * M, which cannot be captured, and calls on one bank are ordered on one stream. (A call is
 * several launches; those of two host threads on one stream and one bank follow each other.)
 */
q4_status q4_matmul_adapters(const q4_matrix* h, q4_adapters* bank, const uint16_t* x, const uint16_t* bias,
                             const int32_t* index, uint16_t* out, int M, int bf16, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_H */
