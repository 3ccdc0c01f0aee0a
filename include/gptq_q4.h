/*
 * gptq_q4.h -- C ABI of the GB300 (sm_103a) fused GPTQ W4A16 linear layer.
 *
 *     y[M][N] = x[M][K] . W[K][N] + bias[N]
 *
 * W is a GPTQ (v1) 4-bit weight matrix:
 *   qweight  int32 [K/8][N]   eight 4-bit codes per word along K, code k%8 in
 *                             bits 4(k%8) .. 4(k%8)+3 (lowest nibble first)
 *   qzeros   int32 [G][N/8]   eight 4-bit zero points per word along N, same
 *                             nibble order
 *   scales   fp16  [G][N]     one scale per (group, column)
 *   g_idx    int32 [K]        group of each row (act-order), or NULL
 *   w[k][n] = scales[g][n] * (q[k][n] - (z[g][n] + 1)),  g = g_idx[k]
 *             (g = k / groupsize when g_idx is NULL; G = K / groupsize, or
 *              G = 1 and one group over all of K when groupsize == -1)
 *
 * Sources (web pages; sections named):
 *   "GPTQ's 'Exllama Kernel Not Installed' Warning" -- "Why the kernel is
 *     missing" (4-bit integers packed in 32-bit words, a scale and a zero per
 *     group) and "What the fallback actually does" (the fused kernel reads
 *     packed weights, dequantizes in registers and never writes a dequantized
 *     matrix; the fallback rebuilds W and runs an ordinary matmul, reaching the
 *     same answer with several times the memory traffic).
 *   "Implementation: Predibase Lorax GPTQ Exllama V1" -- "Description" (a
 *     Q4Matrix handle built from qweight, qzeros, scales and optional g_idx;
 *     q4_matmul computes x @ q4 into a (batch, width) fp16 output; temp_state
 *     reorders activations for act-order; temp_dq holds dequantized weights
 *     for the prefill matmul; create_exllama_buffers sizes both) and "I/O
 *     Contract" (dtypes; bits must be 4; None or trivial g_idx = no act-order).
 *   "Inference Backends" -- "Packing, conversion, and runtime initialization"
 *     (runtime init repacks into a private execution layout and builds native
 *     handles), "Numeric epilogues and input gradients" (bias joins the fp32
 *     accumulator before the one final cast; split reductions stay fp32;
 *     no atomic partial-output reduction), "Strided tensor operands" (one
 *     stable argsort gives the reorder; an identity permutation skips the
 *     gather), "Runtime cache lifetime" (no dense weight cache is kept
 *     between operations).
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" must be CUDA device (or managed) memory of the
 *     device that is current when the call is made; "host" means host memory.
 *     Arrays are dense and row-major; fp16 values are passed as their 16-bit
 *     patterns (uint16_t).
 *   - Every call except gptq_q4_make returns GPTQ_Q4_OK (0) or a negative
 *     status.  gptq_q4_make returns NULL on failure.  The status and a message
 *     with the specific reason are kept per host thread and read back with
 *     gptq_q4_last_status() / gptq_q4_last_error().  Nothing is ever printed,
 *     and no call silently falls back to another route: there is no CPU path.
 *   - Work is enqueued on the caller's stream and the calls return without
 *     waiting, except gptq_q4_make, gptq_q4_reserve, gptq_q4_free and
 *     gptq_q4_device_error, which synchronize as stated.
 *   - A handle may be used from one stream at a time (its workspaces are
 *     reused by every call).  Distinct handles are independent.
 *   - A work buffer that a call outgrows is replaced by one of at least twice
 *     its size (where there is room), by stream order; on a capturing stream by
 *     an ordinary allocation, which is no part of the graph.  The replaced ones
 *     stay allocated until the handle is freed, so that graphs captured before
 *     go on running; they add up to no more than the present buffer.
 */
#ifndef GPTQ_Q4_H
#define GPTQ_Q4_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ status codes */
#define GPTQ_Q4_OK                 0
#define GPTQ_Q4_INVALID_ARGUMENT (-1) /* NULL, bad sizes, g_idx out of range, misalignment */
#define GPTQ_Q4_UNSUPPORTED      (-2) /* valid GPTQ data outside what the GPU kernels take,
                                         or a device that is not sm_103 */
#define GPTQ_Q4_CUDA_ERROR       (-3) /* a CUDA runtime call failed; message holds its text */
#define GPTQ_Q4_OUT_OF_MEMORY    (-4) /* a device allocation failed */
#define GPTQ_Q4_DEVICE_FAULT     (-5) /* a kernel reported an error through its status word */

/* Paths gptq_q4_matmul can take (see gptq_q4_set_path). */
#define GPTQ_Q4_PATH_AUTO      0  /* decode below the prefill threshold, fused prefill above */
#define GPTQ_Q4_PATH_DECODE    1  /* always decode: the stream-K kernel on tall layers of 100 Mi
                                     weights or more that the column tiles cannot fill (K >= 2 N,
                                     fewer than two 32-column tiles per SM) at M = 1 with groups of
                                     at most 128 rows, at M = 2 with 32-row groups and at M = 3..8
                                     with groups of 128 rows or more; otherwise the
                                     register-streaming kernel at M <= 4, at M <= 8 on layers below
                                     64 Mi weights or with groups of at most 64 rows, and on any
                                     layer below 24 Mi weights; the TMA-ring kernel (M <= 16)
                                     elsewhere, where the shape allows it */
#define GPTQ_Q4_PATH_PREFILL   2  /* always the fused shared-memory-dequant tensor-core kernel */
#define GPTQ_Q4_PATH_DECODE_MMA 3 /* always the register-streaming decode kernel */
#define GPTQ_Q4_PATH_DECODE_TC 4  /* decode on tcgen05 with one tensor-memory accumulator per
                                     quantization group (M <= 16 on 4-bit handles with fp16
                                     activations; otherwise as GPTQ_Q4_PATH_DECODE) */
#define GPTQ_Q4_PATH_DECODE_RING 5 /* the TMA-ring decode kernel whenever the shape allows it
                                      (M <= 16, a K slice within 48 groups), else
                                      register-streaming */
#define GPTQ_Q4_PATH_DECODE_STREAM 6 /* the stream-K decode kernel (M <= 8): every warp of the
                                        grid streams an equal run of 32-column x 64-row units,
                                        quantization groups ride in the MMAs' spare columns;
                                        larger M as GPTQ_Q4_PATH_DECODE */

typedef struct gptq_q4_s *gptq_q4_handle;   /* opaque; owns device memory */

/* Build a handle (the Q4Matrix of the Lorax page's "Description": make_q4).
 *
 *   qweight  device int32 [K/8][N]
 *   qzeros   device int32 [G][N/8]
 *   scales   device fp16  [G][N]
 *   g_idx    device int32 [K], or NULL for the trivial map k / groupsize
 *   groupsize  > 0 dividing K, or -1 for one group over all of K
 *
 * Validates the arguments; copies g_idx to the host, checks every entry is in
 * [0, G), and derives the act-order row permutation P with one stable argsort
 * (rows sorted by group, original order kept within a group).  An identity P
 * means no act-order.  When the groups do not all hold the same whole number
 * of 32-row blocks (g_idx with groups of unequal size, or a groupsize that is
 * not a multiple of 32), every group is padded to the largest one rounded up
 * to 32 rows: the padding rows hold code 0 and P = -1, and the activation
 * gather writes 0 for them, so they add nothing to y.  Then repacks the codes,
 * in P order, into a private tile-ordered layout (same byte count as qweight
 * without padding), and the scales into a private pairing; zero points keep
 * the checkpoint layout.  All of it is
 * copied into handle-owned device memory, so the caller may free or change its
 * tensors afterwards.  Also sizes the split-K workspace for M <= 16.
 * Synchronizes the device before returning.  The caller must have finished
 * writing the input tensors (e.g. synchronized its stream) before the call.
 *
 * Errors (NULL return; reason in gptq_q4_last_error):
 *   INVALID_ARGUMENT  NULL qweight/qzeros/scales, K or N <= 0, K % 8 or N % 8
 *                     != 0, groupsize not -1 and not a positive divisor of K,
 *                     a g_idx entry outside [0, G), a pointer that is not
 *                     device memory of the current device
 *   UNSUPPORTED       K % 64 or N % 64 != 0; groups whose padding to the
 *                     largest one would make the layout more than 4 x K
 *                     rows; current device is not compute 10.3
 *   OUT_OF_MEMORY, CUDA_ERROR */
gptq_q4_handle gptq_q4_make(const int32_t *qweight, const int32_t *qzeros,
                            const uint16_t *scales, const int32_t *g_idx,
                            int K, int N, int groupsize);

/* Attach (or with NULL, detach) a bias: device fp16 [N], copied into the
 * handle.  Bias is added to the fp32 accumulator before the single rounding
 * to fp16 ("Inference Backends", "Numeric epilogues and input gradients").
 * Enqueued on the legacy default stream and synchronized before returning.
 * The handle keeps one copy until it is freed: a graph captured with a bias
 * goes on adding it, or another that is attached later.
 * Errors: INVALID_ARGUMENT (NULL handle), OUT_OF_MEMORY, CUDA_ERROR. */
int gptq_q4_set_bias(gptq_q4_handle h, const uint16_t *bias);

/* Size the handle's work buffers for calls with up to max_m rows: the
 * act-order activation buffer temp_state [max_m][K] fp16 and the split-K
 * partial sums.  The counterpart of the Lorax page's create_exllama_buffers
 * (max_total_tokens).  A later gptq_q4_matmul with more rows grows the buffers
 * itself (stream-ordered allocation on the caller's stream; the smaller ones
 * stay until the handle is freed); calling this
 * first keeps allocation out of gptq_q4_matmul.  Synchronizes the device.
 * Errors: INVALID_ARGUMENT (NULL handle, max_m < 0), OUT_OF_MEMORY. */
int gptq_q4_reserve(gptq_q4_handle h, int max_m);

/* out = x . W + bias  (q4_matmul; the Lorax page's "Description").
 *
 *   x    device [M][K] of the handle's activation type (fp16 by default;
 *        bf16 or fp32 after gptq_q4_set_act_dtype), 16-byte aligned
 *   out  device [M][N] of the same type, 16-byte aligned; written entirely,
 *        never read
 *   M    rows; 0 is a valid no-op
 *
 * With act-order, x is first gathered into temp_state (temp_state[m][j] =
 * x[m][P[j]]).  Rows below the prefill threshold run one of two decode
 * kernels (GPTQ_Q4_PATH_DECODE says which).  The TMA-ring kernel (M <= 16):
 * packed-word tiles and x tiles stream through a ring of shared-memory
 * stages by TMA; each warp owns 32 columns for a whole K slice, turns code
 * pairs into fp16 with one LOP3 each and accumulates on mma.sync in fp32,
 * the zero point removed per group from MMA-accumulated sums of x; the K
 * slices of a 128-column tile (at most 8) are summed in slice order inside a
 * thread-block cluster.  The register-streaming kernel: packed weights
 * streamed with 128-bit loads, through a per-warp ring of asynchronous
 * copies in shared memory at M <= 8 (x staged once per CTA, or carried with
 * each chunk when the x slice is long) and straight into registers above,
 * exact (q - z - 1) in fp16 (or raw code pairs with per-group sums of x),
 * fp32 accumulation on mma.sync, split-K summed in a fixed order inside a
 * cluster or, past eight slices, by the last CTA to finish.
 * GPTQ_Q4_PATH_DECODE_TC selects the
 * tcgen05 decode instead (M <= 16): packed weights streamed by TMA,
 * dequantized in shared memory to the exact integers (q - z - 1), one
 * tensor-memory accumulator per quantization group, scales applied once per
 * group in an fp32 epilogue.
 * Larger M runs the fused prefill (tcgen05/TMEM with shared-memory
 * dequantization).  Results do not depend on the path beyond fp32 rounding.
 * Errors: INVALID_ARGUMENT (NULL handle/pointers with M > 0, M < 0,
 * misaligned x or out, handle made on another device), OUT_OF_MEMORY (growing
 * a work buffer), CUDA_ERROR (launch failure). */
int gptq_q4_matmul(gptq_q4_handle h, const void *x, int M, void *out,
                   cudaStream_t stream);

/* temp_dq[k][n] = fp16(scales[g][n] * (q[k][n] - (z[g][n] + 1))), rounded
 * once to nearest-even, in the ORIGINAL row order (the permutation is undone
 * on write).  The dequantized matrix of the Lorax page's "Description"
 * (temp_dq), used for debugging and by the unfused prefill comparison.
 *   temp_dq  device fp16 [K][N], 16-byte aligned, caller-owned: the handle
 *            keeps no dense copy ("Runtime cache lifetime").
 * Errors: INVALID_ARGUMENT, CUDA_ERROR. */
int gptq_q4_dequant(gptq_q4_handle h, uint16_t *temp_dq, cudaStream_t stream);

/* The unpacked codes, read back from the handle's private layout (a debug
 * read-back; no passage of the pages defines it: "Inference Backends",
 * "Packing, conversion, and runtime initialization" only says runtime
 * initialization may repack into a private layout, and this call shows that
 * the repack kept every code):
 *   q  device uint8 [K][N], q[k][n] in 0..15, ORIGINAL row order
 *   z  device uint8 [G][N], stored zero points (without the +1)
 * Either pointer may be NULL to skip it.  For checking the repack bit-exactly.
 * Errors: INVALID_ARGUMENT, CUDA_ERROR. */
int gptq_q4_debug_unpack(gptq_q4_handle h, uint8_t *q, uint8_t *z, cudaStream_t stream);

/* The unfused comparison route ("What the fallback actually does", with the
 * matmul on the tensor cores): gptq_q4_dequant into the caller's temp_dq, then
 * out = x . temp_dq + bias by the tcgen05 GEMM below.  Same arguments as
 * gptq_q4_matmul plus temp_dq (device fp16 [K][N], caller-owned scratch).
 * Errors: as gptq_q4_matmul and gptq_q4_dequant. */
int gptq_q4_matmul_unfused(gptq_q4_handle h, const void *x, int M,
                           uint16_t *temp_dq, void *out, cudaStream_t stream);

/* Dense fp16 GEMM on the 5th-generation tensor cores (tcgen05, accumulators
 * in tensor memory, operands staged by TMA): out = a . b + bias with fp32
 * accumulation and one rounding to fp16.  The matmul the Lorax page runs on
 * temp_dq "during prefill".
 *   a     device fp16 [M][K] row-major, b device fp16 [K][N] row-major,
 *   bias  device fp16 [N] or NULL, out device fp16 [M][N];
 *   all 16-byte aligned; K % 64 == 0, N % 64 == 0, M >= 0.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (sizes), CUDA_ERROR. */
int gptq_q4_gemm_f16(const uint16_t *a, const uint16_t *b, const uint16_t *bias,
                     int M, int K, int N, uint16_t *out, cudaStream_t stream);

/* Bytes of the fixed device scratch used by gptq_q4_matmul_noalloc (16 MiB). */
#define GPTQ_Q4_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

/* out = x . W + bias through the decode kernel, allocating nothing.
 *
 * The web pages this library follows have no counterpart for this call.  It
 * is for callers that cannot allocate device memory while they run a layer:
 * a plugin inside a framework that owns all device memory, a service whose
 * device memory is budgeted in full up front, a loop that must never hit
 * cudaMalloc/cudaFree (which can synchronize the device).  gptq_q4_matmul may
 * grow the handle's work buffers; this call never allocates or frees.
 *
 * It runs the decode kernel (any M) with its scratch -- split-K partial sums,
 * per-tile tickets and, for act-order, temp_state -- taken from one static
 * device array of GPTQ_Q4_NOALLOC_SCRATCH_BYTES bytes that every GPU loading
 * the library holds until the process exits.  Arguments, layouts and results
 * are those of gptq_q4_matmul (x, out: device fp16, 16-byte aligned).
 *
 *   - The first call in each CUDA context does a one-time set-up: it looks
 *     up the array's device address with cudaGetSymbolAddress, with the
 *     handle's device current, and keeps it keyed by the context's unique ID
 *     (the primary context, or one the caller made current).  A context made
 *     after cudaDeviceReset is a new context and gets its own set-up.  Make
 *     the first call in a context before any stream capture.
 *   - All calls share the one array, which keeps the last call's contents;
 *     the call clears what must start at zero (the tickets) on its stream.
 *     Calls that overlap on the GPU (other streams, other handles, other
 *     threads) race on the array: order them, e.g. use one stream.
 *   - Errors: as gptq_q4_matmul, plus INVALID_ARGUMENT when M (with this
 *     layer's K and N) would need more scratch than the array holds; the
 *     message gives both sizes. */
int gptq_q4_matmul_noalloc(gptq_q4_handle h, const uint16_t *x, int M, uint16_t *out,
                           cudaStream_t stream);

/* Force a path for gptq_q4_matmul (tests, benchmarks): GPTQ_Q4_PATH_*. */
int gptq_q4_set_path(gptq_q4_handle h, int path);

/* GPU packer ("Inference Backends", "Packing, conversion, and runtime
 * initialization": packing takes the original layer's weights with the
 * quantizer's scales, zeros and optional act-order index; a GPU path does the
 * packing math; symmetric modules without zeros use 2^(bits-1)).
 *   w       dev [K][N] fp16, the float weights (row k = input feature k)
 *   scales  dev [G][N] fp16
 *   zeros   dev [G][N] int32 effective zero points (0..15), or NULL: all 8
 *   g_idx   dev [K] int32 group of each row, or NULL: k / groupsize
 *   format  GPTQ_Q4_FORMAT_GPTQ (stores z - 1) or GPTQ_Q4_FORMAT_GPTQ_V2 (z)
 *   qweight dev [K/8][N] int32 out, qzeros dev [G][N/8] int32 out
 * Code q = clamp(rint(w / s) + z, 0, 15) with w / s the IEEE binary32
 * quotient, ties to even (0/0 gives z); qweight and qzeros in the
 * checkpoint layout gptq_q4_make reads; stored zeros are taken mod 16.
 * Asynchronous on `stream` once its arguments are checked (g_idx is copied to
 * the host for the range check).  Errors: INVALID_ARGUMENT (NULL, sizes,
 * groupsize, format, g_idx out of [0, G), non-device pointers), CUDA_ERROR. */
int gptq_q4_pack(const uint16_t *w, const uint16_t *scales, const int32_t *zeros, const int32_t *g_idx, int K,
                 int N, int groupsize, int format, int32_t *qweight, int32_t *qzeros, cudaStream_t stream);

/* Test hook for failure detection (the pages have no counterpart).  The TMA
 * and tcgen05 kernels bound every mbarrier wait: a wait that runs out sets
 * a bit in the handle's status word (reported by gptq_q4_device_error) and
 * the kernel returns instead of hanging.  This launches one CTA whose thread
 * runs that same wait, limited to limit_us microseconds (1 .. 2,000,000), on
 * an mbarrier that nothing arrives at; when the limit runs out it ORs 1 into
 * *status (a device int the caller owns and zeroes).  Asynchronous on
 * `stream`.  Errors: INVALID_ARGUMENT (NULL status, limit out of range),
 * CUDA_ERROR (launch). */
int gptq_q4_debug_wait_probe(int *status, unsigned limit_us, cudaStream_t stream);

/* Test hook, host only (no device call): the work split that the fused
 * prefill ("Inference Backends", "How AUTO selection works": the prefill
 * path for larger M) plans for an M x K x N call on a GPU with `sms` SMs.
 * out[0..6] (caller-owned host ints) = tile rows BM, tile columns BN,
 * stream-K (1) or whole tiles round robin (0), CTAs of the stream-K launch
 * (0 for round robin), the most pieces any tile is cut into, whether each
 * cut tile is finished by the CTA holding its first k blocks (1) or by every
 * piece's CTA, a share of the rows each (0), and the rows of K per pipeline
 * stage (64, or 128).  Errors: INVALID_ARGUMENT
 * (NULL out, M < 1, K or N not a positive multiple of 64, sms < 1). */
int gptq_q4_debug_prefill_plan(int M, int K, int N, int sms, int *out);

/* Test hook, host only (no device call): the kernel that gptq_q4_matmul runs
 * for M fp16 rows on a K x N layer with this group size (-1: one group; no
 * padding, GPTQ zero points), with `path` as the handle's
 * GPTQ_Q4_PATH_* setting (AUTO resolved by the default prefill threshold)
 * on a GPU with `sms` SMs.  *kernel (caller-owned host int) = 0 the fused
 * prefill, 1 the register-streaming decode, 2 the stream-K decode, 3 the
 * TMA-ring decode, 4 the tcgen05 decode.  Errors: INVALID_ARGUMENT (NULL
 * kernel, M < 1, K or N not a positive multiple of 64, a group size that is
 * not -1 or a multiple of 32 dividing K, sms < 1, an unknown path). */
int gptq_q4_debug_dispatch(int M, int K, int N, int groupsize, int path, int sms, int *kernel);

/* Projection fusion ("Inference Backends", "How AUTO selection works":
 * post-quantization QKV or gate/up projections that read the same input are
 * combined into one call).  One handle over `parts` GPTQ layers that share
 * K, groupsize and g_idx, concatenated along N in the given order:
 *   qweight[i] dev [K/8][N[i]], qzeros[i] dev [G][N[i]/8], scales[i] dev
 *   [G][N[i]] fp16, N[i] a positive multiple of 8, sum of N[i] a multiple of
 *   64 (the handle's N); g_idx as for gptq_q4_make, shared by all parts.
 * gptq_q4_matmul on the handle writes out [M][sum N[i]]: part i occupies
 * columns [sum_{j<i} N[j], + N[i]) of each row (views of one buffer, no copy);
 * a bias set with gptq_q4_set_bias is the parts' biases concatenated the same
 * way.  The parts' tensors are copied; the caller may free them on return.
 * Returns NULL on error (status and message as for gptq_q4_make). */
#define GPTQ_Q4_MAX_FUSED_PARTS 16
gptq_q4_handle gptq_q4_make_fused(int parts, const int32_t *const *qweight, const int32_t *const *qzeros,
                                  const uint16_t *const *scales, const int32_t *g_idx, int K, const int *N,
                                  int groupsize);

/* Checkpoint zero-point convention of a handle ("Inference Backends",
 * "Concepts": GPTQ and GPTQ_V2 are distinct checkpoint formats).  The two
 * store qweight, qzeros and scales in the same layout and differ in the
 * zero point: GPTQ keeps z_eff - 1 in qzeros, so w = s * (q - (z + 1));
 * GPTQ_V2 keeps z_eff itself, so w = s * (q - z).  Default GPTQ.  Changes
 * what later matmul/dequant calls compute; the handle's other state is
 * untouched.  Errors: INVALID_ARGUMENT (NULL handle, unknown format). */
#define GPTQ_Q4_FORMAT_GPTQ    0
#define GPTQ_Q4_FORMAT_GPTQ_V2 1
int gptq_q4_set_format(gptq_q4_handle h, int format);

/* Type of x and out for later matmul calls on this handle ("Inference
 * Backends", "Hardware, dependency, and format requirements": the ExLlama v2
 * row declares FP16/BF16/FP32 activation dtypes, keeps the activation/output
 * dtype, fp16 scales and fp32 accumulation).  Default FP16.  bias stays the
 * handle's fp16.
 *   BF16: x and out are bf16 [M][K] / [M][N]; every row of x is first scaled
 *     by a power of two 2^-e (its largest magnitude times 2^-e in [2^14,
 *     2^15)) and rounded once to fp16 (exact for values within ~2^28 of the
 *     row's largest: bf16 has an 8-bit significand), the fp16 kernels run
 *     unchanged, and each output is acc * 2^e + bias rounded once to bf16.
 *     Covers gptq_q4_matmul, gptq_q4_matmul_unfused and
 *     gptq_q4_matmul_noalloc; one extra launch per call prepares x (fused
 *     with the act-order gather).
 *   FP32: x and out are fp32 [M][K] / [M][N]; every row is scaled by 2^-e
 *     as above and split into two fp16 rows, hi = fp16(v) and lo = fp16(v -
 *     hi) (v - hi is exact, so hi + lo carries v to about 2^-22 of itself);
 *     the fp16 kernels run on the 2M rows and write their raw fp32 sums, and
 *     a last launch forms out = (sum_hi + sum_lo) * 2^e + bias in fp32 (no
 *     rounding to a narrower type).  Covers gptq_q4_matmul and
 *     gptq_q4_matmul_unfused (two extra launches per call);
 *     gptq_q4_matmul_noalloc returns UNSUPPORTED for an FP32 handle.
 * Errors: INVALID_ARGUMENT (NULL handle, unknown dtype). */
#define GPTQ_Q4_DTYPE_FP16 0
#define GPTQ_Q4_DTYPE_BF16 1
#define GPTQ_Q4_DTYPE_FP32 2
int gptq_q4_set_act_dtype(gptq_q4_handle h, int dtype);

/* Rows at and above which GPTQ_Q4_PATH_AUTO takes the prefill kernel (the
 * decode/prefill switch of the Lorax page's set_tuning_params).  Default 17,
 * or 9 for groups of at most 32 rows and for groups of at most 64 rows on
 * layers of 100 Mi weights or more: measured on GB300, the fused prefill is
 * faster than the decode kernels from there.  Results never depend on it. */
int gptq_q4_set_prefill_min_m(gptq_q4_handle h, int min_m);

/* Facts about a handle (host outputs; any pointer may be NULL). */
int gptq_q4_info(gptq_q4_handle h, int *K, int *N, int *groupsize, int *G,
                 int *act_order, size_t *device_bytes);

/* Synchronize the handle's device and return GPTQ_Q4_DEVICE_FAULT if any
 * kernel of this handle has set its status word (a bounded wait that ran out,
 * a failed internal check), else GPTQ_Q4_OK.  Clears the word. */
int gptq_q4_device_error(gptq_q4_handle h);

/* Release everything the handle owns (waits for its device; ends no stream
 * capture).  NULL is a no-op.  Lifecycle only; the pages' nearest passage is "Inference
 * Backends", "Runtime cache lifetime" (native runtime storage belongs to the
 * handle, and nothing outlives it). */
void gptq_q4_free(gptq_q4_handle h);

/* Q4Matrix handle for an 8-bit GPTQ layer.  "Inference Backends",
 * "Hardware, dependency, and format requirements": the GPTQ Marlin row
 * declares bits 4 and 8, and the Swordfish row says GPTQ supports 4/8-bit.
 * The pages print no 8-bit layout; this library reads it as the 4-bit
 * GPTQ packing with 32 / 8 = 4 codes per int32:
 *   qweight  device int32 [K/4][N]   four 8-bit codes per word along K,
 *                                   lowest byte = lowest row
 *   qzeros   device int32 [G][N/4]   four 8-bit zero points per word along N
 *   scales   device fp16  [G][N], |scale| < 4094
 *   g_idx, groupsize as for gptq_q4_make
 * w[k][n] = scales[g][n] * (q[k][n] - (z[g][n] + 1)) (GPTQ; GPTQ_V2 after
 * gptq_q4_set_format: q - z).  With q = 16 qh + ql and z = 16 zh + zl,
 * s (q - z - 1) = 16 s (qh - zh) + s (ql - zl - 1) exactly, so the handle
 * holds a 4-bit layer over 2K rows (the high nibbles with scale 16 s and zero
 * offset 0, then the low nibbles with scale s) whose two halves read the same
 * column of x; every matmul path, gptq_q4_dequant and gptq_q4_debug_unpack
 * (8-bit codes and zero points, one byte each) work as for 4-bit handles,
 * with twice the packed bytes.  gptq_q4_info reports the caller's K and G.
 * Errors as for gptq_q4_make. */
gptq_q4_handle gptq_q4_make8(const int32_t *qweight, const int32_t *qzeros,
                             const uint16_t *scales, const int32_t *g_idx,
                             int K, int N, int groupsize);

/* ------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection.
 *
 *     out[m] = y[m] + scale_a * (x[m] . A_a^T) . B_a^T,   a = row_slot[m]
 *
 * A pool holds up to `slots` adapters of one projection (K inputs, N
 * outputs), each with its own rank; every row of a call names the slot of its
 * adapter, or a negative number for none.  x and y are the projection's input
 * and output (gptq_q4_matmul), so one call adds every request's adapter to
 * the shared product.  For one part of a fused projection, pass that part's
 * columns of y and out with the fused row strides.
 *
 * A pool may be used from one stream at a time (gptq_q4_lora_set and _add
 * are ordered by the streams they are enqueued on; the sums x . A^T live in
 * the pool's workspace). */
typedef struct gptq_q4_lora_s *gptq_q4_lora;

/* An empty pool.  dtype: GPTQ_Q4_DTYPE_FP16 or _BF16, the type of x, y, out,
 * A and B.  K and N positive multiples of 8, 1 <= slots <= 4096,
 * 1 <= max_rank <= 256.  Device memory: slots * ceil16(max_rank) * (ceil64(K) + N)
 * 16-bit values.  Synchronizes.  NULL on error (status and message as for
 * gptq_q4_make): INVALID_ARGUMENT, UNSUPPORTED (device not sm_103, fp32),
 * OUT_OF_MEMORY, CUDA_ERROR. */
gptq_q4_lora gptq_q4_lora_make(int K, int N, int slots, int max_rank, int dtype);

/* Put an adapter into a slot (it replaces the slot's last one):
 *   a  device [rank][K], b  device [N][rank], dense, of the pool's type;
 *   rank 0 with NULL a and b empties the slot.
 * Copied on `stream`; the caller may change a and b once the stream has
 * passed this call.  Errors: INVALID_ARGUMENT (NULL, slot or rank out of
 * range, non-device pointers), CUDA_ERROR. */
int gptq_q4_lora_set(gptq_q4_lora h, int slot, const void *a, const void *b, int rank, float scale,
                     cudaStream_t stream);

/* Size the workspace for calls with up to max_m rows.  A later call with more
 * rows replaces it by a larger one, by stream order (on a capturing stream by
 * an ordinary allocation, which is no part of the graph).  A workspace that was
 * replaced stays allocated until the pool is freed, so a graph captured before
 * goes on running; the replaced ones of such calls add up to no more than the
 * present one.  Synchronizes.  Errors: INVALID_ARGUMENT, OUT_OF_MEMORY. */
int gptq_q4_lora_reserve(gptq_q4_lora h, int max_m);

/* out = y + the adapters' part, as above.
 *   x         device [M][K], row stride x_stride elements
 *   row_slot  device int32 [M]: the row's slot; negative or an empty slot: out = y.
 *             An entry >= slots counts as none and is reported by gptq_q4_lora_device_error
 *   y, out    device [M][N], row strides y_stride, out_stride; out may be y itself
 *             (same stride), and must not overlap x or otherwise overlap y
 * Pointers 16-byte aligned, strides multiples of 8 and at least the row's
 * length; M = 0 is a no-op.  Sums are fp32 and the output is rounded once;
 * x . A^T goes into its product with B as two 16-bit parts, which hold it to
 * 2^-16 (bf16) or 2^-22 (fp16) of itself.  Infinities and NaN in x, y or an
 * adapter reach the rows that they belong to and no other.  Errors:
 * INVALID_ARGUMENT, OUT_OF_MEMORY (growing the workspace), CUDA_ERROR. */
int gptq_q4_lora_add(gptq_q4_lora h, const void *x, int64_t x_stride, const int32_t *row_slot, int M, const void *y,
                     int64_t y_stride, void *out, int64_t out_stride, cudaStream_t stream);

/* As gptq_q4_device_error and gptq_q4_free, for a pool. */
int gptq_q4_lora_device_error(gptq_q4_lora h);
void gptq_q4_lora_free(gptq_q4_lora h);

/* ------------------------------------------------------------------------
 * Rotary positions, a paged cache, and attention over it: what lies between
 * a decoder layer's fused QKV projection and its output projection.
 *
 * One handle serves all layers of a model: it holds the table of rotary
 * cosines and sines, a fixed workspace, and the status word.  It may be used
 * from one stream at a time.
 *
 * The cache of one layer: keys and values in pages of page_size tokens,
 *   k, v  device [pages][kv_heads][page_size][head_dim], 16-byte aligned;
 *         page_stride elements from page to page (at least
 *         kv_heads * page_size * head_dim, a multiple of 8). */
typedef struct {
    void *k, *v;
    int pages;
    int64_t page_stride;
} gptq_q4_cache;

/* The requests of one step.  Request b has q_len = cu_q[b+1] - cu_q[b] new
 * tokens, rows cu_q[b] .. cu_q[b+1]-1 of the step's `tokens` rows, and
 * kv_len[b] tokens in the cache, the new ones (its last q_len) among them:
 * new token t has index kv_len - q_len + t in the request's context.  Token j
 * lies in page table[b][j / page_size], at j % page_size.
 *   cu_q   device int32 [batch + 1], ascending
 *   kv_len device int32 [batch], each 0 .. width * page_size, at most 2^30
 *   table  device int32 [batch][width], table_stride elements from row to row;
 *          only entries of pages that a call reads or writes have to be valid
 *          (NULL if width is 0: contexts without a token)
 *   max_q  no request has more new tokens (a larger number is allowed and
 *          changes no result, only which kernel runs)
 * The arrays are read on the GPU when the call runs.  A length or page index
 * outside its range is cut to it (no access leaves the caller's arrays),
 * makes that request's results meaningless, and is reported by
 * gptq_q4_attn_device_error (by an append, if the request holds a row);
 * nothing is written to the cache for it. */
typedef struct {
    const int32_t *cu_q, *kv_len, *table;
    int64_t table_stride;
    int width, batch, tokens, max_q;
} gptq_q4_batch;

typedef struct gptq_q4_attn_s *gptq_q4_attn;

/* A handle for q_heads query heads that share kv_heads key/value heads
 * (q_heads a multiple of kv_heads, at most 128 query heads for each),
 * head_dim 64 or 128, page_size a power of two from 8 to 1024; dtype
 * GPTQ_Q4_DTYPE_FP16 or _BF16: the type of q, k, v and the output.
 * Synchronizes.  NULL on error: INVALID_ARGUMENT, UNSUPPORTED (head_dim,
 * page_size, fp32, device not sm_103), OUT_OF_MEMORY, CUDA_ERROR. */
gptq_q4_attn gptq_q4_attn_make(int q_heads, int kv_heads, int head_dim, int page_size, int dtype);

/* Angles per position for gptq_q4_attn_set_rope; host only, no device call.
 * inv_freq (host, rotary_dim / 2 doubles): f_i = base^(-2i / rotary_dim), then
 *   ROPE_PLAIN   as it is
 *   ROPE_LINEAR  f_i / factor
 *   ROPE_NTK     base replaced by base * factor^(rotary_dim / (rotary_dim - 2))
 *   ROPE_BANDS   with r = original * f_i / 2 pi turns over the original context and
 *                s = clamp((r - low) / (high - low), 0, 1):  s f_i + (1 - s) f_i / factor
 *   ROPE_YARN    with the pair index d(r) = rotary_dim ln(original / 2 pi r) / (2 ln base) at which a pair makes
 *                r turns, l = max(floor(d(high)), 0), h = min(ceil(d(low)), rotary_dim - 1) and
 *                s = 1 - clamp((i - l) / max(h - l, 0.001), 0, 1):  s f_i + (1 - s) f_i / factor
 * length_scale (host): what the rotated vectors are multiplied by: 1, and
 * 0.1 ln(factor) + 1 for ROPE_YARN.  factor, low, high and original are read
 * only where the formula has them.
 * Errors: INVALID_ARGUMENT (NULL, rotary_dim not even and positive, base <= 1,
 * factor < 1, high <= low, low <= 0, original < 1, unknown kind). */
#define GPTQ_Q4_ROPE_PLAIN  0
#define GPTQ_Q4_ROPE_LINEAR 1
#define GPTQ_Q4_ROPE_NTK    2
#define GPTQ_Q4_ROPE_BANDS  3
#define GPTQ_Q4_ROPE_YARN   4
int gptq_q4_rope_freqs(int rotary_dim, double base, int kind, double factor, double low, double high, int original,
                       double *inv_freq, double *length_scale);

/* Rotary positions for gptq_q4_attn_append: pair i of the first rotary_dim
 * elements of every query and key head turns by position * inv_freq[i] and
 * is multiplied by length_scale.  Pair i is elements (i, i + rotary_dim / 2),
 * or (2i, 2i + 1) if interleaved.  inv_freq: host, rotary_dim / 2 doubles.
 * Builds a table of fp32 cosines and sines for positions 0 .. max_pos - 1
 * (angles in fp64), 4 * max_pos * rotary_dim bytes.  rotary_dim: even, at most
 * head_dim, a multiple of 16; 0 turns rotation off again (the state of a new
 * handle).  The table of the same rotary_dim, interleaved and max_pos is
 * written anew in its place, and a graph captured before turns by the new
 * angles; any other table stays allocated until the handle is freed, and such
 * a graph goes on with it.  Synchronizes.  Errors: INVALID_ARGUMENT,
 * OUT_OF_MEMORY, CUDA_ERROR. */
int gptq_q4_attn_set_rope(gptq_q4_attn h, int rotary_dim, int interleaved, const double *inv_freq,
                          double length_scale, int max_pos);

/* Rotate the step's queries and keys and put keys and values into the cache.
 *   qkv        device [tokens][(q_heads + 2 kv_heads) * head_dim], row stride
 *              qkv_stride: the fused projection's output, queries, keys, values
 *   positions  device int32 [tokens], or NULL: a token's index in its context
 *   q_out      device [tokens][q_heads * head_dim], row stride q_stride, the
 *              rotated queries; may be qkv itself (same stride), else must not overlap it
 * 16-byte aligned, strides multiples of 8.  Rotation in fp32, rounded once.
 * Rows that no request owns are left alone.  A token whose index is negative
 * (kv_len < q_len, say), whose position is outside 0 .. max_pos - 1 or whose
 * page index is outside the cache is not written anywhere, nor is any token of
 * a request with a length outside its range (a kv_len past the table, say);
 * gptq_q4_attn_device_error reports either.  Errors: INVALID_ARGUMENT,
 * UNSUPPORTED (batch > 4096), CUDA_ERROR. */
int gptq_q4_attn_append(gptq_q4_attn h, const void *qkv, int64_t qkv_stride, const gptq_q4_cache *cache,
                        const gptq_q4_batch *batch, const int32_t *positions, void *q_out, int64_t q_stride,
                        cudaStream_t stream);

/* Attention of the step's new tokens over the cache:
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * over the tokens j <= i of the request's context, i = kv_len - q_len + t the
 * token's own index, and, if window > 0, j > i - window.  A row that sees
 * nothing (i < 0) gets zeros.
 *   q, out  device [tokens][q_heads * head_dim], row strides q_stride,
 *           out_stride; 16-byte aligned, strides multiples of 8, not overlapping
 * Cache slots past kv_len (and pages before the window) are not part of any
 * result, whatever they hold.  Scores, softmax and sums are fp32; each
 * weight p is rounded to 16 bits for its product with v (in fp16 one far below
 * the row's largest is off by at most 2^-32 of that); the output is rounded
 * once.  Rows that no request owns are left alone.  The order of the
 * sums depends on the lengths of the whole batch, not on timing: the same
 * call gives the same bits.  A NaN or infinity in a key reaches the rows that
 * see it.  One in a value reaches those, and may reach new tokens of the same
 * request that do not see it but share a tile with one that does (256 rows of
 * a key/value head, a row being a token for one query head): earlier ones of
 * the chunk and, with a window, later ones (their weight for it is 0, and 0
 * times it is NaN).  A call of more than 2^31
 * tiles of work (a prompt of over a million tokens at once) is not done and
 * reported by gptq_q4_attn_device_error.  Errors: INVALID_ARGUMENT (NULL, sizes, strides,
 * alignment, scale not finite, window < 0), UNSUPPORTED (batch > 4096),
 * CUDA_ERROR. */
int gptq_q4_attn_attend(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache *cache,
                        const gptq_q4_batch *batch, float scale, int window, void *out, int64_t out_stride,
                        cudaStream_t stream);

/* gptq_q4_attn_attend with the first `sinks` tokens of each context visible
 * besides the window: token j <= i is seen if j > i - window or j < sinks.  Keys
 * stay as they were appended, rotated to their positions in the text: the first
 * tokens are not moved up to the window.
 * Pages that hold neither a token below `sinks` nor one of a window are not
 * read, and their table entries may be anything.  sinks = 0, or window = 0
 * (all tokens are visible), is gptq_q4_attn_attend.  The sums, and their
 * order, may differ from that call's where sinks > 0 adds no token (a context
 * within its window).  Errors: as gptq_q4_attn_attend, and INVALID_ARGUMENT for
 * sinks < 0. */
int gptq_q4_attn_attend_sinks(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache *cache,
                              const gptq_q4_batch *batch, float scale, int window, int sinks, void *out,
                              int64_t out_stride, cudaStream_t stream);

/* What the cache holds for the step's new tokens:
 *   k_out, v_out  device [tokens][kv_heads * head_dim], row strides k_stride,
 *                 v_stride; 16-byte aligned, strides multiples of 8, not overlapping
 * (a batch whose requests have q_len = kv_len reads whole contexts).  Rows
 * that no request owns are left alone, as are those of a token whose index or
 * page index, or whose request's length, is outside its range;
 * gptq_q4_attn_device_error reports those.  Errors: INVALID_ARGUMENT,
 * UNSUPPORTED (batch > 4096), CUDA_ERROR. */
int gptq_q4_attn_read(gptq_q4_attn h, const gptq_q4_cache *cache, const gptq_q4_batch *batch, void *k_out,
                      int64_t k_stride, void *v_out, int64_t v_stride, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * A paged cache held in 4 bits, for the same handle and batch.
 *
 * Keys and values of one layer, a record of bytes for each token and head:
 *   kv  device uint8 [pages][kv_heads][page_size][record], 16-byte aligned;
 *       page_stride bytes from page to page (at least kv_heads * page_size *
 *       record, a multiple of 16);  record = head_dim + 8 * head_dim / group
 * A record holds, in this order,
 *   head_dim / 2 bytes     codes of the key: eight to a 32-bit word, code e of
 *                          a word's eight at bit 4 (e / 2) + 16 (e % 2)
 *   head_dim / 2 bytes     codes of the value
 *   4 * head_dim / group   for each group of the key its step s and least value m
 *   4 * head_dim / group   for each group of the value
 * with s and m of the handle's 16-bit type and groups of 32 or 64 elements.
 * Code c stands for m + s * c, rounded to the handle's type. */
typedef struct {
    void *kv;
    int pages;
    int64_t page_stride;
    int group;
} gptq_q4_cache4;

/* gptq_q4_attn_append into a cache of 4 bits.  Keys are rotated (the exact sum
 * of products with the fp32 cosines and sines, rounded to fp32 and from there to
 * the handle's type) and values taken as they are; then for each group
 *   m = the least element,  s = (greatest - m) / 15 rounded to the type,
 *   c = (x - m) / s rounded to the nearest (ties to even), at most 15;  0 where s is 0.
 * all of them of the exact differences and quotients.  A group with an infinity
 * or NaN, or whose span is past fp32, reads as NaN throughout.  A rounded step
 * may be too large by 2^-11 of itself (bf16: 2^-8), so the greatest elements of
 * a group whose greatest + 2^-11 (2^-8) * (greatest - m) is past the type's
 * largest number may read as infinity (fp16: 0 and 65504; 15 * 4368 = 65520). */
int gptq_q4_attn_append4(gptq_q4_attn h, const void *qkv, int64_t qkv_stride, const gptq_q4_cache4 *cache,
                         const gptq_q4_batch *batch, const int32_t *positions, void *q_out, int64_t q_stride,
                         cudaStream_t stream);

/* gptq_q4_attn_attend_sinks and gptq_q4_attn_read over a cache of 4 bits: over
 * the values that its codes stand for. */
int gptq_q4_attn_attend4(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache4 *cache,
                         const gptq_q4_batch *batch, float scale, int window, int sinks, void *out,
                         int64_t out_stride, cudaStream_t stream);
int gptq_q4_attn_read4(gptq_q4_attn h, const gptq_q4_cache4 *cache, const gptq_q4_batch *batch, void *k_out,
                       int64_t k_stride, void *v_out, int64_t v_stride, cudaStream_t stream);

/* As gptq_q4_device_error and gptq_q4_free, for an attention handle. */
int gptq_q4_attn_device_error(gptq_q4_attn h);
void gptq_q4_attn_free(gptq_q4_attn h);

/* ------------------------------------------------------------------------
 * The pages of a cache: which are free, forks that share them, copies, and
 * moving those in use together.
 *
 * A handle serves the caches of all layers, which share tables and page
 * numbers.  No counts are kept: a page is in use if the table, up to the
 * lengths, names it, however often (requests may share pages), and with a
 * window only if it holds one of the last `window` tokens or of the first
 * `sinks`.  (A step of n new tokens reads window - 1 + n tokens back from the
 * length after it; give a window that covers the next step's.)  Entries that
 * are needed but negative are no page and are passed over, ones past the last
 * page are and are reported by gptq_q4_pages_device_error.
 *
 * The handle has a workspace: one stream at a time.  It does not own the
 * buffers, which have to outlive it. */
typedef struct gptq_q4_pages_s *gptq_q4_pages;

/* One buffer with `bytes` of each page (k, v or kv of a layer's cache), page
 * p at data + p * stride; 16-byte aligned, bytes and stride multiples of 16. */
typedef struct {
    void *data;
    int64_t bytes, stride;
} gptq_q4_buffer;

/* The table's rows, as in gptq_q4_batch. */
typedef struct {
    int32_t *table, *kv_len;
    int64_t table_stride;
    int width, batch;
} gptq_q4_rows;

/* buffers: host, n of them (0: only the numbers are managed); pages at most
 * 2^22; page_size positive.  Device memory: about 12 bytes a page.
 * Synchronizes.  NULL on error: INVALID_ARGUMENT (a buffer of another device
 * than the current one among them), UNSUPPORTED (device not sm_103),
 * OUT_OF_MEMORY, CUDA_ERROR. */
gptq_q4_pages gptq_q4_pages_make(const gptq_q4_buffer *buffers, int n, int pages, int page_size);

/* The pages that are not in use: ids, device int32 [pages], ascending, then
 * -1; count, device int32 [1].  Errors: INVALID_ARGUMENT, CUDA_ERROR. */
int gptq_q4_pages_free_list(gptq_q4_pages h, const gptq_q4_rows *rows, int window, int sinks, int32_t *ids,
                            int32_t *count, cudaStream_t stream);

/* Rows child[i] become copies of rows parent[i], i < n: the entries up to the
 * parent's length (-1 past them) and the length.  A page that the parent has
 * filled in part is not shared: its contents go to page fresh[i] in every
 * buffer, and the child's entry is fresh[i] (which may be anything where the
 * length is a multiple of page_size).  A negative parent or child, or parent =
 * child, is no fork.  Left out, and reported by gptq_q4_pages_device_error: a
 * fork whose row numbers, parent's length or pages are outside their range,
 * whose child is the parent of another, is to stay (parent = child elsewhere)
 * or is the child of an earlier one, or whose fresh page an earlier one needs
 * (with a parent's number and length in their range).  fresh pages have to be
 * free.  parent, child, fresh:
 * device int32 [n], n at most 4096.  Errors: INVALID_ARGUMENT, UNSUPPORTED (n),
 * CUDA_ERROR. */
int gptq_q4_pages_fork(gptq_q4_pages h, const gptq_q4_rows *rows, const int32_t *parent, const int32_t *child,
                       const int32_t *fresh, int n, cudaStream_t stream);

/* Contents of pages src[i] to pages dst[i], i < n, in every buffer; a negative
 * number is no copy, one past the last page neither and is reported.  No page
 * may be a destination twice, or a destination and a source.  src, dst: device
 * int32 [n].  Errors: INVALID_ARGUMENT, CUDA_ERROR. */
int gptq_q4_pages_copy(gptq_q4_pages h, const int32_t *src, const int32_t *dst, int n, cudaStream_t stream);

/* Moves the pages in use together: with n of them, those numbered n and up go,
 * in ascending order, to the numbers below n that are not in use, ascending,
 * in every buffer; the others stay.  table_out (row stride out_stride; the
 * table itself if equal) gets the new numbers of the entries in use, -1
 * elsewhere; count, device int32 [1], gets n.  Pages from n on are free
 * afterwards.  Errors: INVALID_ARGUMENT, CUDA_ERROR. */
int gptq_q4_pages_compact(gptq_q4_pages h, const gptq_q4_rows *rows, int window, int sinks, int32_t *table_out,
                          int64_t out_stride, int32_t *count, cudaStream_t stream);

/* As gptq_q4_device_error and gptq_q4_free. */
int gptq_q4_pages_device_error(gptq_q4_pages h);
void gptq_q4_pages_free(gptq_q4_pages h);

/* Status and message of the last call made on this host thread.
 * "Inference Backends", "Hardware, dependency, and format requirements":
 * device-validation errors keep the kernel's specific reason (an unsupported
 * compute capability, a missing kernel image) instead of a generic one; the
 * message names the argument or limit that failed. */
int gptq_q4_last_status(void);
const char *gptq_q4_last_error(void);

/* Number of kernels this library has launched in this process. */
uint64_t gptq_q4_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_Q4_H */
