/*
 * qgemv.h -- C ABI of the weight-only quantized decode GEMV for GB300 (sm_103a)
 *
 *     y[M x N] = x[M x K] . dequant(W)^T ,   1 <= M <= 16
 *
 * W is an N x K weight matrix (N outputs, K inputs) held in a packed low-bit
 * format; x holds M fp16 activation rows; y receives M fp32 output rows.  The
 * packed weights stream from HBM, are decoded in registers and multiplied and
 * accumulated in fp32 by the library's CUDA kernels.  The problem statement
 * (M rows, N outputs, K inputs per output) is the one of "Making a ternary
 * reasoning model fast in vLLM", section "Reading the prompt and writing the
 * answer"; the formats are listed with their sources below.
 *
 * Conventions for every call:
 *   - Sizes are int64_t element counts; all multi-byte values little-endian.
 *   - Device pointers are CUDA device (or managed) addresses on the current
 *     device.  `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *     default stream).
 *   - A call returns QGEMV_OK (0) or one of the QGEMV_ERR_* codes; the handle
 *     constructor returns NULL on error.  qgemv_last_error() then gives a
 *     thread-local message.  No call aborts the process or throws.
 *   - Argument errors are found on the host before anything is launched or
 *     allocated.
 *   - Calls that launch kernels are asynchronous on `stream` unless stated
 *     otherwise.
 */
#ifndef QGEMV_H
#define QGEMV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Weight formats.  "Canonical" is the byte layout the caller passes in. */
typedef enum {
  /* ggml-style Q4_0 ("Model quantization, read carefully", sections "The
   * ladder" and "Anatomy of a block"): blocks of 32 weights along K, each
   * {fp16 d; uint8 qs[16]} = 18 bytes, 4.5 bits per weight.  Byte i of qs
   * holds element i in its low nibble and element i+16 in its high nibble;
   * the weight is (q - 8) * d.  packed = N*K/32 blocks, row-major over rows
   * n; K % 32 == 0; scales = codebooks = NULL.                              */
  QGEMV_Q4_0 = 1,
  /* Scalar 4-bit codebook ("Trapetum benchmarks", "Kernel microbenchmarks":
   * 4-bit index into K = 16 centroids): packed = uint8 [N][K/2], byte j of a
   * row holds k = 2j (low nibble) and k = 2j+1 (high nibble); codebooks =
   * 16 fp16 centroids shared by the whole matrix; K % 2 == 0; scales = NULL. */
  QGEMV_CBK4 = 2,
  /* Scalar 8-bit codebook (same page: uint8 index into 256 centroids, the
   * 8-bit LM head): packed = uint8 [N][K]; codebooks = 256 fp16; any K.    */
  QGEMV_CBK8 = 3,
  /* PQ2_0 ternary ("Making a ternary reasoning model fast in vLLM", "Anatomy
   * of a PQ2_0 block"): blocks of 128 weights along K, {fp16 d; uint8
   * qs[32]} = 34 bytes; byte j holds elements 4j..4j+3 as two-bit codes from
   * the low end; codes 0,1,2,3 decode to -1,0,+1,+2 times d.  packed = N*K/128
   * blocks, one row of blocks per output; K % 128 == 0.                      */
  QGEMV_PQ2_0 = 4,
  /* AQLM 2x8 additive codebooks ("Trapetum benchmarks", "Additive
   * vector-quantization GEMV" and "Llama-2-70B in 2 bits"): per group of 8
   * weights along K two uint8 codes; w[n][8g+j] = s[n] * (C0[c0][j] +
   * C1[c1][j]).  packed = codes uint8 [N][K/8][2] (codebook 0 first);
   * scales = fp16 [N]; codebooks = fp16 [2][256][8]; K % 8 == 0.          */
  QGEMV_AQLM_2X8 = 5,
  /* AQLM 1x16 ("Trapetum benchmarks", the PV-tuned Llama-2-70B in 1x16): one
   * codebook of 65,536 entries of 8 fp16 values per matrix and one 16-bit
   * code per group of 8 weights along K (2 bits per weight); w[n][8g+j] =
   * s[n] * C[code][j].  packed = codes uint16 little-endian [N][K/8];
   * scales = fp16 [N]; codebooks = fp16 [65536][8] (1 MiB); K % 8 == 0.
   * (Value 6 is reserved inside the library.)                              */
  QGEMV_AQLM_1X16 = 7,
  /* CBK4 with one codebook per output row, the pages' own 4-bit file layout
   * ("Trapetum benchmarks", "Model-level results": a 16-centroid k-means
   * codebook per output channel, stored in fp32): packed = uint8 [N][K/2]
   * as QGEMV_CBK4; codebooks = fp32 [N][16], row n's centroids together
   * (64 bytes per row); K % 2 == 0; scales = NULL.  Every M runs the
   * CUDA-core kernel (fp32 centroids), eight activation rows per launch
   * while eight remain, then two, then one; a row's bits do not depend on M
   * in batch-invariant mode (which keeps to the two- and one-row launches),
   * and otherwise differ at most in the last places between calls below and
   * above eight rows.                                                      */
  QGEMV_CBK4_ROW = 8,
  /* CBK8 with one codebook per output row, the 8-bit LM head of the same
   * files (256 fp32 centroids per row): packed = uint8 [N][K]; codebooks =
   * fp32 [N][256] (1 KB per row); 1 <= K <= 65536; scales = NULL.  One warp
   * per output row, the row's codebook in shared memory; a row's bits do not
   * depend on M.                                                            */
  QGEMV_CBK8_ROW = 9
} qgemv_format;

/* Status codes. */
enum {
  QGEMV_OK = 0,
  QGEMV_ERR_ARG = 1,     /* bad format, size, M, null pointer or handle     */
  QGEMV_ERR_ALIGN = 2,   /* x or y not aligned as required                  */
  QGEMV_ERR_CUDA = 3,    /* a CUDA call failed (message has its error text) */
  QGEMV_ERR_TIMEOUT = 4, /* a kernel's bounded wait gave up (qgemv_status)  */
  QGEMV_ERR_NOMEM = 5    /* device or host allocation failed                */
};

typedef struct qgemv_ctx* qgemv_handle; /* opaque */

/* Bytes of the canonical packed weights for (format, N, K); 0 if invalid. */
int64_t qgemv_packed_bytes(int format, int64_t N, int64_t K);

/* Create a handle for one weight matrix.
 *   packed, scales, codebooks: canonical inputs as described per format
 *     (unused ones must be NULL).  Each may be a host or a device pointer
 *     (told apart with cudaPointerGetAttributes); the data is copied into
 *     library-owned device memory and re-laid out there ("prepared" tiles),
 *     so the caller may free its buffers once this call returns.
 *   The call allocates the handle's device buffers (prepared weights and a
 *   small per-handle workspace), runs the re-layout kernel on the legacy
 *   default stream and synchronizes before returning.
 * Returns NULL on error (see qgemv_last_error).                              */
qgemv_handle qgemv_create(int format, int64_t N, int64_t K, const void* packed,
                          const void* scales, const void* codebooks);

/* Create one handle for several projections that share K and therefore the
 * activations (the attention's q, k and v, or an MLP's gate and up): their
 * weight rows stacked in order, so that one qgemv_run computes all of them,
 * y = [y_0 | y_1 | ...] along N, with one launch instead of one per
 * projection.  The pages fuse such projections in their runtimes; this call
 * has no further counterpart there.
 *   nseg >= 1 segments; segment s has seg_rows[s] > 0 output rows, and every
 *     segment but the last must have a multiple of the prepared tile height
 *     (128 rows; AQLM 2x8: 2048, its row block), so that no tile mixes two
 *     codebooks.
 *   packed: the segments' canonical bytes one after the other, which is the
 *     canonical layout of the stacked matrix (rows of all formats are
 *     independent).
 *   codebooks (CBK4, CBK8, AQLM 2x8): nseg codebooks one after the other
 *     (16 or 256 fp16 each; AQLM 2x8: a [2][256][8] fp16 pair each); segment
 *     s decodes with codebook s.  NULL for Q4_0 and PQ2_0, whose stacked
 *     handle is the plain concatenation.
 *   scales (AQLM 2x8): the N row scales of all segments in order.
 *   A stacked AQLM 2x8 handle runs its per-group-table kernel at every M (a
 *     pass per two activation rows), without the tensor-core form that a
 *     single-matrix handle uses from M = 3.
 *   AQLM 1x16, CBK4_ROW and CBK8_ROW are not accepted (QGEMV_ERR_ARG; 1x16
 *   keeps one 1 MiB codebook per handle, and the rows of a per-row-codebook
 *   matrix carry their own codebooks, so one handle over the concatenated
 *   rows does the same).
 * Host or device pointers, copying, errors: as for qgemv_create.             */
qgemv_handle qgemv_create_stacked(int format, int nseg, const int64_t* seg_rows, int64_t K,
                                  const void* packed, const void* scales, const void* codebooks);

/* Create one handle for the gate and up projections of a decoder MLP whose
 * runs store the fused activation y[m][n] = SiLU(x . G^T)[m][n] * (x . U^T)
 * [m][n], SiLU(v) = v / (1 + e^-v): the gate/up GEMV with "SiLU(gate) * up
 * in the reduce" of "Trapetum benchmarks" ("Short-context decode, step by
 * step"), with no separate activation kernel.  Q4_0, PQ2_0, CBK4 and CBK8
 * run every M in one launch (M >= 2 on the tensor-core kernel, the weights
 * read once per call); CBK4_ROW launches once per activation row.
 *   format: QGEMV_Q4_0, QGEMV_PQ2_0, QGEMV_CBK4, QGEMV_CBK8 or QGEMV_CBK4_ROW
 *     (CBK4 / CBK8: the gate and up tables share the kernels' table region,
 *     each lookup still one shared-memory read; per-row codebooks travel
 *     with their rows).
 *   N: rows of each projection (the output width), a positive multiple of
 *     64; K as for qgemv_create.
 *   packed_gate, packed_up: each projection's canonical bytes (host or
 *     device), copied.  The handle holds them interleaved in 64-row blocks.
 *   codebooks_gate, codebooks_up: each projection's codebook -- CBK4 fp16
 *     [16], CBK8 fp16 [256], CBK4_ROW fp32 [N][16]; NULL for Q4_0 and PQ2_0.
 * Runs: qgemv_run with y fp32 [M][N]; the residual form is refused, and so
 * are qgemv_set_x_int8 and qgemv_run_xq.  qgemv_dequant of such a handle
 * writes the 2N interleaved rows (64 gate rows, then the 64 up rows of the
 * same block, and so on).  The result is SiLU and the product in fp32
 * (expf, an IEEE division, one product) of the two GEMV sums.
 * Returns NULL on error (QGEMV_ERR_ARG for another format or a bad N).     */
qgemv_handle qgemv_create_glu(int format, int64_t N, int64_t K, const void* packed_gate,
                              const void* packed_up, const void* codebooks_gate, const void* codebooks_up);

/* y = x . dequant(W)^T for M rows.
 *   x: device fp16 [M][K] row-major, 4-byte aligned.
 *   y: device fp32 [M][N] row-major, 4-byte aligned; fully overwritten.
 *   1 <= M <= 16.
 * Asynchronous on `stream`; no allocation, no synchronization, so it can be
 * captured in a CUDA graph.  The handle's workspace is shared by its runs:
 * one handle must not run on two streams at the same time.  Results are
 * bitwise reproducible run to run for a given (handle, M).                  */
int qgemv_run(qgemv_handle h, const void* x, int M, float* y, void* stream);

/* y = residual + x . dequant(W)^T for M rows: the residual add of a decoder
 * layer's attention-output and MLP-down projections done in the GEMV's own
 * store instead of a separate kernel ("Trapetum benchmarks", "Short-context
 * decode, step by step": the residual add inside the o and down reduces).
 *   residual: device fp32 [M][N] row-major, 4-byte aligned, not NULL.  It may
 *     be y itself (y += x . W^T): each element is read and then written by
 *     the same thread.
 *   x, y, M, stream and the handle: as for qgemv_run.
 * Each output is the value qgemv_run would store, plus the residual in one
 * fp32 add (round to nearest), so the two calls agree bit for bit.         */
int qgemv_run_residual(qgemv_handle h, const void* x, int M, float* y, const float* residual,
                       void* stream);

/* Batch-invariant mode (off by default): when on, row m of y from any call
 * is bitwise the same whatever M the call has and wherever the row sits in
 * the batch (the same x row gives the same y row alone or batched, as a
 * verifier comparing batched and single-row decodes needs).  Off, M = 1 and
 * M = 2..8 run faster kernel geometries (and AQLM 2x8 with M <= 2 its
 * per-group table path), whose bits may differ in the last places (all
 * within the accuracy bound).  On, every M runs the tensor-core kernel's
 * default geometry (AQLM 2x8: its tensor-core layout; a stacked AQLM 2x8
 * handle: a one-row pass of its table kernel per row; CBK4_ROW: launches of
 * at most two rows; AQLM 1x16 and CBK8_ROW are batch invariant in either
 * mode).  Takes effect for runs issued after the call; returns
 * QGEMV_ERR_ARG for an invalid handle. */
int qgemv_set_batch_invariant(qgemv_handle h, int on);

/* INT8 activations for a PQ2_0 handle (off by default): the integer path of
 * "Making a ternary reasoning model fast in vLLM" (the section on quantising
 * the activation too).  When on, runs quantize each group of 128 activations
 * of a row to signed INT8 exactly as qgemv_quantize_x_int8 does, take every
 * block's inner sum over its codes in integer arithmetic (four-way INT8 dot
 * products) and apply d * a once per block in fp32.  The result is that of
 * the quantized activations: lossy against qgemv_run with the mode off (the
 * quantization error is a property of the method, at most half a step of
 * each group's scale per nonzero weight), and accurate to the usual fp32
 * bound against the exact integer-path value.  Up to three activation rows
 * run the CUDA-core kernel (DP4A inner sums, up to four rows per launch);
 * four or more run, in one call, the quantizer of qgemv_prepare_x_int8 into
 * a handle-owned workspace and one launch of the tensor-core kernel (the
 * INT8 codes as exact fp16 operands, exact integer block sums), so the
 * weights are read once per call.  A row's bits are the same in every call
 * of up to three rows and in every call of four or more; the two kernels
 * may differ in the last places (same bound) unless batch-invariant mode is
 * on, which puts every M on the tensor-core kernel.  Works with qgemv_run and qgemv_run_residual; takes
 * effect for runs issued after the call.  The first call that turns the mode
 * on allocates the workspace (qgemv_xq_bytes(16, K) bytes, freed with the
 * handle): QGEMV_ERR_NOMEM if that fails.  Returns QGEMV_ERR_ARG for an
 * invalid handle or a handle that is not PQ2_0 (stacked PQ2_0 handles are
 * accepted).                                                                */
int qgemv_set_x_int8(qgemv_handle h, int on);

/* The INT8 activation quantizer of the PQ2_0 integer path, on the device:
 *   x: device fp16 [M][K] row-major, K a positive multiple of 128, M >= 1;
 *   q_out: device int8 [M][K];  a_out: device fp32 [M][K/128].
 * Per group g of 128 consecutive inputs of a row: a = fl32(max|x| / 127),
 * q = clamp(rint(fl32(x / a)), -127, 127) with IEEE fp32 divisions and
 * ties to even; an all-zero group gives a = 0 and q = 0.  The same device
 * arithmetic as the GEMV's staging (for tests and for callers that keep
 * the quantized activations).  Asynchronous on `stream`.                   */
int qgemv_quantize_x_int8(const void* x, int M, int64_t K, int8_t* q_out, float* a_out, void* stream);

/* Prepared INT8 activations for PQ2_0 handles: the activation prologue of
 * the integer path, run once per activation vector and shared by every
 * projection that reads it (q, k and v; gate and up), with the Hadamard
 * mixing of "Making a ternary reasoning model fast in vLLM" (the section on
 * mixing the inputs) fused in when asked.
 *
 * Bytes of the prepared buffer of M rows of K inputs (K % 128 == 0), or 0
 * for invalid sizes: M*K codes, then M*K/128 fp32 scales, then M*K/128
 * int32 code sums.                                                          */
int64_t qgemv_xq_bytes(int M, int64_t K);

/* Fill xq (device, qgemv_xq_bytes(M, K) bytes, 4-byte aligned) from x
 * (device fp16 [M][K], 4-byte aligned).
 *   hadamard_block = 0: the codes of x itself, exactly as
 *     qgemv_quantize_x_int8 computes them.
 *   hadamard_block = 1024 (K % 1024 == 0): each block of 1024 inputs is
 *     first mixed, v = 2^-5 H (s . x) with H the 1024 x 1024 Sylvester
 *     Hadamard matrix, computed in fp32 as the page does (signs, then
 *     butterfly stages h = 1, 2, ..., 512 replacing (u, w) by (u + w,
 *     u - w), then the scaling), and the fp32 values v are quantized.
 *     signs: device int8 [K] of +1 / -1 over the row width (the same for
 *     every row), or NULL for none.
 * Layout of xq: row m's codes at byte m*K; within each group of 128 inputs
 * the code of input 16i + 4b + s (i = 0..7, b = 0..3, s = 0..3) is at byte
 * 16i + 4s + b of the group (the order the GEMV stages them); the scale of
 * group g of row m is float m*K/128 + g after the codes, and its code sum
 * the int32 of the same index after the scales.  Asynchronous on `stream`; returns
 * QGEMV_ERR_ARG for bad sizes, a block other than 0 or 1024, or signs
 * without the mixing; QGEMV_ERR_ALIGN for misaligned pointers.             */
int qgemv_prepare_x_int8(const void* x, int M, int64_t K, const int8_t* signs, int hadamard_block, void* xq,
                         void* stream);

/* y = residual + (prepared INT8 activations) . dequant(W)^T for a PQ2_0
 * handle: the integer path of qgemv_set_x_int8 on codes from
 * qgemv_prepare_x_int8 (with the same M and the handle's K): up to three
 * rows on the CUDA-core kernel, four or more in one launch of the
 * tensor-core kernel (as for qgemv_set_x_int8).  With hadamard_block = 0 the result equals qgemv_run in INT8 mode
 * bit for bit.
 * residual may be NULL (plain store) or y itself.  The handle's INT8 mode
 * setting does not matter here.  Asynchronous; as qgemv_run otherwise.     */
int qgemv_run_xq(qgemv_handle h, const void* xq, int M, float* y, const float* residual, void* stream);

/* Write the decoded weights, fp32 [N][K] row-major, to device memory w_out
 * (the exact value of every weight; read back from the prepared tiles, so it
 * also checks the re-layout).  Asynchronous on `stream`.                     */
int qgemv_dequant(qgemv_handle h, float* w_out, void* stream);

/* Q4_0 quantizer on the device: fp32 weights [N][K] (device) -> canonical
 * Q4_0 blocks (device, N*K/32*18 bytes).  Per block: d = (signed value of
 * largest magnitude, first on ties) / -8 in fp32; q = clamp(round(w/d) + 8,
 * 0, 15) with an IEEE fp32 division and round half away from zero; d stored
 * as fp16 (nearest even).  An all-zero block stores q = 8.  Asynchronous.  */
int qgemv_quantize_q4_0(const float* w, int64_t N, int64_t K, void* packed_out,
                        void* stream);

/* Synchronize with the handle's last run and return QGEMV_ERR_TIMEOUT if a
 * kernel of it gave up a bounded wait (then clear that flag), else QGEMV_OK. */
int qgemv_status(qgemv_handle h);

/* Release the handle's device memory (synchronizes the device first).
 * NULL is accepted and ignored.                                             */
void qgemv_destroy(qgemv_handle h);

/* Allocation-free Q4_0 GEMV.  No counterpart in the source pages: a service
 * for callers that cannot allocate device memory when they need the product,
 * for instance code running inside a framework whose caching allocator owns
 * all device memory, or a latency-critical loop that must not pay for (or
 * synchronize on) cudaMalloc.  It needs no handle: it reads the caller's
 * canonical Q4_0 blocks directly (same layout as QGEMV_Q4_0 above).
 *   packed: device, N*K/32 blocks of 18 bytes, 2-byte aligned; K % 32 == 0.
 *   x: device fp16 [M][K]; y: device fp32 [M][N] (4-byte aligned); 1<=M<=16.
 * The call allocates nothing: its scratch (split-K partial sums and arrival
 * counters) lives in one static device array of 8 MiB that every GPU which
 * loads this library holds until the process exits.  A shape needs
 * ceil(K/2048) * M * N * 4 bytes of partial sums (none when K <= 2048) plus
 * 4 bytes per 64 rows of counters; a shape that needs more than 8 MiB is
 * rejected with QGEMV_ERR_ARG and a message giving both sizes.
 * All calls share that array and leave in it whatever the last one wrote; the
 * counters, which must start at zero, are cleared by every call.  Calls whose
 * executions overlap on the GPU (different streams, or several processes'
 * worth of work on one context) race on the array: serialize them.
 * The first call on a device finds the array's device address
 * (cudaGetSymbolAddress) with that device current and sets the kernel's
 * shared-memory limit; make that first call before any stream capture.  If
 * that set-up fails, the call returns QGEMV_ERR_CUDA, nothing is remembered
 * and the next call on the device tries the set-up again.
 * Asynchronous on `stream`; results are bitwise reproducible call to call.  */
int qgemv_run_q4_0_noalloc(const void* packed, int64_t N, int64_t K, const void* x, int M,
                           float* y, void* stream);

/* The stream-K work split (host only, no GPU needed), as the handles use it:
 * `units` work units (prepared tiles; for AQLM_2X8 blocks of 2048 rows x 128
 * inputs) in row-major order, `units_per_row_tile` of them per row tile of
 * `rows` output rows, split over `grid` CTAs: split_unit 0, CTA c runs
 * units [c*units/grid, (c+1)*units/grid); split_unit 1 or 2, in chunks of
 * that many consecutive units, n = ceil(units / split_unit) chunks, q = n /
 * grid, r = n % grid, CTA c runs chunks [c*q + min(c, r), (c+1)*q + min(c+1,
 * r)) (the last chunk may be short).  A handle uses its format's mode.
 * Writes 12
 * int64 per CTA into `out` (caller-owned, grid*12 entries): for its two
 * shared-row-tile segments s = 0 (first row tile of its run), 1 (last):
 * out[c*12 + 0 + s] row tile (-1: none), [2 + s] first contributing CTA,
 * [4 + s] number of contributors, [6 + s] first row of this CTA's slice of
 * the rows to finish, [8 + s] rows in that slice, [10 + s] flags: bit 0 set
 * if the first contributor's run began before the row tile, bit 1 set if
 * this CTA finishes the whole row tile when it has at most 256 items (rows x
 * activation rows; then the others finish nothing).  Returns QGEMV_ERR_ARG if a
 * size is not positive, units % units_per_row_tile != 0, grid > units or
 * split_unit is not 0, 1 or 2.                                               */
int qgemv_stream_k_plan(int64_t units, int grid, int64_t units_per_row_tile, int rows, int split_unit,
                        int64_t* out);

/* ------------------------------------------------- cache and attention ----
 *
 * The attention of a decoder layer between its q|k|v and o projections: a
 * paged key/value cache (fp16 or quantised), attention of one or several
 * drafted tokens of each sequence over it, and causal attention over packed
 * prompts.  No counterpart in the source pages, whose runtimes keep their
 * own; formulas:
 *
 *   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j),
 *   lse_i = log sum_j p_ij,  over the keys j that row i sees.
 *
 * A row that sees no key gives out = 0 and lse = -infinity.  Key/value head
 * h serves the query heads h * g .. h * g + g - 1, g = q_heads / kv_heads.
 * Scores, softmax statistics and sums are held in fp32 (over INT8 and Q4_0
 * keys a score's error is about 2^-24 max|k_j| sum|q_i| scale, the codes being
 * summed with an offset); the probabilities, INT8 and Q4_0: times the values'
 * scales, are rounded to the values' 16-bit type (fp16 over a cache) for the
 * tensor cores.  A value or key that a row does not see never reaches it,
 * infinities and NaN included.
 *
 * Rows of heads are given as a device pointer and two element strides,
 * between tokens and between heads; the head_dim values of a row are
 * contiguous.  Inputs and outputs need 16-byte aligned pointers and strides
 * that are multiples of 16 bytes (QGEMV_ERR_ALIGN), so that slices of a
 * stacked projection's output can be passed as they are; two rows of an
 * output share no element (QGEMV_ERR_ARG).  head_dim is 64 or 128.  Calls
 * run on the current device, which all of their memory belongs to.  Empty
 * calls (no tokens) return QGEMV_OK.  Index arrays (slots, page table,
 * lengths, offsets) live on the device and are not checked on the host; the
 * kernels never read or write outside the buffers that the sizes describe,
 * whatever they hold.                                                       */

/* Element types of rows. */
typedef enum { QGEMV_DT_F32 = 0, QGEMV_DT_F16 = 1, QGEMV_DT_BF16 = 2 } qgemv_dtype;

/* Cache formats; per token and head, a vector x of head_dim values. */
typedef enum {
  /* x rounded to fp16. */
  QGEMV_KV_F16 = 1,
  /* a = fl32(max|x| / 127) (fp32, kept), code = clamp(rint(fl32(x / a)),
   * -127, 127), all 0 if a = 0; the value is code * a.                      */
  QGEMV_KV_INT8 = 2,
  /* The Q4_0 quantiser of qgemv_quantize_q4_0 on each 32 values: a =
   * (signed value of largest magnitude) / -8, kept as fp16, code =
   * clamp(round(x / a) + 8, 0, 15); the value is (code - 8) * fp16(a).      */
  QGEMV_KV_Q4_0 = 3
} qgemv_kv_format;
/* A vector (Q4_0: a group of 32) with an infinity or NaN is kept as all NaN
 * in the quantised formats; so is a Q4_0 group whose a is past fp16's range
 * (values from 524160 on).                                                  */

/* A cache: n_pages pages of page_tokens tokens for each of kv_heads heads,
 * in the caller's device memory (qgemv_kv_bytes bytes, 128-byte aligned).
 * page_tokens is 16, 32, 64, 128 or 256.  A slot is page * page_tokens +
 * token of the page.  The byte layout inside a page is the library's; pages
 * are independent and may be copied whole (all bytes / n_pages each).       */
typedef struct {
  void* pages;
  int format; /* qgemv_kv_format */
  int head_dim;
  int kv_heads;
  int page_tokens;
  int64_t n_pages;
} qgemv_kv_cache;

/* Bytes of a cache, or 0 for invalid sizes. */
int64_t qgemv_kv_bytes(int format, int64_t n_pages, int page_tokens, int kv_heads, int head_dim);

/* Quantise n_tokens tokens' k and v rows ([n_tokens][kv_heads][head_dim] of
 * dtype, any qgemv_dtype) into the slots slots[i] (device int64).  A negative
 * slot, or one past the cache, skips its token.  No two tokens of a call may
 * share a slot.  Asynchronous on `stream`.                                  */
int qgemv_kv_write(const qgemv_kv_cache* cache, int dtype, const void* k, int64_t k_token_stride,
                   int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                   const int64_t* slots, int64_t n_tokens, void* stream);

/* Read cached tokens back as rows of dtype (rounded once from fp32):
 * sequence b's positions starts[b] .. (0 .. if starts is NULL) go to the rows
 * cu[b] .. cu[b + 1] - 1 of k and v ([n_tokens][kv_heads][head_dim]); cu is
 * device int32 [n_seqs + 1], not decreasing.  table: device int32 [n_seqs]
 * [table_stride], the page of each page_tokens positions of a sequence.  A
 * position whose page is missing (an entry outside the cache, or past the
 * table) gives zeros.  Rows that belong to no sequence are left as they are.  */
int qgemv_kv_read(const qgemv_kv_cache* cache, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                  const int32_t* starts, const int32_t* cu, int64_t n_tokens, int dtype, void* k,
                  int64_t k_token_stride, int64_t k_head_stride, void* v, int64_t v_token_stride,
                  int64_t v_head_stride, void* stream);

/* Workspace of the attention calls for up to n_seqs sequences: device memory,
 * 256-byte aligned, set up once by qgemv_attn_ws_init (asynchronous on
 * stream) and then reused by any number of calls of both kinds, one at a
 * time (calls that overlap on the GPU need a workspace each).               */
int64_t qgemv_attn_ws_bytes(int64_t n_seqs, int q_heads, int head_dim);
int qgemv_attn_ws_init(void* ws, int64_t ws_bytes, void* stream);

/* Synchronise the device and return QGEMV_ERR_TIMEOUT if an attention kernel
 * gave up a bounded wait since the last call (the workspace then needs
 * qgemv_attn_ws_init), else QGEMV_OK.                                       */
int qgemv_attn_status(void* ws);

/* Attention of drafted tokens over the cache.  The tokens are in it already:
 * token i of sequence b (row cu_q[b] + i of q and out, fp16 [n_q][q_heads]
 * [head_dim]) is at position ctx_lens[b] + i.  It sees the positions before
 * ctx_lens[b] and, of the drafted ones, ctx_lens[b] + j where bit j of
 * masks[row] is set (masks: device uint64 [n_q], or NULL for bits 0 .. i: a
 * chain, which for one token is plain decoding).  A sequence has at most 64
 * drafted tokens; further rows are left as they are.  Positions whose page is
 * missing are not seen.
 *   ctx_lens, cu_q: device int32 [n_seqs], [n_seqs + 1].
 *   max_ctx, max_new: upper bounds on the lengths, for the host's choice of
 *     kernel and split only: results are right whatever they are.
 *   lse: device fp32 [n_q][q_heads], or NULL.
 * Asynchronous on `stream`, no allocation, can be captured in a CUDA graph;
 * bitwise reproducible for given sizes and lengths.                         */
int qgemv_attn_tree(const qgemv_kv_cache* cache, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                    const int32_t* ctx_lens, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                    int q_heads, const int32_t* cu_q, int64_t n_q, const uint64_t* masks, int64_t max_ctx,
                    int64_t max_new, float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                    float* lse, void* ws, int64_t ws_bytes, void* stream);

/* Causal attention over packed prompts: sequence b has the queries cu_q[b] ..
 * cu_q[b + 1] - 1 of q [n_q][q_heads][head_dim] and the keys cu_k[b] ..
 * cu_k[b + 1] - 1 of k and v [n_k][kv_heads][head_dim]; the last query sees
 * all of the keys, the one before it all but the last, and so on (query i of
 * nq sees the keys j <= i + nk - nq of nk: chunks after a past, or rows that
 * see nothing where nk < nq).  dtype: QGEMV_DT_F16 or QGEMV_DT_BF16, of q, k,
 * v and out; no strides of zero, and at most
 * 128 query heads of a key/value head.
 *   cu_q, cu_k: device int32 [n_seqs + 1], not decreasing.
 *   max_q: the most queries of a sequence; 0 for a call with nothing to do,
 *     which then does nothing.  Its other values change nothing at present.
 *   lse: device fp32 [n_q][q_heads], or NULL.
 * Asynchronous on `stream`, no allocation, can be captured in a CUDA graph;
 * bitwise reproducible.                                                     */
int qgemv_attn_prompt(int dtype, int head_dim, int q_heads, int kv_heads, const void* q, int64_t q_token_stride,
                      int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                      const void* v, int64_t v_token_stride, int64_t v_head_stride, int64_t n_seqs,
                      const int32_t* cu_q, const int32_t* cu_k, int64_t n_q, int64_t n_k, int64_t max_q,
                      float scale, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                      void* ws, int64_t ws_bytes, void* stream);

/* ------------------------------------------------------ rotary positions ----
 *
 * Pair j of a head vector, (a, b), becomes (a cos - b sin, a sin + b cos) of
 * the angle position[axes[j]] * freqs[j]: up to four axes, as for images and
 * video (time, height, width).  Values behind the pairs stay as they are.
 * The angle is taken in 64-bit fixed point, so that far positions lose
 * nothing (it is off by at most |position| 2^-65 turns and then rounded once to
 * fp32); the products are fp32, the results rounded once.  Negative positions
 * turn backwards: rotating by -position undoes a rotation (and is its
 * gradient), rotating kept keys by a difference moves them.                  */
typedef enum {
  QGEMV_ROPE_HALVES = 0,    /* pair j: values j and j + pairs */
  QGEMV_ROPE_NEIGHBOURS = 1 /* pair j: values 2j and 2j + 1 */
} qgemv_rope_pairing;

/* A plan of `pairs` pairs (1 .. 64): 16 bytes each; 0 for invalid numbers.
 * qgemv_rope_plan fills host memory, which the caller copies to the device
 * (16-byte aligned there); freqs in radians a position, within [-1024, 1024],
 * axes 0 .. 3.                                                               */
int64_t qgemv_rope_plan_bytes(int pairs);
int qgemv_rope_plan(const double* freqs, const int32_t* axes, int pairs, void* plan);

/* Rotate the rows x [n_tokens][heads][head_dim] of dtype into out (of
 * out_dtype; x itself, where pointer, strides and types are the same, but no
 * other rows that overlap x).  positions: device int32 [n_tokens][n_axes];
 * a pair of an axis past n_axes takes position 0.  head_dim 64 or 128, at most
 * head_dim / 2 pairs.  Asynchronous on `stream`.                             */
int qgemv_rope_rows(const void* plan, int pairs, int pairing, int n_axes, const int32_t* positions, int dtype, int heads,
                    int head_dim, const void* x, int64_t x_token_stride, int64_t x_head_stride, int64_t n_tokens,
                    int out_dtype, void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* qgemv_kv_write of rotated keys, and the rotated queries beside it, in one
 * launch: q [n_tokens][q_heads][head_dim] goes rotated to q_out (of
 * out_dtype), k rotated and v as it is are quantised into the slots.  Rows
 * and slots as for qgemv_kv_write (the keys' codes are of their rotated fp32
 * values); a token whose slot is skipped still gets its q.                  */
int qgemv_kv_write_rotated(const qgemv_kv_cache* cache, const void* plan, int pairs, int pairing, int n_axes,
                           const int32_t* positions, int dtype, const void* q, int64_t q_token_stride,
                           int64_t q_head_stride, int q_heads, const void* k, int64_t k_token_stride,
                           int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                           const int64_t* slots, int64_t n_tokens, int out_dtype, void* q_out,
                           int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* --------------------------------------------------- beam search's choice ----
 *
 * Of each sequence's candidates (beam b, token t) the `width` of largest
 *
 *   scores[b] + x[b][t] - log sum_u exp x[b][u],
 *
 * in descending order; ties go to the lower beam, then to the lower token.
 *   logits: device rows of dtype (any qgemv_dtype), one for each beam of each
 *     sequence ([n_seqs * beams], row_stride elements apart; any alignment of
 *     elements), of vocab tokens: an LM head's output.
 *   scores: device fp32 [n_seqs][beams], the beams' sums of log
 *     probabilities so far.
 *   out_scores, out_beams, out_tokens: device [n_seqs][width], apart from the
 *     inputs and from one another.
 * A beam whose score is not finite (-infinity: not in use), or whose log sum
 * is not (a NaN or +infinity among its logits, or nothing but -infinity), has
 * no candidates, nor have tokens of -infinity; places for which there is no
 * candidate hold (-infinity, -1, -1).  The sums of exponentials are fp32, off by
 * less than 2^-17 of themselves however long a row is; log sums and scores are
 * compared in 64 bits and rounded once.  Equal rows have equal log sums, wherever
 * they lie: beams of equal scores and rows tie.  beams and width are at most 64,
 * sequences 4096 a call.
 * ws: qgemv_beam_ws_bytes bytes, 16-byte aligned, zeroed once by the caller
 * and then reused by calls of any sizes that it is large enough for; calls
 * that overlap on the GPU need one each.  Asynchronous on `stream`, no allocation,
 * can be captured in a CUDA graph; bitwise reproducible.                     */
int64_t qgemv_beam_ws_bytes(int64_t n_seqs, int beams, int64_t vocab, int width);
int qgemv_beam_select(int dtype, const void* logits, int64_t row_stride, int64_t vocab, const float* scores, int64_t n_seqs,
                      int beams, int width, float* out_scores, int32_t* out_beams, int32_t* out_tokens, void* ws,
                      int64_t ws_bytes, void* stream);

/* --------------------------------------------------------- pages of a cache ----
 *
 * A pool's bookkeeping of pages, for any number of caches with the same
 * numbers of pages and tokens (a cache a layer, one page table): refs, device
 * int32 [n_pages], counts the rows of page tables that hold a page; pages of
 * count 0 (or less) are free.  state is device int32 [2].  The caller zeroes
 * both once.  Tables are device int32 [rows][table_stride], lengths device
 * int32 in tokens; a row of length n holds the pages of its first
 * ceil(n / page_tokens) entries.  Entries that are no page's number are passed
 * over.  Free pages are given out lowest first, in the order of the rows, so
 * results depend on the inputs alone.  Where there are none left, the entry
 * becomes -1 and state[0] counts it (state[1] is the calls' own, 0 between
 * them).  At most 4096 rows of 2^20 entries a call; calls of one pool one at a
 * time.  All are asynchronous on `stream`, allocate nothing, can be captured
 * in a CUDA graph.
 *
 * reserve: row b, which holds have[b] tokens, gets the pages that need[b]
 * tokens take beyond them.  Entries past the table's width are not there: they
 * are neither filled nor counted as missing.                                 */
int qgemv_pool_reserve(int32_t* refs, int64_t n_pages, int page_tokens, int32_t* table, int64_t table_stride, int64_t n_seqs,
                       const int32_t* have, const int32_t* need, int32_t* state, void* stream);

/* fork (a step of beam search): the rows are replaced by n_new new ones, row
 * r of new_table (same table_stride; no overlap with table) what row
 * parents[r] was; lens has the old rows' lengths.  A parent outside the rows
 * gives an empty row.  Whole pages are shared: their counts change by the
 * children of each row that held them, less one, so that rows without
 * children return theirs.  The page that a row has filled in part must be
 * that row's alone; it stays with the row's first child, and each further
 * child r gets a free page instead, to which tokens[r] tokens have to be
 * copied: src[r] to dst[r], by qgemv_kv_copy_pages for each cache; -1 for rows
 * without a copy (device int32 [n_new] each).  Entries behind a row's
 * length become -1 and are not counted.                                      */
int qgemv_pool_fork(int32_t* refs, int64_t n_pages, int page_tokens, const int32_t* table, int64_t table_stride, int64_t n_rows,
                    const int32_t* parents, int64_t n_new, const int32_t* lens, int32_t* new_table, int32_t* src, int32_t* dst,
                    int32_t* tokens, int32_t* state, void* stream);

/* release: row b, of lens[b] tokens, keeps the pages of its first keep[b]
 * tokens (none where keep is NULL); the others' counts go down by one and
 * their entries become -1.  A page that is kept in part stays shared with the
 * rows that hold it, and no call makes it this row's alone: a row that goes on
 * from there writes into theirs.                                             */
int qgemv_pool_release(int32_t* refs, int64_t n_pages, int page_tokens, int32_t* table, int64_t table_stride, int64_t n_seqs,
                       const int32_t* lens, const int32_t* keep, void* stream);

/* compact: with U pages in use, those numbered U and more move, in order, to
 * the free ones below U.  src and dst (device int32 [n_moves], n_moves at
 * least n_pages / 2) are the moves for qgemv_kv_copy_pages, followed by -1;
 * refs follows, and new_table is table with the new numbers (or table
 * itself; every entry that is a page in use is renumbered).  ws:
 * qgemv_pool_ws_bytes bytes, no setting up.                                  */
int64_t qgemv_pool_ws_bytes(int64_t n_pages);
int qgemv_pool_compact(int32_t* refs, int64_t n_pages, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                       int32_t* new_table, int32_t* src, int32_t* dst, int64_t n_moves, void* ws, int64_t ws_bytes, void* stream);

/* Copy page src[i] of a cache to page dst[i] (device int32 [n]), whole, or the
 * first tokens[i] tokens of every head, up to a multiple of 16.  Pairs with a
 * number that is no page are passed over.  No page may be the destination of
 * two copies, or of one and the source of another.  A page is kv_heads runs
 * of page_tokens / 16 blocks of 16 tokens, all of the same size.
 * Asynchronous on `stream`.                                                  */
int qgemv_kv_copy_pages(const qgemv_kv_cache* cache, const int32_t* src, const int32_t* dst, const int32_t* tokens, int64_t n,
                        void* stream);

/* ------------------------------------------- attention over selected pages ----
 *
 * Long contexts without reading all of them: of a sequence's whole pages
 * (those that end at or before ctx_lens[b]) each key/value head attends the
 * n_select with the highest score, and all positions behind the last whole
 * page.  Scores come from summaries of the pages' keys, which qgemv_kv_summarize
 * takes once a page is full (and again when it was written anew):
 *
 *   hi_d, lo_d = the largest and smallest of the page's key values, as the
 *   cache stands for them, of channel d; a = fl32(max_d max(|hi_d|, |lo_d|) /
 *   127), codes clamp(rint(fl32(x / a)), -127, 127), 0 if a = 0;
 *   up_d, down_d = sum of max(q_d, 0), min(q_d, 0) over the sequence's queries
 *   (all drafted tokens, all heads of the group), exact, rounded once to
 *   fp32; codes the same way, with the largest of both;
 *   score = fl32(sum_d (up_d hi_d + down_d lo_d, of the codes) * a).
 *
 * Without the roundings to codes no key of a page has a product with the
 * queries above its score.  Ties go to the earlier page.  A page whose keys
 * hold an infinity or NaN (scale NaN) comes before all others; queries that
 * do give codes of 0.  Pages whose entry in the table is missing are no
 * candidates.
 *
 * codes: device int8 [n_pages][kv_heads][2][head_dim] (hi, lo), 16-byte
 * aligned; scales: device fp32 [n_pages][kv_heads].  Both are the caller's.
 * summarize: of the pages pages[i] (device int32 [n]; numbers that are no
 * page's are passed over), all page_tokens tokens of each.                   */
int qgemv_kv_summarize(const qgemv_kv_cache* cache, const int32_t* pages, int64_t n, int8_t* codes, float* scales, void* stream);

/* Choose: pages (device int32 [n_seqs][kv_heads][width], width =
 * qgemv_kv_select_width, n_select and the pages that a context's end and 64
 * drafted tokens take; 0 for invalid sizes) gets, for each head, the chosen pages in
 * the context's order, then the table's entries from the last whole page on,
 * then -1; lens (device int32 [n_seqs]) the context's length over them: a page
 * table for qgemv_attn_pages.  Sequences, q, cu_q and the table as for
 * qgemv_attn_tree; cache's pages are not read; table_stride is at most
 * 49152.  Asynchronous on `stream`, no allocation, can be captured in a CUDA
 * graph; the same inputs give the same choice.                               */
int64_t qgemv_kv_select_width(int page_tokens, int64_t n_select);
int qgemv_kv_select(const qgemv_kv_cache* cache, const int8_t* codes, const float* scales, const int32_t* table,
                    int64_t table_stride, int64_t n_seqs, const int32_t* ctx_lens, const void* q, int64_t q_token_stride,
                    int64_t q_head_stride, int q_heads, const int32_t* cu_q, int64_t n_q, int64_t n_select, int32_t* pages,
                    int32_t* lens, void* stream);

/* qgemv_attn_tree with a page table for each key/value head: pages is device
 * int32 [n_seqs][kv_heads][pages_stride], and ctx_lens are lengths over it (as
 * qgemv_kv_select gives both).                                               */
int qgemv_attn_pages(const qgemv_kv_cache* cache, const int32_t* pages, int64_t pages_stride, int64_t n_seqs,
                     const int32_t* ctx_lens, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                     int q_heads, const int32_t* cu_q, int64_t n_q, const uint64_t* masks, int64_t max_ctx,
                     int64_t max_new, float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                     float* lse, void* ws, int64_t ws_bytes, void* stream);

/* Message and code of the last error on the calling thread ("" / 0 if none). */
const char* qgemv_last_error(void);
int qgemv_last_error_code(void);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H */
