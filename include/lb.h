/*
 * lb.h -- C ABI of the GB300 (sm_103a) low-bit product library.
 *
 * The library computes the products of packed low-bit weights and quantized activations that
 * dominate per-token time in low-bit LLM inference:
 *   - ggml Q1_0     : 128 sign bits + an fp16 scale per 18-byte block;
 *   - ggml Q2_0_g64 : 64 two-bit codes (code c means weight c-1) + an fp16 scale per 18 bytes;
 *   - planar ternary: one 16-byte {u64 pos, u64 neg} beat per 64 columns of a row;
 *   - a bf16 dense head.
 *
 * Sources the operations follow:
 *   [TR] "bankml: verified low-bit inference on commodity CPUs -- a technical report",
 *        sections III.2 (Q1_0 and its arithmetic), III.3 (float order, per-token activation
 *        scales, prefill tile), III.5 (Q2_0_g64), III.8 (offset code).
 *   [BH] bankml BUILD_HISTORY.md, ledger item "P2 -- own the kernels" (q8_0 quantizer: 127/amax,
 *        round half to even; Q2_0 codes (v >> 2r) & 3).
 *   [TA] tritium.technology "Architecture": section 1 (select-accumulate), 2 (bit planes),
 *        3 (bf16 dense head), 4.1 (int32 accumulators, x = -128), 5 (w_scale and x_scale applied
 *        as two multiplies).
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise, allocated and owned
 *     by the caller; the library allocates nothing and keeps no per-call state.
 *   - Every pointer must be 16-byte aligned (LB_ERR_ALIGN otherwise).
 *   - Matrices are row-major. Weights W are [N][K]: N output rows, K input columns.
 *     Activations are token-major [B][K] (or [M][K]); outputs are [B][N] (or [M][N]) fp32.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Every call
 *     only enqueues work on it and returns; results are ready when the stream is.
 *   - Every call returns LB_OK (0) or a negative LB_ERR_* code. Arguments are checked on the
 *     host before anything is enqueued; a refused call enqueues nothing. There is no fallback
 *     path: a device that is not sm_103 is refused with LB_ERR_ARCH.
 *   - Inputs must be finite; NaN or Inf activations give unspecified (but in-bounds) results.
 *   - Calls that write the same output buffer must not overlap on the GPU.
 *   - Kernels are launched with programmatic dependent launch: a GEMV may start streaming its
 *     WEIGHTS while the previous kernel of this library in the stream is still finishing, and
 *     waits for that kernel before touching activations or outputs.  lb_repack_* (the only call
 *     that writes weights) always completes before the next kernel starts; weights written by
 *     other code are read only after that code's kernels have completed.
 */
#ifndef LB_H_
#define LB_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LB_OK 0
#define LB_ERR_NULL (-1)    /* a required pointer is NULL */
#define LB_ERR_ALIGN (-2)   /* a pointer is not 16-byte aligned */
#define LB_ERR_SHAPE (-3)   /* a size is out of range or not a multiple of the block */
#define LB_ERR_BATCH (-4)   /* GEMV batch outside [1, 8] */
#define LB_ERR_ARCH (-5)    /* the current device is not compute capability 10.3 */
#define LB_ERR_LAUNCH (-6)  /* a CUDA launch or kernel setup call failed (lb_last_cuda_error) */
#define LB_ERR_DEVICE (-7)  /* a kernel gave up on a bounded wait (see lb_device_status) */

/* Name of a status code ("LB_OK", "LB_ERR_SHAPE", ...); never NULL. */
const char *lb_status_string(int status);

/* The cudaError_t value of the last CUDA call of this library that failed on the calling thread
 * (the cause behind LB_ERR_LAUNCH), then reset to 0; 0 if none failed since the last read. */
int lb_last_cuda_error(void);

/* CUDA's name for a cudaError_t value ("cudaErrorInvalidValue", ...); never NULL. */
const char *lb_cuda_error_name(int code);

/* Library version as 10000*major + 100*minor + patch. */
int lb_version(void);

/* Synchronizes `stream`, then reads and clears the current device's error word (a device
 * variable of the library whose address is looked up once per device and kept: do not use the
 * library across cudaDeviceReset).  Returns LB_OK,
 * or LB_ERR_DEVICE if a kernel of this library gave up on a bounded wait since the last call
 * (its outputs are then incomplete).  Kernels never hang: every wait gives up after about 2 s. */
int lb_device_status(void *stream);

/* Test hook for failure detection: the next Q1_0 / Q2_0_g64 / planar GEMV call (plain or
 * grouped) that runs on the streaming or lane-per-row kernel (1-2 tokens, or 3-8 tokens outside
 * the tensor-core kernel's shapes) makes its first CTA copy no weights, so that CTA's bounded
 * wait gives up after `wait_us` microseconds instead of about 2 s: the call then leaves part of
 * y unwritten and lb_device_status() reports LB_ERR_DEVICE.  So does the next product kernel of lb_gemv_q4, lb_gemm_q4
 * or lb_experts_q4, whichever comes first, with the first CTA that has work (parts of y are then wrong).  Nothing faults, traps or hangs.
 * One-shot, process-wide.  1 <= wait_us <= 10^6, else LB_ERR_SHAPE.  Not for production use. */
int lb_test_inject_wait_timeout(int wait_us);

/* ---------------------------------------------------------------------------------------
 * Activation quantizers
 * ------------------------------------------------------------------------------------- */

/* q8_0 ([TR] III.2, [BH]): for every token b and every block of 32 values,
 *   amax = max|x|, d = fp16_rne(amax / 127), id = amax != 0 ? 127 / amax : 0,
 *   q[i] = round_half_even(x[i] * id)  (binary32 arithmetic, IEEE division).
 *   x : [B][K] fp32.   q : [B][K] int8 (codes in [-127, 127]).
 *   d : [B][K/32] fp16 bit patterns.
 * K % 32 == 0, K >= 32, B >= 1 (LB_ERR_SHAPE otherwise). */
int lb_quantize_q8_0(const float *x, int8_t *q, uint16_t *d, int64_t B, int64_t K,
                     void *stream);

/* Per-token absmax int8 for the planar path (the pages say only "int8 activations"; the
 * reading is the plainest one): amax = max_k |x[b][k]|, s = amax != 0 ? 127/amax : 0,
 *   q[b][k] = clamp(round_half_even(x[b][k] * s), -128, 127), x_scale[b] = amax / 127.
 *   x : [B][K] fp32.  q : [B][K] int8.  x_scale : [B] fp32.
 * K % 16 == 0, K >= 16, B >= 1. */
int lb_quantize_i8_absmax(const float *x, int8_t *q, float *x_scale, int64_t B, int64_t K,
                          void *stream);

/* ---------------------------------------------------------------------------------------
 * Load-time repack: split the 18-byte source blocks into two aligned planes.
 *   blocks18 : [N][K/QK][18] source bytes (fp16 d little-endian, then 16 data bytes);
 *              QK = 128 for Q1_0, 64 for Q2_0_g64. This pointer needs no alignment.
 *   bits     : [N][K/QK * 16] data bytes, bit order unchanged.
 *   scales   : [N][S] fp16 bit patterns, S = LB_SCALE_STRIDE(K, QK) = K/QK rounded up to a
 *              multiple of 8, so every row of scales is 16-byte aligned; the S - K/QK padding
 *              entries of each row are written as 0.
 * Q1_0: K % 128 == 0. Q2_0_g64: K % 64 == 0. N >= 1.
 * ------------------------------------------------------------------------------------- */
#define LB_SCALE_STRIDE(K, QK) ((((K) / (QK)) + 7) / 8 * 8)
int lb_repack_q1_0(const void *blocks18, int64_t N, int64_t K, uint8_t *bits, uint16_t *scales,
                   void *stream);
int lb_repack_q2_0_g64(const void *blocks18, int64_t N, int64_t K, uint8_t *codes,
                       uint16_t *scales, void *stream);

/* ---------------------------------------------------------------------------------------
 * Decode GEMVs (batch B in [1, 8] tokens sharing the weights)
 *
 * Every GEMV exists in a single-matrix form and a grouped form.  The grouped form computes the
 * products of up to LB_MAX_GROUP weight matrices with the SAME activation in one launch (for
 * example the q, k and v projections, or gate and up), which amortizes the launch over all of
 * them; each matrix has its own rows N, weights and output.  The descriptor array is read on the
 * host during the call (it may be freed on return).  Output buffers must not overlap.
 * Shared memory bounds the activation: B * K * 1.25 bytes must stay below about 120 KB
 * (LB_ERR_SHAPE otherwise).
 * ------------------------------------------------------------------------------------- */
#define LB_MAX_GROUP 64

typedef struct lb_q_matrix {
    const uint8_t *bits;     /* [N][K/QK*16] repacked sign bytes (Q1_0) or code bytes (Q2_0_g64) */
    const uint16_t *scales;  /* [N][LB_SCALE_STRIDE(K, QK)] fp16 scales */
    float *y;                /* [B][N] fp32 output */
    int32_t *isum_opt;       /* NULL, or [B][N][K/32] int32 block sums (test hook) */
    int64_t N;               /* rows, 1 <= N <= 2^30 */
} lb_q_matrix;

typedef struct lb_trit_matrix {
    const uint64_t *planes;  /* [N][K/64][2] {pos, neg} beats */
    float w_scale;           /* per-tensor weight scale */
    float *y;                /* [B][N] fp32 output */
    int32_t *acc_opt;        /* NULL, or [B][N] int32 accumulators */
    int64_t N;               /* rows, 1 <= N <= 2^30 */
} lb_trit_matrix;

/* Q1_0 x q8_0 ([TR] III.2-III.3). For token b, row n, weight block k (128 weights) and its
 * four q8_0 blocks j:
 *   isum_j = sum_{i in j} s_i * q_i  (s_i = +1 for a set bit, -1 otherwise; integer, exact)
 *   y[b][n] = sum_k d_w[n][k] * sum_j d_x[b][j] * isum_j      (fp32 accumulation)
 *   bits   : [N][K/8] repacked sign bytes (lb_repack_q1_0).
 *   scales : [N][LB_SCALE_STRIDE(K, 128)] fp16 (lb_repack_q1_0).
 *   q, d   : q8_0 activations [B][K] int8, [B][K/32] fp16 (lb_quantize_q8_0 layout).
 *   y      : [B][N] fp32.
 *   isum_opt : NULL, or [B][N][K/32] int32 that receives every isum_j (a test hook; the same
 *              kernel writes it).
 * Accuracy: |y - exact| <= 1e-5 * sum |d_w d_x isum| + 1e-6, where exact is the real-number
 * value of the formula above. K % 128 == 0; N >= 1; B in [1, 8]. */
int lb_gemv_q1_0(const uint8_t *bits, const uint16_t *scales, const int8_t *q,
                 const uint16_t *d, float *y, int32_t *isum_opt, int64_t N, int64_t K, int B,
                 void *stream);

/* Grouped Q1_0 GEMV: mats[0..G-1] (host array, 1 <= G <= LB_MAX_GROUP) against one q8_0
 * activation q, d of B tokens and K columns; same arithmetic and limits as lb_gemv_q1_0. */
int lb_gemv_q1_0_grouped(const lb_q_matrix *mats, int G, const int8_t *q, const uint16_t *d,
                         int64_t K, int B, void *stream);

/* Q2_0_g64 x q8_0 ([TR] III.5, III.8): as lb_gemv_q1_0 with 64-weight blocks, weight i of a
 * block = ((codes byte i/4) >> 2*(i%4)) & 3, minus 1, in {-1, 0, +1, +2}, and two q8_0
 * blocks per weight block.
 *   codes : [N][K/4] repacked code bytes (lb_repack_q2_0_g64).
 *   scales : [N][LB_SCALE_STRIDE(K, 64)] fp16.
 * K % 64 == 0; N >= 1; B in [1, 8]. */
int lb_gemv_q2_0_g64(const uint8_t *codes, const uint16_t *scales, const int8_t *q,
                     const uint16_t *d, float *y, int32_t *isum_opt, int64_t N, int64_t K,
                     int B, void *stream);

/* Grouped Q2_0_g64 GEMV (see lb_gemv_q1_0_grouped). */
int lb_gemv_q2_0_g64_grouped(const lb_q_matrix *mats, int G, const int8_t *q, const uint16_t *d,
                             int64_t K, int B, void *stream);

/* Planar ternary select-accumulate ([TA] 1, 2, 4.1, 5):
 *   acc[b][r] = sum_{c: pos bit set} q[b][c] - sum_{c: neg bit set} q[b][c]   (int32, exact,
 *               correct for q = -128)
 *   y[b][r]   = (float(acc) * x_scale[b]) * w_scale   (two binary32 roundings, in this order)
 *   planes  : [N][K/64][2] u64, beat g of row r = {pos, neg}, bit c <-> column 64g + c,
 *             little-endian. A column set in both planes gives an unspecified result.
 *   q       : [B][K] int8.   x_scale : [B] fp32.   y : [B][N] fp32.
 *   acc_opt : NULL, or [B][N] int32 that receives acc.
 * K % 64 == 0; K <= 2^24 / 128 (so acc is exact in int32 and in binary32); N >= 1; B in [1,8].*/
int lb_gemv_trit_planes(const uint64_t *planes, float w_scale, const int8_t *q,
                        const float *x_scale, float *y, int32_t *acc_opt, int64_t N, int64_t K,
                        int B, void *stream);

/* Grouped planar GEMV: mats[0..G-1] (host array) against one activation q, x_scale. */
int lb_gemv_trit_planes_grouped(const lb_trit_matrix *mats, int G, const int8_t *q,
                                const float *x_scale, int64_t K, int B, void *stream);

/* Dense bf16 head ([TA] 3): y[b][n] = sum_k float(W[n][k]) * x[b][k], fp32 accumulation,
 * bf16 widened exactly (16-bit left shift).
 *   w : [N][K] bf16 bit patterns.   x : [B][K] fp32.   y : [B][N] fp32.
 * Accuracy: |y - exact| <= 1e-5 * sum_k |w x| + 1e-6. K % 8 == 0; N >= 1; B in [1, 8]. */
int lb_gemv_bf16(const uint16_t *w, const float *x, float *y, int64_t N, int64_t K, int B,
                 void *stream);

/* ---- Prefill GEMM ([TR] III.3: one weight block reused across several activation columns,
 * the prefill tile).  Same arithmetic and accuracy as the GEMVs above, for M tokens:
 *   y[m][n] = sum_k d_w[n][k] * sum_j d_x[m][j] * isum_j
 * computed on the tensor cores as exact per-32-column partial products d_w * isum_j (integers
 * times an fp16 scale, exact in binary32), each scaled by d_x[m][j] with one fused multiply-add
 * into a binary32 accumulator of at most 32 + K/1024 additions.
 *   bits / codes, scales : as lb_gemv_q1_0 / lb_gemv_q2_0_g64 (repacked).
 *   q, d      : q8_0 activations [M][K] int8 and [M][K/32] fp16.
 *   y         : [M][N] fp32, overwritten.
 *   workspace : device scratch of at least lb_gemm_workspace_bytes(M, K) bytes, owned by the
 *               caller; it receives the activations converted to the tensor-core operand
 *               layout, and must not be used by another call that may run at the same time.
 * Limits: 1 <= M, N <= 2^30; K % QK == 0 (QK = 128 for Q1_0, 64 for Q2_0_g64), K <= 2^24.
 * Q2_0_g64 weight scales must satisfy |d_w| <= 32752 (so that 2 * d_w is finite in fp16);
 * fp16 scales of real weights are many orders of magnitude smaller.
 * Errors: LB_ERR_NULL, LB_ERR_ALIGN, LB_ERR_SHAPE (shape limits, or a workspace too small),
 * LB_ERR_ARCH, LB_ERR_LAUNCH; a bounded wait that gives up sets the device status
 * (lb_device_status). */
size_t lb_gemm_workspace_bytes(int64_t M, int64_t K);  /* 0 for M < 1 or K < 1 */

int lb_gemm_q1_0(const uint8_t *bits, const uint16_t *scales, const int8_t *q, const uint16_t *d,
                 float *y, int64_t M, int64_t N, int64_t K, void *workspace,
                 size_t workspace_bytes, void *stream);

int lb_gemm_q2_0_g64(const uint8_t *codes, const uint16_t *scales, const int8_t *q,
                     const uint16_t *d, float *y, int64_t M, int64_t N, int64_t K,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Grouped prefill GEMM: mats[0..G-1] (host array, 1 <= G <= LB_GEMM_MAX_GROUP, read during
 * the call) against ONE q8_0 activation q, d of M tokens and K columns, in one launch -- for
 * example the q, k and v projections, or gate and up.  Same arithmetic, accuracy, workspace and
 * errors as the single-matrix calls, whose results it reproduces bit for bit; each matrix has
 * its own rows N, weights and output y [M][N].  Outputs must not overlap.  A convenience of this
 * library (the pages run projections one at a time); it lets small matrices (k, v: N = 1024)
 * share the GPU with the others instead of running alone. */
#define LB_GEMM_MAX_GROUP 8
typedef struct lb_gemm_matrix {
    const uint8_t *bits;     /* repacked sign bytes (Q1_0) or code bytes (Q2_0_g64) */
    const uint16_t *scales;  /* [N][LB_SCALE_STRIDE(K, QK)] fp16 */
    float *y;                /* [M][N] fp32 output */
    int64_t N;               /* rows, 1 <= N <= 2^30 */
} lb_gemm_matrix;

int lb_gemm_q1_0_grouped(const lb_gemm_matrix *mats, int G, const int8_t *q, const uint16_t *d,
                         int64_t M, int64_t K, void *workspace, size_t workspace_bytes,
                         void *stream);
int lb_gemm_q2_0_g64_grouped(const lb_gemm_matrix *mats, int G, const int8_t *q,
                             const uint16_t *d, int64_t M, int64_t K, void *workspace,
                             size_t workspace_bytes, void *stream);

/* ---- Planar ternary prefill GEMM ([TA] 1, 2, 4.1, 5 for the arithmetic; [TR] III.3 for the
 * prefill tile that reuses one weight tile across many tokens).  lb_gemv_trit_planes for each
 * of M tokens:
 *   acc[m][n] = sum_{c: pos bit set} q[m][c] - sum_{c: neg bit set} q[m][c]   (int32, exact)
 *   y[m][n]   = (float(acc) * x_scale[m]) * w_scale    (two binary32 roundings, in this order)
 * computed on the tensor cores with exact integer sums, so acc and y are bit-identical to the
 * GEMV's for the same token.
 *   planes    : [N][K/64][2] u64 {pos, neg} beats (layout of lb_gemv_trit_planes).
 *   q         : [M][K] int8 (for example lb_quantize_i8_absmax).   x_scale : [M] fp32.
 *   y         : [M][N] fp32, overwritten.   acc_opt : NULL, or [M][N] int32 that receives acc.
 *   workspace : device scratch of at least lb_gemm_trit_workspace_bytes(M, K) bytes (the same
 *               size as lb_gemm_workspace_bytes), owned by the caller and rewritten by every
 *               call with the activations in the tensor-core operand layout; it must not be
 *               used by another call that may run at the same time.  Its contents need no
 *               initialization.
 * Calls with few tiles split K across the CTAs of a thread-block cluster; the integer partial
 * sums are added exactly, so the split never changes a result.
 * Limits: 1 <= M, N <= 2^30; K % 64 == 0, 64 <= K <= 2^24 / 128 (so |acc| <= 2^24 and every
 * partial sum is exact in binary32).  A column set in both planes gives an unspecified result.
 * Errors: LB_ERR_NULL, LB_ERR_ALIGN, LB_ERR_SHAPE (limits, or a workspace too small),
 * LB_ERR_ARCH, LB_ERR_LAUNCH; a bounded wait that gives up sets the device status. */
size_t lb_gemm_trit_workspace_bytes(int64_t M, int64_t K);  /* 0 for M < 1 or K < 1 */

int lb_gemm_trit_planes(const uint64_t *planes, float w_scale, const int8_t *q,
                        const float *x_scale, float *y, int32_t *acc_opt, int64_t M, int64_t N,
                        int64_t K, void *workspace, size_t workspace_bytes, void *stream);

/* Grouped planar prefill GEMM: mats[0..G-1] (host array of lb_trit_matrix, 1 <= G <=
 * LB_GEMM_MAX_GROUP, read during the call) against ONE activation q, x_scale of M tokens, in one
 * launch (for example q, k and v, or gate and up).  Same arithmetic, limits, workspace and
 * errors as lb_gemm_trit_planes; each matrix has its own rows N, w_scale, output y [M][N] and
 * optional acc [M][N]; outputs must not overlap. */
int lb_gemm_trit_planes_grouped(const lb_trit_matrix *mats, int G, const int8_t *q,
                                const float *x_scale, int64_t M, int64_t K, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Quantize-then-GEMM in two launches instead of three: lb_quantize_i8_absmax_tiles quantizes x
 * [M][K] fp32 exactly as lb_quantize_i8_absmax (q and x_scale bit-identical) and also writes into
 * `workspace` the activation operand tiles that lb_gemm_trit_planes* would build from q in a
 * prologue launch; lb_gemm_trit_planes_grouped_tiles then runs the grouped planar GEMM from those
 * tiles (no q argument, no prologue).  Outputs, limits and errors as lb_gemm_trit_planes_grouped.
 *   workspace : at least lb_gemm_trit_workspace_bytes(M, K) bytes; between the two calls it must
 *               not be used by any other call (the GEMM reads the tiles the quantizer wrote;
 *               several GEMMs may read them in turn, for example q|k|v and a second group).
 * Limits of the quantizer: 1 <= M <= 2^30; K % 64 == 0, 64 <= K <= 2^24 / 128.  Errors:
 * LB_ERR_NULL, LB_ERR_ALIGN (x, q, x_scale or workspace not 16-byte aligned), LB_ERR_SHAPE
 * (limits, or a workspace too small), LB_ERR_ARCH, LB_ERR_LAUNCH. */
int lb_quantize_i8_absmax_tiles(const float *x, int8_t *q, float *x_scale, int64_t M, int64_t K,
                                void *workspace, size_t workspace_bytes, void *stream);
int lb_gemm_trit_planes_grouped_tiles(const lb_trit_matrix *mats, int G, const float *x_scale,
                                      int64_t M, int64_t K, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------------
 * Dequantization ([TR] III.4 and IV.2: every weight of a tensor dequantized and compared with
 * the reference's floats; III.2 and III.5 define w).  Every weight as the binary32 product
 *   out[n][k] = (float)w[n][k] * d      (exact: w in {-1, +1} or {-1, 0, +1, +2})
 * with d the fp16 block scale widened to binary32 (Q1_0, Q2_0_g64, from the repacked planes)
 * or w_scale (planar, w in {-1, 0, +1}).  A zero weight gives +0 or -0 with the sign of d.
 *   out_format LB_OUT_F32  : out [N][K] fp32.
 *   out_format LB_OUT_BF16 : out [N][K] bf16 bit patterns, the binary32 value rounded to
 *                            nearest, ties to even (the pages print no bf16 weights; this is
 *                            the plainest reading).
 * Q1_0: K % 128 == 0; Q2_0_g64 and planar: K % 64 == 0; 1 <= N <= 2^30, K <= 2^26.
 * Errors: LB_ERR_NULL, LB_ERR_ALIGN, LB_ERR_SHAPE (also an unknown out_format), LB_ERR_ARCH,
 * LB_ERR_LAUNCH. */
#define LB_OUT_F32 0
#define LB_OUT_BF16 1
int lb_dequantize_q1_0(const uint8_t *bits, const uint16_t *scales, int64_t N, int64_t K,
                       int out_format, void *out, void *stream);
int lb_dequantize_q2_0_g64(const uint8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                           int out_format, void *out, void *stream);
int lb_dequantize_trit_planes(const uint64_t *planes, float w_scale, int64_t N, int64_t K,
                              int out_format, void *out, void *stream);

/* ---------------------------------------------------------------------------------------
 * Base-3 packed ternary weights ([TR] III.8: 3^5 = 243 <= 256, five trits per byte, 1.6 bits
 * per trit; [TA] open questions: base-3 packing against its unpack cost).  The pages fix no
 * layout; this library's reading: byte j of 16-byte group g of a row holds columns
 * 80g + 5j + i (i = 0..4) as sum_i (t + 1) * 3^i, the lowest column in the lowest digit; a row
 * is LB_BASE3_ROW_BYTES(K) = ceil(K/80) * 16 bytes and columns past K hold trit 0.
 * ------------------------------------------------------------------------------------- */
#define LB_BASE3_ROW_BYTES(K) ((((K) + 79) / 80) * 16)

/* Load-time packing from the planar layout:
 *   planes : [N][K/64][2] u64 {pos, neg} (layout of lb_gemv_trit_planes; a column set in both
 *            planes gives an unspecified byte).
 *   packed : [N][LB_BASE3_ROW_BYTES(K)] bytes, every byte written (values 0..242).
 * Like lb_repack_*, it completes before the next kernel of this library starts.
 * K % 64 == 0, 64 <= K <= 2^24 / 128; 1 <= N <= 2^30. */
int lb_pack_base3(const uint64_t *planes, int64_t N, int64_t K, uint8_t *packed, void *stream);

/* Decode GEMV on base-3 packed weights, the planar arithmetic ([TA] 1, 4.1, 5):
 *   acc[b][r] = sum_{c: t = +1} q[b][c] - sum_{c: t = -1} q[b][c]     (int32, exact)
 *   y[b][r]   = (float(acc) * x_scale[b]) * w_scale                    (two roundings)
 * bit-identical to lb_gemv_trit_planes on the same trits.  A byte above 242 (never written by
 * lb_pack_base3) gives an unspecified, in-bounds result.
 *   packed : [N][LB_BASE3_ROW_BYTES(K)] (lb_pack_base3).   q : [B][K] int8.
 *   x_scale : [B] fp32.   y : [B][N] fp32.   acc_opt : NULL or [B][N] int32.
 * K % 64 == 0, 64 <= K <= 2^24 / 128; 1 <= N <= 2^30; B in [1, 8]; shared memory bounds the
 * activation: 32 KB + B * ceil(K/80) * 80 bytes must stay within 200 KB (LB_ERR_SHAPE). */
int lb_gemv_base3(const uint8_t *packed, float w_scale, const int8_t *q, const float *x_scale,
                  float *y, int32_t *acc_opt, int64_t N, int64_t K, int B, void *stream);

/* ---- Q2_0_g64 prefill GEMM without caller scratch.
 * No counterpart in the source pages: a convenience of this library for callers that cannot
 * allocate device memory.  Same arithmetic, accuracy, layouts and errors as lb_gemm_q2_0_g64,
 * but the converted activations go to a fixed scratch array of LB_NOALLOC_SCRATCH_BYTES inside
 * the library (a file-scope device array; the call itself allocates nothing).
 *   Limit: round_up(M, 128) * K * 2 <= LB_NOALLOC_SCRATCH_BYTES (8 MiB), e.g. M = 512 with
 *   K <= 8192, or M <= 256 with K = 12288; larger sizes are refused with LB_ERR_SHAPE before any
 *   device work.  Nothing in the scratch needs to start at zero.
 *   There is one scratch per device: calls that may run at the same time on one device (another
 *   stream, another host thread) race on it and give wrong results; serialize them.
 *   The first call on each device looks the scratch up (cudaGetSymbolAddress).  Under lazy
 *   module loading that lookup may load the library's device code, and the driver then
 *   reserves the 8 MiB array: a one-time allocation by the driver, not by this call.  Make one
 *   warm-up call per device before an allocation-free region or a stream capture.
 *   The looked-up address is kept for the life of the process: do not use the library across
 *   cudaDeviceReset (the same holds for every entry point's device error word). */
#define LB_NOALLOC_SCRATCH_BYTES (8u << 20)

int lb_gemm_q2_0_g64_noalloc(const uint8_t *codes, const uint16_t *scales, const int8_t *q,
                             const uint16_t *d, float *y, int64_t M, int64_t N, int64_t K,
                             void *stream);

/* ---------------------------------------------------------------------------------------
 * Serving step: what stands between the products of one decoder layer and after its head.  No
 * counterpart in the source pages; conveniences of this library for a server that keeps its
 * keys and values in a paged cache of 4-bit codes:
 *   lb_kv_plan        pages and slots of a step's new tokens from the requests' lengths
 *   lb_kv4_append     new keys and values -> cache;  lb_dequantize_kv4: cache -> values
 *   lb_attn_kv4       attention of the new tokens over the cache
 *   lb_logits_adjust  penalties, biases and grammar masks on the head's logits
 *
 * Cache: one byte buffer [pages][kv_heads][page_size / 16][16 * (head_dim + 8)], page_size in
 * {16, 32, 64, 128, 256}, head_dim in {64, 128}, kv_heads up to 16384.  The innermost piece, a chunk, holds 16
 * consecutive tokens of one head:
 *   16 key rows of head_dim/2 bytes, 16 value rows of head_dim/2 bytes (the code of dimension 2j
 *   in the low half of byte j, of 2j + 1 in the high half),
 *   16 key pairs {d, z}, 16 value pairs {d, z}, each two fp16.
 * A code c in 0..15 stands for d * (c - z); z is a whole number in 0..15.  A token's slot is
 * page * page_size + its place in the page.
 * ------------------------------------------------------------------------------------- */
#define LB_KV4_CHUNK 16
#define LB_KV4_CACHE_BYTES(pages, kv_heads, page_size, head_dim) \
    ((size_t)(pages) * (size_t)(kv_heads) * (size_t)(page_size) * ((size_t)(head_dim) + 8))
#define LB_KV_MAX_REQUESTS 8192

/* Page plan of one step.  Request r holds past[r] tokens in the cache and brings fresh[r] new
 * ones (0 allowed; a negative length counts as 0).  With P = page_size,
 *   have[r] = ceil(past[r] / P),  take[r] = ceil((past[r] + fresh[r]) / P) - have[r],
 *   first[r] = sum of take[0..r-1]:
 *   block_table[r][have[r] + i] = free_pages[from + first[r] + i], i < take[r]  (other entries
 *               stay; from = free_from_opt ? *free_from_opt : 0)
 *   q_start[r]  = sum of fresh[0..r-1], r = 0..R
 *   kv_len[r]   = past[r] + fresh[r]
 *   position[t] = past[r] + (t - q_start[r]) of the request r that new token t belongs to
 *   slot[t]     = block_table[r][position / P] * P + position % P
 *   counts      = {q_start[R], from + first[R]}: the new tokens, and the first entry of
 *               free_pages that is still free (the next step's free_from).
 *   past, fresh : [R] int32.   free_pages : [n_free] int32.   block_table : [R][table_width]
 *   int32, read and written.   q_start : [R + 1] int32.   kv_len : [R] int32.
 *   position : [T] int32, slot : [T] int64; entries past q_start[R] are set to -1.
 *   counts : [2] int32.
 * No output may overlap past, fresh, free_pages or free_from_opt (LB_ERR_SHAPE): lengths that
 * advance in place need a second buffer, as counts does.
 * Where free_pages runs out or a row of the table is full, the entries without a page are -1
 * and the slots of their tokens are -1 (lb_kv4_append skips them and lb_attn_kv4 does not see
 * them); counts[1] > n_free tells of the first case, counts[0] > T that tokens were left out.
 * The pages of one call are different if those of free_pages are.
 * 1 <= R <= LB_KV_MAX_REQUESTS; 0 <= n_free, T < 2^31; 1 <= table_width < 2^31; sums of lengths
 * below 2^31.  4-byte alignment (slot: 8).  free_pages may be NULL if n_free is 0; position and
 * slot if T is 0. */
int lb_kv_plan(const int32_t *past, const int32_t *fresh, int64_t R, const int32_t *free_pages,
               int64_t n_free, const int32_t *free_from_opt, int page_size,
               int32_t *block_table, int64_t table_width, int64_t T, int32_t *q_start,
               int32_t *kv_len, int32_t *position, int64_t *slot, int32_t *counts, void *stream);

/* New keys and values -> cache.  For each token t, head h and each of its two rows x of head_dim
 * values, in binary32 arithmetic with IEEE division and round-half-even:
 *   lo = min(min x, 0), hi = max(max x, 0), d = fp16_rne(min((hi - lo) / 15, 65504)),
 *   id = d != 0 ? 1 / d : 0,  z = clamp(rne(-lo * id), 0, 15),
 *   c_i = clamp(rne(x_i * id) + z, 0, 15).
 *   k, v : [T][kv_heads][head_dim], fp32 (type LB_OUT_F32) or bf16 (LB_OUT_BF16); a token's heads
 *          lie together, tokens k_stride / v_stride elements apart (slices of one q|k|v buffer).
 *   slot : [T] int64; a token whose slot is not in [0, pages * page_size) is skipped.  Tokens of
 *          one call have different slots.
 *   cache: LB_KV4_CACHE_BYTES(pages, kv_heads, page_size, head_dim) bytes.
 * Rows with NaN or infinite values store unspecified codes and scales of their own row.
 * 0 <= T < 2^31 (0: nothing is done; k, v and slot may be NULL); strides >= kv_heads * head_dim; k, v, cache and the strides
 * in bytes 16-byte aligned, slot 8-byte. */
int lb_kv4_append(const void *k, const void *v, int type, int64_t k_stride, int64_t v_stride,
                  const int64_t *slot, int64_t T, uint8_t *cache, int64_t pages, int page_size,
                  int kv_heads, int head_dim, void *stream);

/* Cache -> values: k[t][h][i] = d * (c - z) of slot[t]'s key row of head h, v likewise (the exact
 * binary32 product; out_format LB_OUT_BF16 rounds it to nearest even).  A token whose slot is not in
 * [0, pages * page_size) gives zeros.  k, v : [T][kv_heads][head_dim], 16-byte aligned.  T = 0 as in lb_kv4_append. */
int lb_dequantize_kv4(const uint8_t *cache, int64_t pages, int page_size, int kv_heads,
                      int head_dim, const int64_t *slot, int64_t T, int out_format, void *k,
                      void *v, void *stream);

/* Attention over the cache.  Request r's queries are the rows t in [q_start[r], q_start[r + 1])
 * of q; row t is token kv_len[r] - n + i of its request (n its rows, i = t - q_start[r]) and head
 * h reads key/value head h / (heads / kv_heads):
 *   visible(t) = { j : 0 <= j < kv_len[r], j <= position(t) if causal,
 *                  j > position(t) - window if window > 0 }
 *   s_j = scale * sum_i q[t][h][i] * k_j[i],
 *   out[t][h] = sum_j softmax_j(s) * v_j over visible(t), lse[t][h] = ln sum_j exp(s_j).
 * A row that sees nothing (kv_len[r] = 0, or fewer tokens than queries) gives out = 0 and
 * lse = -inf.  Tokens on a page whose block_table entry is not in [0, pages) are not seen.
 *   q, out : [T][heads][head_dim], both fp32 (type LB_OUT_F32) or both bf16 (LB_OUT_BF16); tokens
 *            q_stride / out_stride elements apart.  out may not overlap q.
 *   block_table : [R][table_width] int32.   q_start : [R + 1] int32, not falling, within [0, T].
 *   kv_len : [R] int32, at most table_width * page_size (more is not read).
 *   lse_opt: NULL, or [T][heads] fp32.
 *   workspace : at least lb_attn_kv4_workspace_bytes(heads, kv_heads, head_dim, max_q) bytes, owned
 *            by the caller, not used by another call that may run at the same time; its contents
 *            need no initialization.
 *   max_q  : an upper bound of every request's number of queries, read on the host to choose the
 *            kernels (a request with more is computed all the same, on slower ones).
 * Sums, softmax statistics and outputs accumulate in binary32.  Weights and queries enter the
 * tensor cores as fp16: with fp32 tensors in two parts (22 bits), with bf16 ones in one (weights
 * round to 11 bits, queries are exact; up to four rows per key/value head take two).  The parts end
 * 2^-28 below a row's largest weight times value scale: what is smaller than 2^-6 (one part:
 * 2^-17) of that keeps fewer bits.  Scores' sums are cut by the tensor cores: a score is off by up to 2^-20 of
 * scale * 15 * its key's d * sum_i |q_i|, with bf16 tensors and few rows also by up to 2^-13 of
 * scale * 15 * d * max_i |q_i| (codes enter as fp16 subnormals there).  Scores are expected below
 * 2^20 in size: beyond, binary32 no longer tells close ones apart, and a row's values are unspecified.
 * heads % kv_heads == 0, heads / kv_heads <= 64; 1 <= R <= LB_KV_MAX_REQUESTS; 0 <= T (0: nothing
 * is done; q and out may be NULL), T * heads / kv_heads < 2^31; 1 <= table_width, table_width * page_size <= 2^30; max_q >= 1; 0 < scale
 * finite; window >= 0, and 0 without causal; 16-byte alignment of q, out, cache, workspace and the
 * two strides in bytes, 4-byte of the others. */
size_t lb_attn_kv4_workspace_bytes(int heads, int kv_heads, int head_dim, int64_t max_q);
int lb_attn_kv4(const void *q, int type, int64_t q_stride, const uint8_t *cache, int64_t pages,
                int page_size, int heads, int kv_heads, int head_dim, const int32_t *block_table,
                int64_t table_width, const int32_t *q_start, const int32_t *kv_len, int64_t R,
                int64_t T, int64_t max_q, float scale, int causal, int64_t window, void *out,
                int64_t out_stride, float *lse_opt, void *workspace, size_t workspace_bytes,
                void *stream);

/* Penalties, biases and grammar masks on logits.  Row b, token v, in binary32:
 *   x = logits[b][v]
 *   v in b's prompt or output:  x = x > 0 ? x / repetition[b] : x * repetition[b]
 *   v n > 0 times in b's output: x = (x - n * frequency[b]) - presence[b]
 *   v in b's bias list:         x = x + its value (the later entry's if v stands there twice)
 *   v not allowed by b's mask:  x = -inf, whatever it was
 *   out[b][v] = x
 * The lists are rows of one array: list b is ids[start[b] .. start[b + 1] - 1], start int32
 * [B + 1], not falling; ids int32; an id outside [0, V) is skipped.  Of a row's bias list the first
 * LB_LOGITS_MAX_BIAS entries count; a token stands less than 2^30 times in a list.  NULL ids, values of [B] or mask
 * leave a step out (repetition without lists does nothing).  mask : uint32 words, bit
 * v % 32 of word v / 32 allows v; row mask_row_opt[b] of mask_rows rows, mask_stride words apart, or
 * row b if mask_row_opt is NULL (mask_rows >= B then); a row outside [0, mask_rows) means no mask.
 *   logits, out : [B][V] fp32 (type LB_OUT_F32) or bf16 (LB_OUT_BF16), rows `stride` elements
 *                 apart; out may be logits itself (same stride).
 * 1 <= B <= 65535; 1 <= V <= LB_LOGITS_MAX_V; strides >= V; mask_stride >= ceil(V / 32).
 * Pointers aligned to their elements (16-byte rows are fastest). */
#define LB_LOGITS_MAX_V 400000
#define LB_LOGITS_MAX_BIAS 65535
typedef struct lb_logit_rules {
    const int32_t *prompt_ids, *prompt_start;
    const int32_t *output_ids, *output_start;
    const float *repetition, *presence, *frequency;  /* [B] each, or NULL */
    const int32_t *bias_ids;
    const float *bias_values;
    const int32_t *bias_start;
    const uint32_t *mask;
    int64_t mask_stride, mask_rows;
    const int32_t *mask_row_opt;
} lb_logit_rules;
int lb_logits_adjust(const void *logits, int type, int64_t stride, void *out, int64_t out_stride,
                     int64_t B, int64_t V, const lb_logit_rules *rules, void *stream);

/* ---------------------------------------------------------------------------------------
 * 4-bit weights with group scales, and the mixture of experts around them.  No counterpart in the
 * source pages; conveniences of this library for models that keep some of their matrices in 4 bits:
 *   lb_gemv_q4, lb_gemm_q4   y = W x for one to eight tokens, for any number
 *   lb_route                 gate logits -> experts, weights, and the tokens of each expert
 *   lb_experts_q4            the experts' gated feed-forward blocks, added up per token
 *
 * Weights [N][K]: codes [N][K / 2] bytes, column 2j in the low half of byte j and 2j + 1 in the high
 * one; scales [N][LB_SCALE_STRIDE(K, group)] fp16, one for `group` columns; zeros_opt NULL or [N]
 * [LB_SCALE_STRIDE(K, group)] bytes, one for `group` columns, 0..15.  A code c stands for
 *   w = d * (c - z),   z = 8 without zeros.
 * (What lies in a row's scales and zeros behind K / group is not used.)
 * group in {32, 64, 128}; K a multiple of it.  codes, scales and zeros 16-byte aligned.
 * Like the other products, these may read codes, scales and zeros while the previous kernel of
 * this library in the stream is still finishing.
 * ------------------------------------------------------------------------------------- */
#define LB_Q4_MAX_K 32768

/* y[t][n] = sum_k w[n][k] x[t][k] for B in [1, 8] tokens (LB_ERR_BATCH otherwise), M of any number.
 *   x : [B][K], y : [B][N], both fp32 (type LB_OUT_F32) or both bf16 (LB_OUT_BF16); rows x_stride /
 *       y_stride elements apart.  y may not overlap x.
 *   workspace : at least lb_gemm_q4_workspace_bytes(M, N, K, type) bytes, 16-byte aligned, owned by the
 *       caller, not used by another call that may run at the same time; it needs no initialization.
 * Sums are held in binary32; c - z is exact.  A number of x enters with all of its bits if tensors are bf16, with 22
 * (two fp16 parts) if they are fp32, and loses at most 2^-39 of the largest of its 256 columns (up to eight tokens) or
 * of its row (more) where it is far smaller than that.  With bf16 tensors and more than eight tokens a weight
 * d * (c - z) rounds to 11 bits, beyond 65504 to infinity; otherwise a scale acts on its group's sum in binary32.
 * A token with a NaN or an infinite number gets nothing finite in its row of y; other rows do not change.
 * 1 <= N <= 2^23; group <= K <= LB_Q4_MAX_K; 0 <= M <= 2^20 (0: nothing is done; x and y may be NULL); x and its stride in
 * bytes 16-byte aligned, y aligned to its elements; strides >= K and N, below 2^31. */
int lb_gemv_q4(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros_opt, int group,
               const void *x, int type, int64_t x_stride, void *y, int64_t y_stride, int64_t N,
               int64_t K, int B, void *stream);
size_t lb_gemm_q4_workspace_bytes(int64_t M, int64_t N, int64_t K, int type);
int lb_gemm_q4(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros_opt, int group,
               const void *x, int type, int64_t x_stride, void *y, int64_t y_stride, int64_t M,
               int64_t N, int64_t K, void *workspace, size_t workspace_bytes, void *stream);

/* Routing of T tokens to k of E experts.  Token t, expert e, logit x (bf16 or fp32; +inf counts as
 * the largest finite number):
 *   score  s_e = exp(x_e) / sum of exp(x)  (LB_ROUTE_SOFTMAX)  or  1 / (1 + exp(-x_e))  (LB_ROUTE_SIGMOID)
 *   key    x_e if there is no bias and group_best is 1 (the logits' own order), else the binary64
 *          number s_e + bias_e (bias 0 without one; +inf allowed)
 *   An expert whose logit or bias is NaN or -inf is never chosen and adds nothing to a sum.
 *   With groups > 1, group g holds the experts [g E / groups, (g + 1) E / groups); its value is the sum
 *   of its group_best (1 or 2; fewer if fewer can be chosen) largest keys, and only the experts of the
 *   keep_groups groups of largest value can be chosen.
 *   ids[t]     = the k experts of largest key, in falling order (ties of keys and of groups: the lower
 *                index first); -1 where there are no more
 *   weights[t] = scale * s_e, with renormalize scale * s_e / sum of the chosen experts' s; 0 at -1
 *   expert_start[e], e = 0..E : the number of pairs (t, j) with 0 <= ids[t][j] < e
 *   order      = the pairs t * k + j with ids[t][j] >= 0, by expert and then by t; -1 behind them
 * Tokens from *live_opt on (NULL: none; below 0 counts as 0) get ids -1 and weights 0, and their logits are not read.
 *   logits : [T][E] fp32 (type LB_OUT_F32) or bf16 (LB_OUT_BF16), rows `stride` elements apart.
 *   ids : [T][k] int32.  weights : [T][k] fp32.  expert_start : [E + 1] int32.  order : [T * k] int32.
 *   workspace : lb_route_workspace_bytes(T, E) bytes (never fewer for more tokens), 16-byte aligned, as above.
 * Scores are computed in binary32, and in binary64 where two keys lie too close together for that;
 * exp(x - max) of experts more than 100 below the row's largest logit counts as 0 in the weights; a weight below 2^-126
 * (before the scale) may lose bits or be 0.
 * 0 <= T <= 2^20 (at 0 only expert_start is written; logits, ids, weights and order may be NULL); 1 <= E <= LB_ROUTE_MAX_EXPERTS; 1 <= k <= min(E,
 * LB_ROUTE_MAX_CHOSEN); groups <= 32 divides E; 1 <= keep_groups <= groups; stride >= E; pointers aligned to
 * their elements. */
#define LB_ROUTE_SOFTMAX 0
#define LB_ROUTE_SIGMOID 1
#define LB_ROUTE_MAX_EXPERTS 1024
#define LB_ROUTE_MAX_CHOSEN 32
typedef struct lb_route_rules {
    int32_t scoring, groups, keep_groups, group_best, renormalize;
    float scale;
    const float *bias_opt;   /* [E] */
    const int32_t *live_opt; /* [1] */
} lb_route_rules;
size_t lb_route_workspace_bytes(int64_t T, int E);
int lb_route(const void *logits, int type, int64_t stride, int64_t T, int E, int k,
             const lb_route_rules *rules, int32_t *ids, float *weights, int32_t *expert_start,
             int32_t *order, void *workspace, size_t workspace_bytes, void *stream);

/* The experts' blocks.  Expert e has gate and up rows in one matrix up_e [2 ffn][hidden] (rows 0..ffn-1
 * the gate's) and down_e [hidden][ffn]; both are arrays of E matrices, one behind the other.
 *   h = silu(gate_e x[t]) * (up_e x[t]),   silu(v) = v / (1 + exp(-v))
 *   y[t] = sum over j with ids[t][j] >= 0 of weights[t][j] * (down_e h),  e = ids[t][j]
 * A token without experts gets zeros.
 *   x, y : [T][hidden], both fp32 or both bf16 (type), rows x_stride / y_stride elements apart; y may not
 *          overlap x.
 *   ids, weights, expert_start, order : as lb_route leaves them.  ids at -1 are left out; the experts'
 *          pairs are those of order and expert_start (not falling, at most T * k; entries of order outside
 *          [0, T * k) are passed over).  The sum over j runs from 0 on.
 *   workspace : lb_experts_q4_workspace_bytes(T, E, k, hidden, ffn, type) bytes, 16-byte aligned, as above.
 * Precision as in lb_gemv_q4 / lb_gemm_q4 (weights may round to 11 bits with bf16 tensors, whatever the number of
 * tokens).  h enters the down rows' products with 11 bits where tensors are bf16 and with 22 where they are fp32, below
 * its largest value as x does; the experts' outputs are binary32.
 * 0 <= T (0: nothing is done; x, y, ids, weights and order may be NULL), T * k <= 2^24; 1 <= E <= LB_ROUTE_MAX_EXPERTS; 1 <= k <= LB_ROUTE_MAX_CHOSEN; hidden and
 * ffn multiples of group, at most LB_Q4_MAX_K; alignment as in lb_gemv_q4, 4-byte for the routing's. */
size_t lb_experts_q4_workspace_bytes(int64_t T, int E, int k, int64_t hidden, int64_t ffn, int type);
int lb_experts_q4(const void *x, int type, int64_t x_stride, int64_t T, int E, int k, int64_t hidden,
                  int64_t ffn, int group, const uint8_t *up_codes, const uint16_t *up_scales,
                  const uint8_t *up_zeros_opt, const uint8_t *down_codes, const uint16_t *down_scales,
                  const uint8_t *down_zeros_opt, const int32_t *ids, const float *weights,
                  const int32_t *expert_start, const int32_t *order, void *y, int64_t y_stride,
                  void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LB_H_ */
