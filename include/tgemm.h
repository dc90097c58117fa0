/*
 * tgemm -- layout-aware bf16 GEMM for MI355X (gfx950) with fused epilogues.
 *
 * One C-ABI library.  Plain pointers and sizes only; every data pointer is a
 * DEVICE pointer owned by the caller, and every call is asynchronous on the
 * caller's HIP stream.
 *
 * What is computed
 * ----------------
 *   Y = op(A) . op(B),  op(X) = X for 'N' and X^T for 'T'.
 *
 *   The transpose is a flag, never a copy: a weight stored [N,K] row-major is
 *   read in place as op(B) with transB = 'T' ("Strength reduction: fold
 *   transpose into a subsequent GEMM call", the trace and its discussion of
 *   NT GEMMs; the pitch asks for GEMMs that take transpose arguments).
 *
 * Storage convention (row-major, leading dimension = row stride in elements)
 *   A 'N': [M,K], element (m,k) at A[m*lda + k]     lda >= K
 *   A 'T': [K,M], element (m,k) at A[k*lda + m]     lda >= M
 *   B 'N': [K,N], element (k,n) at B[k*ldb + n]     ldb >= N
 *   B 'T': [N,K], element (k,n) at B[n*ldb + k]     ldb >= K
 *   C    : [M,N], element (m,n) at C[m*ldc + n]     ldc >= N (>= 2N for ROPE)
 *
 * Epilogues (argument `epilogue`)
 *   TGEMM_EPI_STORE_BF16   A, B bf16 -> C bf16, fp32 accumulation, output
 *                          rounded to nearest even.
 *   TGEMM_EPI_STORE_F32    A, B bf16 -> C fp32 (the raw accumulator).
 *   TGEMM_EPI_CE           A, B bf16; the logits y = op(A).op(B) (fp32) are
 *                          reduced per row and never written out:
 *                            loss[m] = logsumexp_n y[m,n] - y[m, labels[m]]
 *                          written to out_loss (fp32[M]).  If out_grad is not
 *                          NULL it receives softmax(y) - onehot(labels) as
 *                          bf16 [M,N] with row stride ldc.  C is ignored.
 *                          ("Allow reductions in matmul epilogues": the
 *                          attempted fusion defines the max / exp / sum / log
 *                          steps, the loss and the softmax-minus-one-hot
 *                          output; its answer on tile-wise row reductions
 *                          describes the cross-tile combine.)
 *                          Labels outside [0,N) are not checked on the host:
 *                          that row's loss is NaN and its gradient row is the
 *                          plain softmax.  No mean over rows, no scaling.
 *   TGEMM_EPI_OUTER_F32    K must be 1.  A, B fp32; C fp32 [M,N] = the exact
 *                          fp32 products a[m]*b[n].
 *   TGEMM_EPI_ROPE_COSSIN  K must be 1.  A int64 positions (cast to fp32 in
 *                          the kernel; exact for |p| < 2^24), B fp32 inverse
 *                          frequencies.  t = fp32(a[m]) * b[n];
 *                          C        = cos(t) as bf16 at columns n and n+N,
 *                          out_grad = sin(t) as bf16 at columns n and n+N,
 *                          both [M, 2N] with row stride ldc.
 *                          ("Schedule a small matmul op as a reduction (or
 *                          pointwise) op": the %kernel_math listing's K=1
 *                          matmul, permute, duplicating cat and cos/cast, and
 *                          the proposed broadcast-multiply decomposition.)
 *
 *   Every call with K == 1 runs pointwise, without matrix cores, as that
 *   page proposes for K=1 matmuls: the STORE epilogues as an outer product,
 *   CE as a per-row reduction of the logits a[m]*b[n] (bf16 operands, the
 *   products exact in fp32).
 *
 * Errors
 *   Arguments are validated before anything is enqueued; on any error
 *   nothing is written.  No exceptions cross the ABI.  The call returns
 *   after enqueueing and never synchronises; faults inside a kernel surface
 *   at the caller's next synchronisation.  Outputs must not alias inputs.
 *
 * Workspace
 *   TGEMM_EPI_CE needs a small scratch buffer (per row and per 128-column
 *   block: the block max and block sum of exponentials, plus per row the
 *   label logit and the logsumexp).  A store-epilogue GEMM whose tiles
 *   alone do not fill the GPU (few output tiles, long K; both operands
 *   K-contiguous) splits K into chunks and needs one fp32 M x N partial
 *   product per chunk; a second kernel adds them in chunk order.
 *   The library keeps one workspace buffer per (device, stream): calls on
 *   a stream run in order and reuse it; it grows with hipFreeAsync /
 *   hipMallocAsync on that stream, so calls on different streams never
 *   share memory.  While `stream` is being captured into a graph, its calls
 *   take a buffer of that capture instead (device memory allocated beside
 *   the capture; a replay allocates nothing).  Graphs never share one.
 *
 * Threads
 *   tgemm_run may be called from several host threads, on the same stream
 *   or on different ones.  A call holds its stream's workspace entry from
 *   the lookup until its last kernel is enqueued, so concurrent calls on
 *   one stream are enqueued one after the other and never see a buffer
 *   freed under them.  The tuning knobs (tgemm_set_*) are process-wide and
 *   must not change while calls are in flight.
 *
 * Retention
 *   A stream's cached buffer is held until the process ends or until
 *   tgemm_release_workspace(stream) frees it; a program that creates many
 *   short-lived streams should release each one's buffer before destroying
 *   the stream.  A stream must not be destroyed while a tgemm call on it is
 *   still executing.  A capture's buffer is held until the process ends,
 *   for a graph may be replayed at any time: one per capture with a call
 *   that needs workspace (a program that captures anew without end takes
 *   tgemm_run_noalloc).
 */
#ifndef TGEMM_H
#define TGEMM_H

#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define TGEMM_API __attribute__((visibility("default")))
#else
#define TGEMM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TGEMM_OK = 0,
  TGEMM_ERR_INVALID_ARG = -1, /* a flag, size, leading dimension or pointer is invalid */
  TGEMM_ERR_UNSUPPORTED = -2, /* valid request this library does not implement      */
  TGEMM_ERR_HIP = -3,         /* the HIP runtime reported an error while enqueueing   */
  TGEMM_ERR_NO_MEMORY = -4,   /* a CE or split-K workspace could not be allocated     */
  TGEMM_ERR_WORKSPACE_LIMIT = -5 /* tgemm_run_noalloc: the call needs more scratch than
                                    its fixed buffer holds (tgemm_noalloc_scratch_bytes);
                                    feed-forward calls: more than the caller's workspace
                                    holds, or any under graph capture without one */
} tgemm_status;

typedef enum {
  TGEMM_EPI_STORE_BF16 = 0,
  TGEMM_EPI_STORE_F32 = 1,
  TGEMM_EPI_CE = 2,
  TGEMM_EPI_OUTER_F32 = 3,
  TGEMM_EPI_ROPE_COSSIN = 4
} tgemm_epilogue;

/*
 * Run one GEMM with the chosen epilogue on `stream` (a hipStream_t; NULL is
 * the null stream).
 *
 *   transA, transB  'N'/'n' or 'T'/'t' (see the storage convention above).
 *   M, N, K         >= 1 and < 2^31.
 *   A, lda          operand A (bf16; fp32 for OUTER_F32; int64 for ROPE).
 *   B, ldb          operand B (bf16; fp32 for OUTER_F32 and ROPE).
 *   C, ldc          output (bf16 or fp32; cos table for ROPE; unused by CE).
 *                   For CE, ldc is the row stride of out_grad.
 *   labels          CE only: int32[M].
 *   out_loss        CE only: fp32[M].
 *   out_grad        CE: optional bf16 [M,N] (row stride ldc);
 *                   ROPE: required sin table bf16 [M,2N] (row stride ldc).
 *
 * Returns TGEMM_OK or a negative tgemm_status.
 */
TGEMM_API int tgemm_run(char transA, char transB, int64_t M, int64_t N, int64_t K,
              const void* A, int64_t lda, const void* B, int64_t ldb,
              void* C, int64_t ldc, int epilogue,
              const int32_t* labels, float* out_loss, void* out_grad,
              void* stream);

/*
 * tgemm_run without allocation, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments, results and errors as tgemm_run (the
 * same kernels), but every scratch buffer the call needs -- the split-K
 * partial products, the cross-entropy block partials, the matrix-vector
 * partials -- lives in one fixed device array of the library,
 * tgemm_noalloc_scratch_bytes() = 64 MiB per device, held from the first
 * use on a device until the process ends.  The call makes no hipMalloc,
 * hipFree or other allocating call; the caller still owns every input and
 * output.  A call whose scratch need exceeds the array returns
 * TGEMM_ERR_WORKSPACE_LIMIT before anything is enqueued (the 768x5120x13824
 * NT product needs 45 MiB: 3 K chunks; split-K needs 4*chunks*M*N bytes, cross-entropy
 * about 8*M*(N/128 + 1) bytes).
 *
 * Every call on a device shares that device's array, and the array keeps
 * the last call's contents (no kernel relies on them: each writes every
 * scratch value it reads).  Calls that may overlap on one device -- on two
 * streams, or from two threads -- race on the array and give wrong
 * results; serialise them (one stream, in order) or use tgemm_run.
 */
TGEMM_API int tgemm_run_noalloc(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                const void* A, int64_t lda, const void* B, int64_t ldb,
                                void* C, int64_t ldc, int epilogue,
                                const int32_t* labels, float* out_loss, void* out_grad,
                                void* stream);

/* Size in bytes of tgemm_run_noalloc's fixed scratch array. */
TGEMM_API int64_t tgemm_noalloc_scratch_bytes(void);

/*
 * Host-only argument check with the same rules as tgemm_run, without
 * touching the GPU.  Returns TGEMM_OK or the status tgemm_run would return.
 */
TGEMM_API int tgemm_validate(char transA, char transB, int64_t M, int64_t N, int64_t K,
                   const void* A, int64_t lda, const void* B, int64_t ldb,
                   const void* C, int64_t ldc, int epilogue,
                   const int32_t* labels, const float* out_loss,
                   const void* out_grad);

/*
 * GEMM on fp8 (e4m3fn) operands made on the fly from bf16 inputs.
 *
 * ("Improve the Inductor generated kernel for the pattern of output1 =
 * pointwise(input); output2 = transpose(output1)", the example: before a
 * float8 linear each input element is scaled, clamped to the largest
 * finite e4m3fn value and cast to e4m3fn, and the page's pattern also
 * writes a transposed copy of the fp8 tensor.  Here no transposed copy is
 * ever stored: the operands are read in their stored layouts.)
 *
 *   transA, transB, M, N, K, A, lda, B, ldb, C, ldc: as for tgemm_run with
 *                   a STORE epilogue; A and B are bf16 in any layout.
 *   epilogue        TGEMM_EPI_STORE_BF16 or TGEMM_EPI_STORE_F32 only.
 *   scales          device pointer to three fp32 values
 *                   {scale_a, scale_b, out_scale}, read by the kernel.
 *
 * Each element x of op(A) becomes q = e4m3fn(clamp(fp32(x) * scale_a,
 * -448, 448)): one fp32 multiply, the clamp (NaN stays NaN), then rounding
 * to nearest e4m3fn value with ties to even; likewise op(B) with scale_b.
 * C = out_scale * sum_k qA[m,k] * qB[k,n], products exact, fp32
 * accumulation, one fp32 multiply by out_scale, then the store epilogue
 * (bf16 with round-to-nearest-even, or fp32).  Pass out_scale =
 * 1 / (scale_a * scale_b) to undo both casts.
 *
 * Large products (at least two 256-row and two 256-column tiles, every
 * stored row 16-byte aligned with a multiple of 8 elements) cast each
 * operand once into a K-contiguous matrix of e4m3fn codes (one byte each,
 * zero-padded to whole tiles) in the library's per-stream workspace, and
 * multiply the codes on the fp8 matrix cores (v_mfma_f32_32x32x64_f8f6f4).
 * Other products cast each element as the GEMM loads it and multiply on
 * the bf16 matrix cores, which hold every e4m3fn value exactly.  Both
 * routes multiply the same e4m3fn values with fp32 accumulation; their
 * sums may differ in the last bits (the matrix cores group the k
 * differently), and both are exact where every partial sum is exactly
 * representable (e.g. integer-valued operands).  tgemm_set_fp8_cast_once(0)
 * forces the cast on load.  If the workspace for the codes cannot be
 * allocated, the product casts on load.
 *
 * Validation, errors, asynchrony and streams as for tgemm_run.  Returns
 * TGEMM_OK or a negative tgemm_status; an unsupported epilogue or a NULL
 * `scales` is TGEMM_ERR_INVALID_ARG.
 */
TGEMM_API int tgemm_run_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                  const void* A, int64_t lda, const void* B, int64_t ldb,
                  void* C, int64_t ldc, int epilogue, const float* scales,
                  void* stream);

/* Host-only argument check of tgemm_run_fp8 (no GPU access). */
TGEMM_API int tgemm_validate_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                  const void* A, int64_t lda, const void* B, int64_t ldb,
                  const void* C, int64_t ldc, int epilogue, const float* scales);

/*
 * Cross-entropy with the gradient left for the backward GEMMs to finish
 * ("Allow reductions in matmul epilogues", the edit note: the
 * softmax-minus-one-hot matrix is kept for the backward pass).
 *
 * As tgemm_run with TGEMM_EPI_CE and a gradient buffer (same arguments,
 * same loss, bit for bit), except that the pass that rescales the gradient
 * is not run.  Instead:
 *   out_e      bf16 [M, N] (row stride lde >= N) receives
 *              e = bf16(exp(y - m_b)), y the fp32 logit and m_b the maximum
 *              of y over the block of columns the GEMM's tile reduced (64 or
 *              128 columns);
 *   out_scale  fp32 [ceil(N/64) * M] receives, for every 64-column chunk c
 *              of every row m, s[c*M + m] = exp(m_b - lse[m]) of the block
 *              holding the chunk.
 * The gradient is then softmax - onehot = bf16(e * s - [n == labels[m]])
 * (one fused multiply-add, rounded once), which tgemm_run_ce_grad computes
 * as it loads e, and which equals bit for bit what the rescale pass of
 * tgemm_run writes.  K must be >= 2 (a K = 1 product takes the pointwise
 * path, which has no deferred form): TGEMM_ERR_UNSUPPORTED otherwise.
 * Validation, errors, asynchrony, streams and workspace as for tgemm_run.
 */
TGEMM_API int tgemm_run_ce_deferred(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                    const void* A, int64_t lda, const void* B, int64_t ldb,
                                    const int32_t* labels, float* out_loss, void* out_e,
                                    int64_t lde, float* out_scale, void* stream);

/*
 * A GEMM whose operand A is a cross-entropy gradient left by
 * tgemm_run_ce_deferred, finished as it is loaded:
 *   C = op(G) . op(B),  G[t][v] = bf16(e[t*lde + v] * scale[(v/64)*T + t]
 *                                      - [v == labels[t]])
 * with G a [T, V] matrix (T token rows, V vocabulary columns) stored as e:
 * transA 'N' reads it as op(A) = G (T = M, V = K; the gradient of the
 * hidden states, dH = G . W), 'T' as op(A) = G^T (T = K, V = M; the
 * gradient of the weight, dW = G^T . H).  B, transB, ldb, C, ldc as for
 * tgemm_run; epilogue TGEMM_EPI_STORE_BF16 or TGEMM_EPI_STORE_F32.  Every
 * shape runs on the matrix-core kernel (no pointwise, matrix-vector or
 * split-K route).  The result equals, bit for bit, tgemm_run on the
 * gradient the rescale pass writes.  Labels outside [0, V) subtract
 * nothing.  Validation, errors, asynchrony and streams as for tgemm_run; a
 * NULL scale or labels, or another epilogue, is TGEMM_ERR_INVALID_ARG.
 */
TGEMM_API int tgemm_run_ce_grad(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                const void* E, int64_t lde, const float* scale,
                                const int32_t* labels, const void* B, int64_t ldb, void* C,
                                int64_t ldc, int epilogue, void* stream);

/*
 * The RoPE region of "Schedule a small matmul op as a reduction (or
 * pointwise) op" as far as that page's %kernel_math listing goes, in one
 * launch (the page's closing remark: the section fused into a single
 * kernel, the K = 1 matmul included):
 *   - the cos / sin tables of the positions, exactly as tgemm_run with
 *     TGEMM_EPI_ROPE_COSSIN and K = 1: t = fp32(pos[p]) * inv_freq[i]
 *     (i < F = D/2), cos_out / sin_out[p, i] and [p, i + F] = bf16(cos t) /
 *     bf16(sin t) (the listing's T19 .. T26 and the second table output);
 *   - the query of the listing's first three steps: q [P, ldq] bf16, row p
 *     holding H heads of D values (head h at columns h*D .. h*D + D-1),
 *     viewed as [P, H, D] (T5), permuted to [H, P, D] (T6) and widened to
 *     fp32 (T34), written to q_out[(h*P + p)*D + d] (fp32, contiguous
 *     [H][P][D]).
 * The rotation that turns these into the region's rotated outputs is not
 * on the page and is not applied.
 *
 *   q, ldq        bf16 query rows, ldq >= H*D (elements).
 *   P, H, D       positions, heads, head width; P, H >= 1, D >= 2 even.
 *   pos, spos     int64 positions, element stride spos >= 1.
 *   inv_freq      fp32 [D/2], contiguous.
 *   cos_out, sin_out  bf16 [P, ldc], ldc >= D.
 *   q_out         fp32 [H*P*D].
 * All pointers are device pointers owned by the caller; outputs must not
 * alias inputs.  Validation, errors, asynchrony and streams as for
 * tgemm_run; no workspace.  Returns TGEMM_OK or a negative tgemm_status.
 */
TGEMM_API int tgemm_rope_region(const void* q, int64_t ldq, int64_t P, int64_t H, int64_t D,
                                const int64_t* pos, int64_t spos, const float* inv_freq,
                                void* cos_out, void* sin_out, int64_t ldc, float* q_out,
                                void* stream);

/* Host-only argument check of tgemm_rope_region (no GPU access). */
TGEMM_API int tgemm_validate_rope_region(const void* q, int64_t ldq, int64_t P, int64_t H,
                                         int64_t D, const int64_t* pos, int64_t spos,
                                         const float* inv_freq, const void* cos_out,
                                         const void* sin_out, int64_t ldc, const float* q_out);

/*
 * ---- The feed-forward block: gated products, 8-bit products, norms ------
 *
 * What a gated feed-forward block adds around its down projection, as it is
 * trained (bf16 operands, with the gradient) and as it is served (8-bit
 * integer operands).  Storage, layout flags, asynchrony, streams, threads
 * and errors as for tgemm_run.
 *
 * Workspace: a call that needs scratch memory takes it from the caller's
 * `workspace` (device memory, 16-byte aligned, workspace_bytes >= 0 bytes;
 * the call's ..._workspace_bytes function says how many it needs, 0 for
 * most; the buffer must not be used by anything else until the call's
 * kernels have run) and fails with TGEMM_ERR_WORKSPACE_LIMIT, before anything
 * is enqueued, if that is too small.  workspace_bytes = -1 (workspace is
 * then ignored) takes the library's buffer of the stream, as tgemm_run does,
 * except while the stream is being captured into a graph: then a call that
 * needs workspace fails with TGEMM_ERR_WORKSPACE_LIMIT, and the caller has to
 * bring its own, which lives and dies with the caller's graph.  The
 * ..._workspace_bytes functions return a negative tgemm_status for invalid
 * arguments; they look at the operands' addresses, strides and layouts, not
 * at their contents, and enqueue nothing.
 */

/* Activations of the gated products (fp32 arithmetic; 0 for g below about
 * -174.7 and -12.9). */
typedef enum {
  TGEMM_ACT_SILU = 0,     /* g / (1 + exp(-g))                                         */
  TGEMM_ACT_GELU_TANH = 1, /* g/2 * (1 + tanh(sqrt(2/pi) * (g + 0.044715 * g^3)))      */
  TGEMM_ACT_NONE = 2,     /* z: linear products only                                   */
  TGEMM_ACT_RELU = 3      /* max(z, 0), NaN stays: linear products only                */
} tgemm_activation;

/*
 * RMS norm of rows, with the residual's addition, to 8-bit codes with one
 * scale per row.  Per row of K elements:
 *   h     = bf16(fp32(x + residual)), written to `sum` (h = x without a
 *           residual)
 *   t     = h * weight, T = max |t|
 *   scale = T / (127 * sqrt(mean(h^2) + eps))                       fp32
 *   q     = 127 * t / T rounded to the nearest integer, ties to even
 * so scale * q is the normed row h * weight / sqrt(mean(h^2) + eps) in 255
 * levels (q in [-127, 127]).  The codes are the exact quotients' roundings:
 * the same row always gives the same codes.  A row with T = 0 gets scale 0
 * and codes 0; a row in which some t is NaN or infinite (in fp32) gets scale
 * NaN and codes 0.  Products t below fp32's normal range lose bits.
 *
 *   x, residual, sum  bf16 [M, K], row strides ldx, ldr, lds >= K (elements).
 *                     residual and sum are both given or both NULL; sum may
 *                     be x or residual itself (same address and stride).
 *   weight            bf16 [K].      eps  finite and >= 0.
 *   q                 int8 [M, K], row stride ldq >= K.
 *   scale             fp32 [M].
 * Rows may start at any element: no alignment is asked for.  No workspace.
 * M times ceil(K / 512) * 64 (at most 1024) below 2^32, else
 * TGEMM_ERR_UNSUPPORTED.
 */
TGEMM_API int tgemm_rms_norm_i8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                const void* weight, float eps, int64_t M, int64_t K, void* sum,
                                int64_t lds, int8_t* q, int64_t ldq, float* scale, void* stream);

/* Host-only argument check of tgemm_rms_norm_i8 (no GPU access). */
TGEMM_API int tgemm_validate_rms_norm_i8(const void* x, int64_t ldx, const void* residual,
                                         int64_t ldr, const void* weight, float eps, int64_t M,
                                         int64_t K, const void* sum, int64_t lds, const int8_t* q,
                                         int64_t ldq, const float* scale);

/*
 * Rows of x (bf16 [M, K]) to 8-bit codes with one scale per row: as above
 * with t = x and scale = T / 127.
 */
TGEMM_API int tgemm_quantize_i8(const void* x, int64_t ldx, int64_t M, int64_t K, int8_t* q,
                                int64_t ldq, float* scale, void* stream);

/* Host-only argument check of tgemm_quantize_i8 (no GPU access). */
TGEMM_API int tgemm_validate_quantize_i8(const void* x, int64_t ldx, int64_t M, int64_t K,
                                         const int8_t* q, int64_t ldq, const float* scale);

/*
 * Product of 8-bit integers with a scale for each row (token) of op(A) and
 * each column (channel) of op(B):
 *   C[m,n] = scale_a[m] * scale_b[n] * sum_k op(A)[m,k] * op(B)[k,n]
 * The sum is exact (int32; K <= 131071, else TGEMM_ERR_UNSUPPORTED); it is
 * converted to fp32 and multiplied by scale_a, then scale_b.
 *
 *   A, B      int8, in any layout (row strides lda, ldb in elements).
 *   scale_a   fp32 [M], scale_b fp32 [N].
 *   C         bf16 (TGEMM_EPI_STORE_BF16) or fp32 (TGEMM_EPI_STORE_F32).
 *
 * A 'N' and B 'T' with 16-byte aligned bases and lda, ldb and K multiples of
 * 16 are read in place; other operands are first copied, K-contiguous, into
 * the workspace.  Up to 64 rows of op(A) run on a kernel that streams B
 * once.
 */
TGEMM_API int tgemm_run_i8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                           const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                           const float* scale_a, const float* scale_b, void* C, int64_t ldc,
                           int epilogue, void* workspace, int64_t workspace_bytes, void* stream);
TGEMM_API int64_t tgemm_i8_workspace_bytes(char transA, char transB, int64_t M, int64_t N,
                                           int64_t K, const int8_t* A, int64_t lda,
                                           const int8_t* B, int64_t ldb);

/* Host-only argument check of tgemm_run_i8 (no GPU access). */
TGEMM_API int tgemm_validate_i8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                const float* scale_a, const float* scale_b, const void* C,
                                int64_t ldc, int epilogue);

/*
 * Gate and up projections, the activation and their product in one call:
 *   [g | u] = op(A) . op(B)   op(B) is [K, 2F]: columns 0 .. F-1 give g,
 *                             F .. 2F-1 give u (fp32 sums)
 *   H       = bf16(act(g) * u)                              [M, F]
 * g and u are not written unless GU is given: fp32 [M, 2F] (row stride ldgu
 * >= 2F), g in the first F columns and u in the last, for the backward call.
 *
 * A 'N' and B 'T' with 16-byte aligned bases and lda, ldb and K multiples of
 * 8 are read in place; other operands are first copied, K-contiguous, into
 * the workspace.  Few rows of op(A) run on a kernel that streams B once.
 */
TGEMM_API int tgemm_run_gated(char transA, char transB, int64_t M, int64_t F, int64_t K,
                              const void* A, int64_t lda, const void* B, int64_t ldb,
                              int activation, void* H, int64_t ldh, float* GU, int64_t ldgu,
                              void* workspace, int64_t workspace_bytes, void* stream);
TGEMM_API int64_t tgemm_gated_workspace_bytes(char transA, char transB, int64_t M, int64_t F,
                                              int64_t K, const void* A, int64_t lda,
                                              const void* B, int64_t ldb);

/* Host-only argument check of tgemm_run_gated (no GPU access). */
TGEMM_API int tgemm_validate_gated(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                   const void* A, int64_t lda, const void* B, int64_t ldb,
                                   int activation, const void* H, int64_t ldh, const float* GU,
                                   int64_t ldgu);

/*
 * The gated product from 8-bit operands: g and u as tgemm_run_i8 computes
 * them (scale_b has 2F entries), H = bf16(act(g) * u).
 */
TGEMM_API int tgemm_run_gated_i8(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                 const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                 const float* scale_a, const float* scale_b, int activation,
                                 void* H, int64_t ldh, void* workspace, int64_t workspace_bytes,
                                 void* stream);
TGEMM_API int64_t tgemm_gated_i8_workspace_bytes(char transA, char transB, int64_t M, int64_t F,
                                                 int64_t K, const int8_t* A, int64_t lda,
                                                 const int8_t* B, int64_t ldb);

/* Host-only argument check of tgemm_run_gated_i8 (no GPU access). */
TGEMM_API int tgemm_validate_gated_i8(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                      const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                      const float* scale_a, const float* scale_b, int activation,
                                      const void* H, int64_t ldh);

/*
 * Gradient of H = act(g) * u with respect to g and u:
 *   dGU[:, :F] = bf16(dH * u * act'(g)),  dGU[:, F:] = bf16(dH * act(g))
 * dH bf16 [M, F], dGU bf16 [M, 2F].  GU [M, 2F] as tgemm_run_gated left it
 * (gu_type TGEMM_EPI_STORE_F32), or rounded to bf16 since
 * (TGEMM_EPI_STORE_BF16: half the memory, and a rounding more in the
 * gradients).  No workspace.  M times F / 2048, rounded up, below 2^24, else
 * TGEMM_ERR_UNSUPPORTED.
 */
TGEMM_API int tgemm_gated_grad(int64_t M, int64_t F, const void* dH, int64_t lddh, const void* GU,
                               int64_t ldgu, int gu_type, int activation, void* dGU, int64_t lddgu,
                               void* stream);

/* Host-only argument check of tgemm_gated_grad (no GPU access). */
TGEMM_API int tgemm_validate_gated_grad(int64_t M, int64_t F, const void* dH, int64_t lddh,
                                        const void* GU, int64_t ldgu, int gu_type, int activation,
                                        const void* dGU, int64_t lddgu);

/*
 * The whole gradient of tgemm_run_gated: dGU = [dg | du] as tgemm_gated_grad
 * (kept in the workspace, bf16), then
 *   dA = dGU . op(B)^T    bf16 [M, K] (op(A)'s shape, row stride ldda >= K)
 *   dB = op(A)^T . dGU    in B's layout: [2F, K] for transB 'T' (row stride
 *                         lddb >= K), [K, 2F] for 'N' (lddb >= 2F); bf16
 *                         (epilogue TGEMM_EPI_STORE_BF16) or fp32
 *                         (TGEMM_EPI_STORE_F32)
 * with fp32 sums.  A, B as in the forward call, dH bf16 [M, F], GU and gu_type
 * as for tgemm_gated_grad.  Both products run in one launch.  Workspace: dGU
 * (about 4 * M * F bytes), copies of operands other than A 'N' and B 'T' with
 * 16-byte aligned bases and lda, ldb multiples of 8 (and of A for transB
 * 'N'), and for few tiles fp32 partial products.  K and 2F up to about 2^23,
 * M about 2^24 (past 2048 columns of F less: a workgroup per row and 2048
 * columns), else TGEMM_ERR_UNSUPPORTED.
 */
TGEMM_API int tgemm_run_gated_backward(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                       const void* A, int64_t lda, const void* B, int64_t ldb,
                                       const void* dH, int64_t lddh, const void* GU, int64_t ldgu,
                                       int gu_type, int activation, void* dA, int64_t ldda, void* dB,
                                       int64_t lddb, int epilogue, void* workspace,
                                       int64_t workspace_bytes, void* stream);
TGEMM_API int64_t tgemm_gated_backward_workspace_bytes(char transA, char transB, int64_t M,
                                                       int64_t F, int64_t K, const void* A,
                                                       int64_t lda, const void* B, int64_t ldb);

/* Host-only argument check of tgemm_run_gated_backward (no GPU access). */
TGEMM_API int tgemm_validate_gated_backward(char transA, char transB, int64_t M, int64_t F,
                                            int64_t K, const void* A, int64_t lda, const void* B,
                                            int64_t ldb, const void* dH, int64_t lddh,
                                            const void* GU, int64_t ldgu, int gu_type,
                                            int activation, const void* dA, int64_t ldda, const void* dB,
                                            int64_t lddb, int epilogue);

/*
 * ---- Linear layers: product, bias, activation, residual -------------------
 *
 *   z = op(A) . op(B) + bias          bf16 operands, fp32 sums
 *   Y = residual + act(z)             rounded once, to Y's type
 *
 *   A, B        bf16, in any layout.
 *   bias        bf16 [N], or NULL.
 *   activation  a tgemm_activation.
 *   Y           [M, N], ldy >= N: bf16 (epilogue TGEMM_EPI_STORE_BF16) or fp32
 *               (TGEMM_EPI_STORE_F32).
 *   residual    [M, N] of Y's type, ldr >= N, or NULL.  It may be Y itself
 *               (same address and stride).
 *   Z           [M, N], ldz >= N, or NULL: receives z for the backward call,
 *               fp32 or bf16 (z_type, an epilogue's name as for Y; ignored
 *               without Z).
 *
 * Operands, workspace and errors as for tgemm_run_gated.
 */
TGEMM_API int tgemm_run_linear(char transA, char transB, int64_t M, int64_t N, int64_t K,
                               const void* A, int64_t lda, const void* B, int64_t ldb,
                               const void* bias, int activation, const void* residual, int64_t ldr,
                               void* Y, int64_t ldy, int epilogue, void* Z, int64_t ldz,
                               int z_type, void* workspace, int64_t workspace_bytes, void* stream);
TGEMM_API int64_t tgemm_linear_workspace_bytes(char transA, char transB, int64_t M, int64_t N,
                                               int64_t K, const void* A, int64_t lda,
                                               const void* B, int64_t ldb);

/* Host-only argument check of tgemm_run_linear (no GPU access). */
TGEMM_API int tgemm_validate_linear(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                    const void* A, int64_t lda, const void* B, int64_t ldb,
                                    const void* bias, int activation, const void* residual,
                                    int64_t ldr, const void* Y, int64_t ldy, int epilogue,
                                    const void* Z, int64_t ldz, int z_type);

/*
 * The gradient of tgemm_run_linear for the gradient dY (bf16 [M, N]) of Y:
 *   dz    = dY * act'(z)
 *   dA    = dz . op(B)^T      bf16 [M, K] (op(A)'s shape, row stride ldda >= K)
 *   dB    = op(A)^T . dz      in B's layout, bf16 or fp32 (epilogue), as in
 *                             tgemm_run_gated_backward
 *   dbias = sum_m dz[m, :]    fp32 [N], or NULL
 * (the residual's gradient is dY).  dz is rounded to bf16 once for the
 * products; dbias is the sum before that rounding, in fp32.  A, B as in the
 * forward call; Z and z_type as it left Z (or rounded to bf16 since), not read
 * for TGEMM_ACT_NONE.  relu's derivative is 0 at z = 0.  Workspace: dz (2 * M
 * * N bytes, padded), the bias's partial sums (up to 4 bytes for every 8
 * elements of it), and copies and partial products as in
 * tgemm_run_gated_backward, whose size limits hold with N for 2F.
 */
TGEMM_API int tgemm_run_linear_backward(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                        const void* A, int64_t lda, const void* B, int64_t ldb,
                                        const void* dY, int64_t lddy, const void* Z, int64_t ldz,
                                        int z_type, int activation, void* dA, int64_t ldda,
                                        void* dB, int64_t lddb, int epilogue, float* dbias,
                                        void* workspace, int64_t workspace_bytes, void* stream);
TGEMM_API int64_t tgemm_linear_backward_workspace_bytes(char transA, char transB, int64_t M,
                                                        int64_t N, int64_t K, const void* A,
                                                        int64_t lda, const void* B, int64_t ldb);

/* Host-only argument check of tgemm_run_linear_backward (no GPU access). */
TGEMM_API int tgemm_validate_linear_backward(char transA, char transB, int64_t M, int64_t N,
                                             int64_t K, const void* A, int64_t lda, const void* B,
                                             int64_t ldb, const void* dY, int64_t lddy,
                                             const void* Z, int64_t ldz, int z_type,
                                             int activation, const void* dA, int64_t ldda,
                                             const void* dB, int64_t lddb, int epilogue,
                                             const float* dbias);

/*
 * ---- The norms before and after a block -----------------------------------
 *
 * Between two blocks of a residual stream: the output y of one, normed, gated
 * and scaled, is added to the stream, whose norm is the input of the next.
 * Per row of K elements:
 *   p = y * ry * post_weight,  ry = 1 / sqrt(mean(y^2) + eps)    (p = y
 *                              without a post_weight)
 *   s = residual + scale * gate * p                              (gate 1
 *                              without one)
 *   n = s * rs * weight,       rs = 1 / sqrt(mean(s^2) + eps)
 * in fp32 (the means in 64 bits); s is rounded for its store only.
 *
 *   y, n             bf16 [M, K], row strides ldy, ldn >= K.
 *   residual, sum    [M, K] of stream_type (TGEMM_EPI_STORE_BF16 or
 *                    TGEMM_EPI_STORE_F32); sum receives s and may be residual
 *                    itself (same address and stride), where no backward call
 *                    follows.
 *   weight           bf16 [K]; post_weight bf16 [K] or NULL.
 *   gate             bf16 [gates, K], row stride ldgate >= K, or NULL.  gates
 *                    divides M; each row of it serves M / gates consecutive
 *                    rows: 1 for a learned gate per channel, the number of
 *                    sequences for one per sequence, M for one per token.
 *   scale, eps       finite; eps >= 0.  With eps 0 a row whose rms is below 2^-128
 *                    gives infinities or NaN, as one of zeros does.
 *   rstd             fp32 [M] of rs, then with a post_weight [M] of ry, for the
 *                    backward call; or NULL.
 * K up to 16384, M times the threads of a row below 2^32, else
 * TGEMM_ERR_UNSUPPORTED.  Rows may start at any element.  No workspace.
 */
TGEMM_API int tgemm_block_norm(const void* y, int64_t ldy, const void* residual, int64_t ldr,
                               int stream_type, const void* post_weight, const void* gate,
                               int64_t ldgate, int64_t gates, float scale, const void* weight,
                               float eps, int64_t M, int64_t K, void* sum, int64_t lds, void* n,
                               int64_t ldn, float* rstd, void* stream);

/* Host-only argument check of tgemm_block_norm (no GPU access). */
TGEMM_API int tgemm_validate_block_norm(const void* y, int64_t ldy, const void* residual,
                                        int64_t ldr, int stream_type, const void* post_weight,
                                        const void* gate, int64_t ldgate, int64_t gates,
                                        float scale, const void* weight, float eps, int64_t M,
                                        int64_t K, const void* sum, int64_t lds, const void* n,
                                        int64_t ldn, const float* rstd);

/*
 * Its gradient, for the gradients dn (bf16 [M, K]) of n and ds (stream_type
 * [M, K], or NULL) of s:
 *   dresidual  stream_type [M, K]; may be ds itself (same address and stride)
 *   dy         bf16 [M, K]; may be dn itself
 *   dweight    fp32 [K]
 *   dpost      fp32 [K], with a post_weight
 *   dgate      fp32 [gates, K], contiguous, with a gate
 * The other arguments as in the forward call; rstd as it left them.  s is
 * computed again from y and residual, in fp32; rows of any size that the
 * forward takes keep their gradient.  The sums over rows are fp32,
 * in an order that depends on the sizes alone.  K up to 16384, else
 * TGEMM_ERR_UNSUPPORTED.  Workspace (as for the feed-forward calls): partial
 * sums of at most 512 groups of rows, at most 16 * 512 * K bytes.
 */
TGEMM_API int tgemm_block_norm_backward(const void* dn, int64_t lddn, const void* ds, int64_t ldds,
                                        const void* y, int64_t ldy, const void* residual,
                                        int64_t ldr, int stream_type, const void* post_weight,
                                        const void* gate, int64_t ldgate, int64_t gates,
                                        float scale, const void* weight, const float* rstd,
                                        int64_t M, int64_t K, void* dresidual, int64_t lddr,
                                        void* dy, int64_t lddy, float* dweight, float* dpost,
                                        float* dgate, void* workspace, int64_t workspace_bytes,
                                        void* stream);
/* post: 1 with a post_weight, else 0; gates: 0 without a gate. */
TGEMM_API int64_t tgemm_block_norm_backward_workspace_bytes(int64_t M, int64_t K, int post,
                                                            int64_t gates);

/* Host-only argument check of tgemm_block_norm_backward (no GPU access). */
TGEMM_API int tgemm_validate_block_norm_backward(
    const void* dn, int64_t lddn, const void* ds, int64_t ldds, const void* y, int64_t ldy,
    const void* residual, int64_t ldr, int stream_type, const void* post_weight, const void* gate,
    int64_t ldgate, int64_t gates, float scale, const void* weight, const float* rstd, int64_t M,
    int64_t K, const void* dresidual, int64_t lddr, const void* dy, int64_t lddy,
    const float* dweight, const float* dpost, const float* dgate);

/*
 * ---- Mixture-of-experts layers for few tokens -----------------------------
 *
 *   Y[m] = sum_j weights[m, j] * H[m, j] . W2[ids[m, j]]^T          bf16 [M, K]
 *   H[m, j] = act(g) * u,  [g | u] = X[m] . W1[ids[m, j]]^T
 * with fp32 sums, and H in 16 bits of mantissa (the sum of two bf16 values):
 * `top` of E gated experts for each token.  With a router the
 * call chooses them: the top largest of the logits X[m] . router^T (sums in 64
 * bits, so that the choice depends on no order of summation; the lowest index
 * first among equals; NaN counts as largest), with the weights
 *   weights[m, j] = scale * exp(l_j - l_0) / sum exp(l_i - l_0),
 * the sum over the chosen (renormalize != 0) or over all experts; ids and
 * weights are then outputs.  Without a router (NULL) they are inputs: an id
 * outside 0 .. E-1 adds nothing (its expert lives elsewhere), one that a token
 * lists twice counts twice, and top may pass E.
 *
 *   X, Y        bf16 [M, K], row strides ldx, ldy >= K.
 *   router      [E, K] bf16 or fp32 (router_type, an epilogue's name as
 *               elsewhere), row stride ldr >= K.
 *   ids         int32 [M, top], weights fp32 [M, top], contiguous.
 *   W1          bf16 [E, 2F, K]: per expert F gate rows, then F up rows, row
 *               stride ldw1 >= K, experts sw1 elements apart.
 *   W2          bf16 [E, K, F], row stride ldw2 >= F, experts sw2 apart.
 *   activation  TGEMM_ACT_SILU or TGEMM_ACT_GELU_TANH.
 * E up to 1024, top up to 16, rows of X, W1 and W2 less than 2^22 elements
 * apart, else TGEMM_ERR_UNSUPPORTED.  The layer is made for few tokens: 64 rows
 * run at a time, and each pass reads the experts it hits.  With X, W1 and W2 all
 * on 16-byte boundaries (bases and strides; K and F multiples of 8) the weights
 * are read at full rate, else in place too, more slowly.  Workspace as for the feed-forward calls;
 * nearly every call needs some.
 */
TGEMM_API int tgemm_run_moe(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top, const void* X,
                            int64_t ldx, const void* router, int64_t ldr, int router_type,
                            int renormalize, float scale, int32_t* ids, float* weights,
                            const void* W1, int64_t ldw1, int64_t sw1, const void* W2,
                            int64_t ldw2, int64_t sw2, int activation, void* Y, int64_t ldy,
                            void* workspace, int64_t workspace_bytes, void* stream);
/* routed: 1 with a router, else 0. */
TGEMM_API int64_t tgemm_moe_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E,
                                            int64_t top, int routed);

/* Host-only argument check of tgemm_run_moe (no GPU access). */
TGEMM_API int tgemm_validate_moe(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top,
                                 const void* X, int64_t ldx, const void* router, int64_t ldr,
                                 int router_type, int renormalize, float scale,
                                 const int32_t* ids, const float* weights, const void* W1,
                                 int64_t ldw1, int64_t sw1, const void* W2, int64_t ldw2,
                                 int64_t sw2, int activation, const void* Y, int64_t ldy);

/* Human-readable name of a status code (static string, never NULL). */
TGEMM_API const char* tgemm_status_string(int status);

/*
 * Tuning / testing knob: force the GEMM tile configuration for subsequent
 * calls from this process.  0 = automatic (default); 1 = 256x256 tiles;
 * 2 = 128x128 tiles; 3 = 192x256 tiles for NT products with a store
 * epilogue (256x256 for any other call).  Returns the previous value, or
 * TGEMM_ERR_INVALID_ARG for an unknown value.
 * Not thread-safe with concurrent tgemm_run calls.
 */
TGEMM_API int tgemm_set_tile_config(int config);

/*
 * Tuning / testing knob: force the number of K chunks a GEMM with a store
 * epilogue is split into (each chunk is a separate workgroup writing an
 * fp32 partial product; a second kernel adds the partials in ascending
 * chunk order, so results do not depend on timing).  Ignored for the CE
 * epilogue.  0 = automatic (default), 1 = never
 * split.  Returns the previous value, or TGEMM_ERR_INVALID_ARG outside
 * 0..64.  Not thread-safe with concurrent tgemm_run calls.
 */
TGEMM_API int tgemm_set_split_k(int split);

/*
 * Tuning / testing knob for tgemm_run_fp8: 1 (default) lets large products
 * (at least two 256-row and two 256-column tiles, 16-byte rows) cast each
 * operand once, in a pass of its own, into K-contiguous e4m3fn codes in the
 * library's per-stream workspace and multiply them on the fp8 matrix
 * cores; 0 always casts on load (bf16 matrix cores).  Both routes multiply
 * the same e4m3fn values; their fp32 sums may differ in the last bits.
 * Returns the previous value,
 * or TGEMM_ERR_INVALID_ARG for anything but 0 or 1.  Not thread-safe with
 * concurrent tgemm_run_fp8 calls.
 */
TGEMM_API int tgemm_set_fp8_cast_once(int enable);

/*
 * Measurement aid, beside the GEMM path: the shader clock the device runs
 * at.  Enqueues on `stream` one wave that polls the device's constant-rate
 * counter until it has advanced by `ticks` (1 <= ticks <= 10^7; at the
 * usual 100 MHz rate, 2000 ticks = 20 us), then writes three uint64 values
 * to out_ticks (device memory, 8-byte aligned, owned by the caller): the
 * shader-clock cycles that elapsed, the constant-rate ticks that elapsed,
 * and the constant rate in Hz.  The shader clock over the wait is
 * out[0] * out[2] / out[1].  Enqueued right after a timed region it reads
 * the clock that region ended at.  Asynchronous like tgemm_run.  Returns
 * TGEMM_OK, TGEMM_ERR_INVALID_ARG (ticks out of range, NULL or misaligned
 * out_ticks; checked before any device call) or TGEMM_ERR_HIP.
 */
TGEMM_API int tgemm_clock_probe(int64_t ticks, uint64_t* out_ticks, void* stream);

/*
 * Matrix-core ceiling (a measurement aid, not part of the GEMM path):
 * enqueue `blocks` workgroups of 4 waves (one workgroup per compute unit,
 * one wave per SIMD) that each issue only MFMAs on operands held in
 * registers: `iters` iterations of 16 MFMAs into 16 independent 32x32
 * accumulator blocks.  kind 0: v_mfma_f32_32x32x16_bf16 on finite bf16
 * values, 524288 flop per wave and iteration; kind 1: the 32x32x64 MFMA on
 * fp8 e4m3fn codes (never NaN), 2097152 flop.  The work is blocks * 4 *
 * iters times that; timing it on `stream` gives the matrix-core rate
 * without loads, LDS or barriers at the clock the chip holds under it.
 * `out` (device, float[blocks * 4], 4-byte aligned, caller-owned) receives
 * element 0 of block 0 of each wave, so the work is kept (iters = 2 gives
 * twice the values of iters = 1 up to the fp32 roundings of the
 * accumulation).  Returns TGEMM_OK, TGEMM_ERR_INVALID_ARG (kind not 0 or
 * 1, iters outside [1, 1e8], blocks outside [1, 65536], NULL or misaligned
 * out; checked before any device call) or TGEMM_ERR_HIP.
 */
TGEMM_API int tgemm_mfma_ceiling(int kind, int64_t iters, int blocks, float* out, void* stream);

/*
 * Free the cached workspace buffer of (current device, `stream`) in stream
 * order (hipFreeAsync on `stream`); the next tgemm_run on that stream
 * allocates a new one.  Work already enqueued keeps a valid buffer.  A
 * stream that has none is a no-op.  Must not race with tgemm_run calls on
 * the same stream from other threads (it waits for a call holding the entry
 * to finish enqueueing).  Returns TGEMM_OK or TGEMM_ERR_HIP.
 */
TGEMM_API int tgemm_release_workspace(void* stream);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
TGEMM_API int tgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_H */
