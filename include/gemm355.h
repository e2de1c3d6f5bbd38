/*
 * gemm355 -- dense GEMM for AMD Instinct MI355X (gfx950), C ABI.
 *
 *   C = act( alpha * (scale_a[m] * scale_b[n]) * sum_k A[m,k] B[k,n] + beta * C + bias[n] )
 *
 * The operation is the general matrix multiply C = alpha*A*B + beta*C of the
 * first DeepGEMM page (sec. 1.1: A is MxK, B is KxN, C is MxN), with 16-bit
 * inputs accumulated in FP32 (same page, sec. 3.1), and the epilogue fused
 * before the store: bias, then activation, then the output cast (same page,
 * sec. 6.1). The FP8 entry point takes E4M3 inputs with one FP32 scale per
 * row of A (per token) and one per column of B (per channel), applied after
 * accumulation and before the store (DeepGEMM: FP8 precision Tensor Core GEMM
 * optimisation, sec. 1.2 and 3.2). Like that page's interface (sec. 5.1) the
 * calls take device pointers, sizes, a scale description, an optional
 * workspace with a size query, and a stream.
 *
 * Conventions common to every entry point
 * ---------------------------------------
 * - All matrix, vector and workspace pointers are DEVICE pointers owned by the
 *   caller. The library never allocates, frees or synchronises, and apart
 *   from the scratch array of gemm_bf16_noalloc keeps no mutable global
 *   state: the other calls are reentrant and may run on any stream.
 * - Operand layouts (per operand, gemm_layout):
 *     A ROW: a(m,k) = A[m*lda + k], lda >= K      A COL: a(m,k) = A[k*lda + m], lda >= M
 *     B ROW: b(k,n) = B[k*ldb + n], ldb >= N      B COL: b(k,n) = B[n*ldb + k], ldb >= K
 *   "K-major" means A ROW and B COL. C is always row-major: C[m*ldc + n],
 *   ldc >= N. C is read (when beta != 0) and written with dtype c_dtype.
 * - Element types: BF16 (1-8-7, stored as uint16), OCP FP8 E4M3FN (1-4-3,
 *   bias 7, max 448, stored as uint8), FP32. bias is BF16[N] (NULL for none).
 *   scale_a is FP32[M] and scale_b FP32[N], contiguous (stride 1).
 * - Rounding: FP32 accumulation; epilogue arithmetic in FP32; the BF16 output
 *   cast rounds to nearest even.
 * - Activations: ReLU max(z,0); GELU_ERF z*Phi(z) = 0.5 z (1 + erf(z/sqrt 2));
 *   GELU_TANH 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))). Both GELUs are
 *   evaluated in forms without cancellation, so they keep their relative
 *   accuracy for large negative z: within 2^-19 relative (+1 ulp) of the exact
 *   value for FP32 output, within one BF16 ulp for BF16 output.
 * - Quick returns: M == 0 or N == 0 returns GEMM_OK and launches nothing.
 *   K == 0 gives C = act(beta*C + bias). beta == 0 means C is not read (NaN in
 *   C is ignored).
 * - Errors: every argument check happens before anything is enqueued; on a
 *   status other than GEMM_OK and GEMM_ERR_HIP nothing was launched and no
 *   memory was touched. GEMM_ERR_HIP means the HIP runtime rejected one of the
 *   call's launches; a call of two launches (a split-K GEMM and its
 *   reduction) whose second launch fails has already enqueued the first, which
 *   writes only the workspace. Before launching, the call consumes any HIP
 *   error that an earlier call on the same thread left pending (hipGetLastError),
 *   so GEMM_ERR_HIP never reports someone else's error. Faults inside a kernel
 *   surface at the caller's next synchronisation. Nothing is printed and
 *   nothing aborts.
 * - Aliasing: C must not overlap A, B, bias, the scales or the workspace.
 * - Asynchrony: work is enqueued on `stream` (a hipStream_t; NULL = the null
 *   stream) and the call returns without waiting.
 * - Determinism: for a given (shape, layouts, dtype) the result is bitwise
 *   reproducible run to run (the split-K reduction sums partials in a fixed
 *   order; no floating-point atomics).
 */
#ifndef GEMM355_H
#define GEMM355_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GEMM_OK = 0,
  GEMM_ERR_NULL_POINTER = 1,       /* a required pointer is NULL */
  GEMM_ERR_BAD_DIM = 2,            /* M, N or K negative, or too large for 32-bit tile indexing */
  GEMM_ERR_BAD_LD = 3,             /* a leading dimension is smaller than its operand's row extent */
  GEMM_ERR_BAD_ENUM = 4,           /* unknown layout, output dtype or activation */
  GEMM_ERR_UNSUPPORTED = 5,        /* a valid combination this library does not implement */
  GEMM_ERR_WORKSPACE_TOO_SMALL = 6,/* workspace_bytes < gemm_workspace_size(...) */
  GEMM_ERR_HIP = 7                 /* the HIP runtime rejected the launch */
} gemm_status;

typedef enum { GEMM_ROW_MAJOR = 0, GEMM_COL_MAJOR = 1 } gemm_layout;
typedef enum { GEMM_OUT_F32 = 0, GEMM_OUT_BF16 = 1 } gemm_out_dtype;
typedef enum {
  GEMM_ACT_NONE = 0,
  GEMM_ACT_RELU = 1,
  GEMM_ACT_GELU_ERF = 2,
  GEMM_ACT_GELU_TANH = 3
} gemm_act;

/*
 * BF16 x BF16 -> FP32 accumulate -> epilogue -> FP32 or BF16 C.
 * A: BF16, logical MxK, layout_a / lda as above. B: BF16, logical KxN.
 * All four layout combinations are accepted.
 * workspace: device scratch of at least gemm_workspace_size(M, N, K, 0) bytes
 * (may be NULL when that size is 0). Its contents on entry do not matter.
 */
gemm_status gemm_bf16(int64_t M, int64_t N, int64_t K, float alpha,
                      const void* A, int64_t lda, gemm_layout layout_a,
                      const void* B, int64_t ldb, gemm_layout layout_b,
                      float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                      const void* bias, gemm_act act,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * gemm_bf16 for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same operation, arguments and kernels, without a workspace argument. Split-K
 * partials go to a scratch array of 32 MiB that the library holds in every
 * GPU's memory from the module load until the process ends; the call
 * allocates and frees nothing. A shape whose plan needs more workspace than
 * that returns GEMM_ERR_WORKSPACE_TOO_SMALL (gemm_workspace_size(M, N, K, 0)
 * tells in advance) before anything is launched. The scratch of the calling
 * thread's current device is used, so that device must be the one the
 * stream and pointers belong to. All calls on one GPU share its array: calls
 * that overlap in time (on different streams, or from several threads) race
 * and give undefined results; calls ordered on one stream are safe. The first
 * call on each device looks up the array's device address
 * (hipGetSymbolAddress); a failure there returns GEMM_ERR_HIP.
 */
gemm_status gemm_bf16_noalloc(int64_t M, int64_t N, int64_t K, float alpha,
                              const void* A, int64_t lda, gemm_layout layout_a,
                              const void* B, int64_t ldb, gemm_layout layout_b,
                              float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                              const void* bias, gemm_act act, void* stream);

/*
 * OCP FP8 E4M3 x E4M3 -> FP32 accumulate -> x scale_a[m]*scale_b[n] -> epilogue.
 * A must be ROW (K-major, per-token rows) and B COL (K-major, per-channel
 * rows); other layouts return GEMM_ERR_UNSUPPORTED. scale_a (FP32[M]) and
 * scale_b (FP32[N]) are required. Codes 0x7F/0xFF (NaN) give undefined results.
 * workspace: at least gemm_workspace_size(M, N, K, 1) bytes.
 */
gemm_status gemm_fp8_scaled(int64_t M, int64_t N, int64_t K, float alpha,
                            const void* A, int64_t lda, gemm_layout layout_a,
                            const void* B, int64_t ldb, gemm_layout layout_b,
                            const float* scale_a, const float* scale_b,
                            float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                            const void* bias, gemm_act act,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * MX FP8 GEMM: E4M3 x E4M3 with one power-of-two (E8M0) scale per 32
 * consecutive K elements of each row of A and of each column of B, i.e. the
 * per-group scaling the FP8 DeepGEMM page (sec. 3.2) names next to the
 * per-token x per-channel form, in the block layout of the OCP
 * Microscaling (MX) formats, which gfx950's scaled MFMA applies in hardware:
 *
 *   C = act( alpha * sum_k a(m,k) 2^(SA[m][k/32]-127) * b(k,n) 2^(SB[n][k/32]-127)
 *            + beta * C + bias[n] )
 *
 * A: E4M3 codes, ROW (K-major), lda >= K. B: E4M3 codes, COL (K-major, N rows
 * of ldb), ldb >= K. Other layouts: GEMM_ERR_UNSUPPORTED.
 * scale_a: E8M0 codes (uint8), M rows of ldsa bytes; byte k/32 of row m
 * scales a(m, k). scale_b: N rows of ldsb bytes; byte k/32 of row n scales
 * b(k, n). Code c means 2^(c-127); code 255 (NaN) gives undefined results.
 * ldsa, ldsb: >= ceil(K/32), multiples of 4, >= 4; the arrays must span
 * M * ldsa and N * ldsb bytes, 4-byte aligned. Bytes past ceil(K/32) in a
 * row are never used.
 * A, B: any byte alignment and any K; the path reads its operands by DMA
 * only, with 32-bit offsets, so an operand spanning 2^31 bytes or more
 * ((rows - 1) * ld + K) gives GEMM_ERR_UNSUPPORTED.
 * There are no FP32 per-token / per-channel scales on this call. Epilogue,
 * C, bias, act, beta, workspace (size: gemm_workspace_size(M, N, K, 1)) and
 * stream as for gemm_fp8_scaled. Errors as for gemm_fp8_scaled, plus
 * GEMM_ERR_BAD_LD for ldsa / ldsb, GEMM_ERR_NULL_POINTER for NULL scales when
 * K > 0, GEMM_ERR_BAD_DIM when (M + 256) * ldsa or (N + 256) * ldsb reaches 2^31.
 */
gemm_status gemm_mxfp8(int64_t M, int64_t N, int64_t K, float alpha,
                       const void* A, int64_t lda, gemm_layout layout_a,
                       const void* B, int64_t ldb, gemm_layout layout_b,
                       const void* scale_a, int64_t ldsa, const void* scale_b, int64_t ldsb,
                       float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                       const void* bias, gemm_act act,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Element type of a quantised output (gemm_*_quant). */
typedef enum { GEMM_QOUT_INT8 = 0, GEMM_QOUT_E4M3 = 1 } gemm_qout_dtype;

/*
 * GEMM with a quantising epilogue: the FP32 epilogue value is quantised per
 * token (row) and written as one byte per element, so the next layer reads a
 * quarter of the FP32 bytes and no separate quantisation pass over C is
 * needed (first DeepGEMM page, sec. 6.2: the quantisation
 * round(x * scale + zero_point) applied to each output fragment inside the
 * epilogue, with one scale per row looked up by the row index). For output
 * element (m, n):
 *
 *   z = alpha * (scale_a[m] * scale_b[n]) * sum_k a(m,k) b(k,n) + bias[n]
 *       (scale_a, scale_b only in gemm_fp8_scaled_quant)
 *   y = act(z)                                     (FP32, as in gemm_bf16)
 *   GEMM_QOUT_INT8: v = fp32(y * out_scale[m] + zp[m]) (fused multiply-add,
 *                   one rounding; zp = out_zero[m], or 0 when out_zero is NULL)
 *                   Q[m*ldq+n] = int8 of round-to-nearest-even(v), saturated
 *                   to [-128, 127]
 *   GEMM_QOUT_E4M3: w = fp32(y * out_scale[m])
 *                   Q[m*ldq+n] = OCP E4M3FN code of w, round to nearest even,
 *                   saturating at +-448 (out_zero must be NULL)
 *
 * out_scale multiplies (it is the inverse of the dequantisation step); the
 * next layer recovers y ~ (q - zp) / out_scale. There is no beta and no C_in:
 * Q is only written. A, B, layouts, bias, act, scale_a / scale_b, workspace
 * and stream are as in gemm_bf16 / gemm_fp8_scaled (same layout rules, same
 * workspace size query with is_fp8 = 0 / 1).
 * Q: device, M x N bytes, row-major, ldq >= N (int8 or E4M3 codes).
 * out_scale: device FP32[M], finite; out_zero: device INT32[M] with values of
 * magnitude below 2^24, or NULL. NaN or infinite y give undefined codes.
 * Errors (before anything is enqueued): GEMM_ERR_BAD_ENUM (q_dtype, layout
 * or act), GEMM_ERR_UNSUPPORTED (out_zero given with GEMM_QOUT_E4M3, or a
 * layout the dtype does not support), GEMM_ERR_NULL_POINTER (out_scale, Q,
 * A / B when K > 0, the FP8 scales), and the other codes as for the plain calls.
 */
gemm_status gemm_bf16_quant(int64_t M, int64_t N, int64_t K, float alpha,
                            const void* A, int64_t lda, gemm_layout layout_a,
                            const void* B, int64_t ldb, gemm_layout layout_b,
                            const void* bias, gemm_act act,
                            const float* out_scale, const int32_t* out_zero,
                            void* Q, int64_t ldq, gemm_qout_dtype q_dtype,
                            void* workspace, size_t workspace_bytes, void* stream);

gemm_status gemm_fp8_scaled_quant(int64_t M, int64_t N, int64_t K, float alpha,
                                  const void* A, int64_t lda, gemm_layout layout_a,
                                  const void* B, int64_t ldb, gemm_layout layout_b,
                                  const float* scale_a, const float* scale_b,
                                  const void* bias, gemm_act act,
                                  const float* out_scale, const int32_t* out_zero,
                                  void* Q, int64_t ldq, gemm_qout_dtype q_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Per-token FP8 quantisation of BF16 activations, producing the A operand and
 * scale_a of gemm_fp8_scaled (the per-token scaling of DeepGEMM: FP8 precision
 * Tensor Core GEMM optimisation, sec. 1.2, done in one pass per row instead of
 * separate scale and cast kernels). For each row m of X:
 *   scale[m]   = fp32(max_k |x(m,k)| / 448), or 1 if the row is all zero
 *   Q[m*ldq+k] = OCP E4M3FN code of x(m,k) / scale[m] (IEEE float32 division,
 *                round to nearest even, saturating at +-448)
 * X: BF16, M x K row-major, ldx >= K (device). Q: uint8, M x K row-major,
 * ldq >= K (device). scale: FP32[M] (device). Columns K..ld-1 are neither read
 * nor written. K == 0 writes scale = 1 for every row. NaN or infinite inputs
 * give undefined codes and scales. Errors: GEMM_ERR_BAD_DIM (M or K negative
 * or above 2^30), GEMM_ERR_BAD_LD, GEMM_ERR_NULL_POINTER (scale, or X / Q when
 * K > 0), GEMM_ERR_HIP; all checks run before anything is enqueued.
 */
gemm_status gemm_quantize_fp8_rows(int64_t M, int64_t K, const void* X, int64_t ldx,
                                   void* Q, int64_t ldq, float* scale, void* stream);

/*
 * INT8 x INT8 product with one FP32 scale per row of A (token) and per column
 * of B (channel), and an optional zero point per row of A:
 *
 *   C = act( alpha * (scale_a[m] * scale_b[n]) * S(m,n) + beta * C + bias[n] )
 *   S(m,n) = sum_k (a(m,k) - zero_a[m]) b(k,n) = sum_k a b - zero_a[m] * sum_b[n]
 *
 * The sum over k is an exact INT32 sum whatever the split of K, and
 * zero_a[m] * sum_b[n] is taken off exactly before the first rounding; the
 * epilogue is FP32, as in the other calls. It reads what gemm_*_quant with
 * GEMM_QOUT_INT8 writes: scale_a[m] = 1 / out_scale[m], zero_a = out_zero.
 * A: INT8, ROW (K-major), lda >= K. B: INT8, COL (K-major), ldb >= K; other
 * layouts return GEMM_ERR_UNSUPPORTED (gemm_pack_b with elem_bytes 1 reorders
 * a weight). Any byte alignment. K at most 131071 (the INT32 sum cannot
 * overflow), else GEMM_ERR_UNSUPPORTED.
 * scale_a FP32[M], scale_b FP32[N]: required. zero_a: INT32[M] of magnitude
 * below 2^24; sum_b: INT32[N], sum_b[n] = sum_k b(k,n) (gemm_int8_col_sums);
 * both NULL for symmetric codes, one alone returns GEMM_ERR_NULL_POINTER.
 * workspace: at least gemm_workspace_size(M, N, K, 1) bytes.
 */
gemm_status gemm_int8_scaled(int64_t M, int64_t N, int64_t K, float alpha,
                             const void* A, int64_t lda, gemm_layout layout_a,
                             const void* B, int64_t ldb, gemm_layout layout_b,
                             const float* scale_a, const int32_t* zero_a,
                             const float* scale_b, const int32_t* sum_b,
                             float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                             const void* bias, gemm_act act,
                             void* workspace, size_t workspace_bytes, void* stream);

/* gemm_int8_scaled with the quantising epilogue of gemm_bf16_quant. */
gemm_status gemm_int8_scaled_quant(int64_t M, int64_t N, int64_t K, float alpha,
                                   const void* A, int64_t lda, gemm_layout layout_a,
                                   const void* B, int64_t ldb, gemm_layout layout_b,
                                   const float* scale_a, const int32_t* zero_a,
                                   const float* scale_b, const int32_t* sum_b,
                                   const void* bias, gemm_act act,
                                   const float* out_scale, const int32_t* out_zero,
                                   void* Q, int64_t ldq, gemm_qout_dtype q_dtype,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Per-token INT8 quantisation of BF16 activations, the A operand and scale_a
 * of gemm_int8_scaled. For each row m of X:
 *   scale[m]   = fp32(max_k |x(m,k)| / 127), or 1 if the row is all zero
 *   Q[m*ldq+k] = round-to-nearest-even of fp32(x(m,k) / scale[m]), in [-127, 127]
 * Arguments, edge cases and errors as for gemm_quantize_fp8_rows. A row with a
 * NaN or an infinity gets undefined codes and scale; other rows are untouched
 * by it.
 */
gemm_status gemm_quantize_int8_rows(int64_t M, int64_t K, const void* X, int64_t ldx,
                                    void* Q, int64_t ldq, float* scale, void* stream);

/*
 * sums[n] = sum_k b(k,n) of an INT8 weight in COL layout (N rows of ldb >= K
 * bytes), the sum_b of the INT8 products. Once per weight. K at most 131071.
 * Errors: GEMM_ERR_BAD_DIM, GEMM_ERR_UNSUPPORTED (K), GEMM_ERR_BAD_LD,
 * GEMM_ERR_NULL_POINTER, GEMM_ERR_HIP. K == 0 writes zeros.
 */
gemm_status gemm_int8_col_sums(int64_t K, int64_t N, const void* B, int64_t ldb,
                               int32_t* sums, void* stream);

/*
 * Products grouped by rows: the rows of A belong to G groups ("experts"), each
 * with a weight of its own. Rows offsets[g] .. offsets[g+1]-1 of A and C are
 * group g's:
 *
 *   C[r,n] = act( alpha * (scale_a[r] * scale_b[g][n]) * sum_k A[r,k] B_g[k,n]
 *                 + beta * C[r,n] + bias[g][n] )          (scales: 8-bit calls)
 *
 * T rows in all. A: T x K, ROW layout (tokens sorted by group), lda >= K.
 * offsets: DEVICE INT32[G+1], 4-byte aligned, non-decreasing, within [0, T];
 * no host copy is needed and nothing is synchronised. Groups may be empty and
 * of any length. Rows before offsets[0] or from offsets[G] on belong to no
 * group: their rows of C are neither read nor written, so A and C may be
 * buffers of a fixed capacity T. Offsets that decrease or leave [0, T] give
 * undefined results in C, but no access outside the arrays.
 * B: group g's weight starts stride_b elements after group g-1's (stride_b >=
 * 0; 0 shares one weight); layout_b and ldb describe each as in gemm_bf16.
 * gemm_grouped_bf16 takes both layouts: with weights stored as N rows of K
 * (COL) the call is the layer's forward pass, and the same array read as
 * ROW, K and N exchanged, is its input gradient dX = dY W. The 8-bit calls
 * take COL only (GEMM_ERR_UNSUPPORTED). bias: BF16[G][N] or NULL; scale_a:
 * FP32[T]; scale_b: FP32[G][N]; zero_a INT32[T] and sum_b INT32[G][N] as in
 * gemm_int8_scaled. C: T x N, ldc >= N. No workspace.
 * G == 0, T == 0 or N == 0 launches nothing; K == 0 as in gemm_bf16.
 * Errors: GEMM_ERR_BAD_ENUM, GEMM_ERR_BAD_DIM (a size negative or above 2^30,
 * G above 65536), GEMM_ERR_BAD_LD (a leading dimension, or stride_b < 0),
 * GEMM_ERR_NULL_POINTER, GEMM_ERR_UNSUPPORTED (layout, INT8 K above 131071,
 * offsets not 4-byte aligned), GEMM_ERR_HIP; before anything is enqueued
 * except the last.
 */
gemm_status gemm_grouped_bf16(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                              const void* A, int64_t lda, const int32_t* offsets,
                              const void* B, int64_t ldb, gemm_layout layout_b, int64_t stride_b,
                              float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                              const void* bias, gemm_act act, void* stream);

gemm_status gemm_grouped_fp8_scaled(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                    const void* A, int64_t lda, const int32_t* offsets,
                                    const void* B, int64_t ldb, gemm_layout layout_b,
                                    int64_t stride_b, const float* scale_a, const float* scale_b,
                                    float beta, void* C, int64_t ldc, gemm_out_dtype c_dtype,
                                    const void* bias, gemm_act act, void* stream);

gemm_status gemm_grouped_int8_scaled(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                     const void* A, int64_t lda, const int32_t* offsets,
                                     const void* B, int64_t ldb, gemm_layout layout_b,
                                     int64_t stride_b, const float* scale_a,
                                     const int32_t* zero_a, const float* scale_b,
                                     const int32_t* sum_b, float beta, void* C, int64_t ldc,
                                     gemm_out_dtype c_dtype, const void* bias, gemm_act act,
                                     void* stream);

/*
 * Weight gradient of gemm_grouped_bf16: for every group g,
 *
 *   C_g[n,k] = alpha * sum over g's rows r of D[r,n] X[r,k] + beta * C_g[n,k]
 *
 * D: BF16, T x N (the gradient of the output), ldd >= N. X: BF16, T x K (the
 * layer's input), ldx >= K. offsets as above; an empty group's gradient is
 * beta * C_g (zeros for beta == 0, C then not being read). C_g: N rows of
 * ldc >= K, c_dtype FP32 or BF16, the layout of a COL weight (exchange D and
 * X for a ROW one); group g's starts stride_c elements after group g-1's,
 * stride_c >= (N-1)*ldc + K where G > 1 (else GEMM_ERR_BAD_LD). beta = 1 adds
 * to the gradient of earlier micro-batches. Sums are FP32. No workspace.
 * G == 0, N == 0 or K == 0 launches nothing; T == 0 leaves beta * C.
 * Other errors as above.
 */
gemm_status gemm_grouped_bf16_wgrad(int64_t G, int64_t T, int64_t N, int64_t K, float alpha,
                                    const void* D, int64_t ldd, const void* X, int64_t ldx,
                                    const int32_t* offsets, float beta, void* C, int64_t ldc,
                                    int64_t stride_c, gemm_out_dtype c_dtype, void* stream);

/*
 * Routing: which experts a token's rows go to, and with what weights.
 * For every token t, from its logits x[t, e] (e < E):
 *
 *   s_e = softmax over e of x[t, e], or sigmoid(x[t, e])
 *   c_e = s_e + bias[e]                          (bias chooses, it is in no weight)
 *   groups > 1: E/groups neighbouring experts are a group; a group's score is the
 *     sum of its group_best (1 or 2) largest c; only experts of the top_groups
 *     best groups are chosen
 *   expert[t, 0..top_k-1] = the experts of the top_k largest c, largest first
 *   weight[t, j] = scale * s_j, or scale * s_j / sum over the chosen s (renormalise != 0)
 *
 * Equal values go to the lowest index, of experts as of groups. Without bias (and with
 * one group or one best of each) the logits themselves are compared, which is exact.
 * Otherwise scores formed in 64 bits are, and what those do not tell apart is equal:
 * sigmoids of logits above 37 are all 1, softmax scores of logits 746 below the row's
 * largest all 0, and a bias of 2^53 leaves nothing of a score. Weights are FP32;
 * renormalised ones are formed from the scores' logarithms, so that scores too small
 * for FP32 still have shares.
 * An expert whose logit (or bias) is -inf is not available. A token with fewer
 * than top_k available experts (in its groups) has expert -1 and weight 0 in
 * the slots that are left: a row that is all -inf, such as padding, in all of
 * them. A row with a NaN (under softmax: or +inf) has expert -1 and weight
 * NaN. A NaN in bias makes its expert unavailable.
 * logits: T rows of E, FP32 or BF16 (l_dtype), ldl >= E. bias: FP32[E] or
 * NULL. expert: INT32[T][top_k]; weight: FP32[T][top_k]; contiguous.
 * E at most 1024, top_k at most 32 and groups at most 64 (else
 * GEMM_ERR_UNSUPPORTED). GEMM_ERR_BAD_DIM: T negative or above 2^30, E < 1,
 * groups that do not divide E, top_groups outside [1, groups], group_best other
 * than 1 or 2, top_k < 1 or above the experts of top_groups groups.
 * GEMM_ERR_BAD_ENUM: l_dtype, score. Then GEMM_ERR_BAD_LD,
 * GEMM_ERR_NULL_POINTER, GEMM_ERR_UNSUPPORTED (a pointer not aligned to its
 * elements), GEMM_ERR_HIP. T == 0 launches nothing. expert and weight may not
 * overlap each other or the inputs.
 */
typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score;

gemm_status gemm_route(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ldl,
                       gemm_out_dtype l_dtype, gemm_score score, const float* bias,
                       int64_t groups, int64_t top_groups, int group_best, int renormalise,
                       float scale, int32_t* expert, float* weight, void* stream);

/*
 * Gradient of gemm_route's weights with respect to its logits, the choice held
 * fixed: dlogits[t, e] = sum_j dweight[t, j] * d weight[t, j] / d x[t, e], for
 * all E columns (zeros where nothing arrives), in the logits' type, FP32
 * before its one rounding. The bias has no gradient.
 * expert as gemm_route wrote it; slots whose expert is outside [0, E) are
 * passed over, and their dweight is not used. A row without any expert gets
 * zeros. An expert named by several slots gets the sum of their gradients.
 * dlogits: T rows of E, ldd >= E; may not overlap the inputs. Limits and
 * errors as for gemm_route.
 */
gemm_status gemm_route_grad(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ldl,
                            gemm_out_dtype l_dtype, gemm_score score, int renormalise, float scale,
                            const int32_t* expert, const float* dweight, void* dlogits,
                            int64_t ldd, void* stream);

/*
 * The order of rows by expert: S slots (S = T * top_k, slot t * top_k + j) with
 * an expert each are sorted by expert, stably, into rows.
 *   offsets[g]  = slots whose expert is below g: the offsets of the grouped
 *                 products, G + 1 of them; offsets[G] slots have an expert
 *   position[s] = the row of slot s, or -1 if its expert is outside [0, G)
 *   order[r]    = the slot of row r, or -1 for the rows from offsets[G] on
 * expert, position: INT32[S]; offsets: INT32[G+1]; order: INT32[S] or NULL.
 * No array may overlap another. Nothing is synchronised.
 * workspace: device scratch of gemm_route_order_workspace_size(S, G) bytes,
 * 4-byte aligned. G at most 8192 (GEMM_ERR_UNSUPPORTED). GEMM_ERR_BAD_DIM: S
 * negative or above 2^30, G < 0. S == 0 writes zeros to offsets.
 */
gemm_status gemm_route_order(int64_t S, int64_t G, const int32_t* expert, int32_t* offsets,
                             int32_t* position, int32_t* order, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Bytes of workspace of gemm_route_order; 0 for sizes it refuses. */
size_t gemm_route_order_workspace_size(int64_t S, int64_t G);

/*
 * Rows of tokens to their experts: Y[position[t * top_k + j], :] = X[t, :]
 * X: T rows of N elements of elem_bytes (1, 2 or 4: codes, BF16, FP32 or the
 * scales of codes; moved as bits), ldx >= N. Y: R rows, ldy >= N. Positions
 * outside [0, R) are passed over. Rows of Y that no slot names are not
 * written. A position named twice gets one of its rows, or parts of several.
 * Y may not overlap X. Its gradient is gemm_combine_rows without weights.
 * Errors: GEMM_ERR_BAD_ENUM (elem_bytes), GEMM_ERR_BAD_DIM (a size negative or
 * above 2^30, T * top_k above 2^30, top_k < 1), GEMM_ERR_UNSUPPORTED (top_k above 64, X or Y not
 * aligned to its elements), GEMM_ERR_BAD_LD,
 * GEMM_ERR_NULL_POINTER, GEMM_ERR_HIP. T == 0, R == 0 or N == 0 launches nothing.
 */
gemm_status gemm_dispatch_rows(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* X,
                               int64_t ldx, int elem_bytes, const int32_t* position, void* Y,
                               int64_t ldy, void* stream);

/*
 * Rows of experts back to their tokens:
 *   C[t, :] = sum_j weight[t, j] * Y[position[t * top_k + j], :] + beta * C[t, :]
 * summed in FP32 in the order of j, rounded once. Slots with a position
 * outside [0, R) add nothing, whatever their weight (a token without slots:
 * beta * C). C may not overlap Y. Y: R rows of N, FP32 or BF16, ldy >= N. weight: FP32[T][top_k],
 * or NULL for ones. C: T rows, FP32 or BF16, ldc >= N, not read for beta == 0.
 * Errors as for gemm_dispatch_rows; GEMM_ERR_BAD_ENUM for the types. T == 0 or
 * N == 0 launches nothing; R == 0 gives beta * C.
 */
gemm_status gemm_combine_rows(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* Y,
                              int64_t ldy, gemm_out_dtype y_dtype, const int32_t* position,
                              const float* weight, float beta, void* C, int64_t ldc,
                              gemm_out_dtype c_dtype, void* stream);

/*
 * Gradients of gemm_combine_rows, D being C's:
 *   dY[position[t * top_k + j], :] = weight[t, j] * D[t, :]
 *   dweight[t, j] = sum over n of D[t, n] * Y[position[t * top_k + j], n]   (0 without a position)
 * D: T rows of N, d_dtype, ldd >= N. Y, dY: R rows, y_dtype. weight as above
 * (NULL: ones). dweight: FP32[T][top_k], or NULL: it is not computed and Y,
 * which may be NULL then, not read. Rows of dY that no slot names are not
 * written; a row that several name gets the gradient of one, or parts of several. dY
 * may not overlap D or Y. Sums are FP32. Errors as above.
 */
gemm_status gemm_combine_rows_grad(int64_t T, int64_t top_k, int64_t R, int64_t N, const void* D,
                                   int64_t ldd, gemm_out_dtype d_dtype, const void* Y, int64_t ldy,
                                   gemm_out_dtype y_dtype, const int32_t* position,
                                   const float* weight, void* dY, int64_t lddy, float* dweight,
                                   void* stream);

/*
 * A shared projection with low-rank adapters, of many requests at once: row m
 * of A belongs to a request that has adapter a = adapter[m] of its own,
 *
 *   C[m,:] = act( alpha * (A[m,:] B + scale[a] * (A[m,:] down_a) up_a) + beta * C[m,:] + bias )
 *
 * and the plain projection where adapter[m] is outside [0, G). Rows come in
 * any order; neighbours that share an adapter share its work.
 * A: BF16, M rows of K (ROW), lda >= K. B: BF16, N rows of K (COL: K-major;
 * gemm_pack_b reorders a weight), ldb >= K. adapter: INT32[M].
 * down: BF16, adapter g's R rows of K start stride_down * g elements in,
 * ld_down >= K. up: BF16, its N rows of R at stride_up * g, ld_up >= R.
 * (An adapter of lower rank has rows of zeros in down.) scale: FP32[G], or
 * NULL for ones. R at most 128; G == 0 or R == 0 is the plain projection.
 * Sums are FP32. scale * (A down) passes to the second product as BF16 values whose sum it
 * is: two for BF16 output, which keep 16 bits of it, three for FP32 output, which keep all
 * 24. An adapter's infinities and NaN
 * stay in its own rows. C, bias, act, beta and alpha as in gemm_bf16.
 * workspace: gemm_lora_workspace_size(M, N, K, R) bytes, 16-byte aligned.
 * Errors as for gemm_bf16; GEMM_ERR_BAD_LD also for a negative stride_down or
 * stride_up; GEMM_ERR_UNSUPPORTED for R above 128 or G above 65536, A or B that spans
 * 2^31 bytes or more (B may where M <= 16, K is a multiple of 8 and the rows of A and B are
 * 16-byte aligned; more than 2^26 - 16 columns take K <= 4096 and R <= 32 as well), BF16
 * operands at odd addresses, a workspace not 16-byte aligned.
 */
gemm_status gemm_lora_bf16(int64_t M, int64_t N, int64_t K, int64_t G, int64_t R, float alpha,
                           const void* A, int64_t lda, const void* B, int64_t ldb,
                           const int32_t* adapter, const void* down, int64_t ld_down,
                           int64_t stride_down, const void* up, int64_t ld_up, int64_t stride_up,
                           const float* scale, float beta, void* C, int64_t ldc,
                           gemm_out_dtype c_dtype, const void* bias, gemm_act act,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of gemm_lora_bf16; 0 for sizes it refuses. */
size_t gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R);

/*
 * One-time reorder of a weight matrix B (logical K x N) into the layout the
 * fast path reads: Bp[n*ldbp + k] = b(k, n), i.e. GEMM_COL_MAJOR (K-major)
 * with leading dimension ldbp. The FP8 DeepGEMM page (sec. 3.2) rearranges B
 * once, before the calls that reuse it, so the reorder is paid once per
 * weight. Pass the result to gemm_bf16 / gemm_fp8_scaled / gemm_mxfp8 with
 * layout_b = GEMM_COL_MAJOR and ldb = ldbp: a K-major B (below 2^31 bytes)
 * is copied to on-chip memory by DMA (the fast path) at any alignment, while
 * an N-contiguous B is read through registers, several times slower, unless
 * it is BF16 with 16-byte aligned rows and N a multiple of 8. With ldbp *
 * elem_bytes and K * elem_bytes multiples of 16 and Bp 16-byte aligned, the
 * DMA reads are aligned and decode-sized M can use the skinny kernel.
 * B: device, elements of elem_bytes (2: BF16, 1: E4M3; moved as bits), in
 * layout_b (ROW: b(k,n) = B[k*ldb + n], ldb >= N; COL: B[n*ldb + k],
 * ldb >= K). Bp: device, N rows of ldbp >= K elements; the elements k >= K of
 * each row are not written. Bp must not overlap B.
 * Errors (before anything is enqueued): GEMM_ERR_BAD_ENUM (layout_b,
 * elem_bytes), GEMM_ERR_BAD_DIM (K or N negative or above 2^30),
 * GEMM_ERR_BAD_LD, GEMM_ERR_NULL_POINTER (B or Bp when K, N > 0),
 * GEMM_ERR_HIP. K == 0 or N == 0 does nothing.
 */
gemm_status gemm_pack_b(int64_t K, int64_t N, const void* B, int64_t ldb, gemm_layout layout_b,
                        int elem_bytes, void* Bp, int64_t ldbp, void* stream);

/*
 * Bytes of device workspace a call with these sizes needs (0 when the chosen
 * kernel needs none). Pure host arithmetic; callable without a GPU. Query
 * once and allocate up front (the FP8 page's interface, sec. 5.1, separates
 * the size query from the call for the same reason). is_fp8: 0 for
 * gemm_bf16, 1 for gemm_fp8_scaled and gemm_int8_scaled. Negative sizes return 0.
 */
size_t gemm_workspace_size(int64_t M, int64_t N, int64_t K, int is_fp8);

/*
 * The launch plan the library would use (host arithmetic only, no GPU
 * needed): tile sizes, split-K factor and grid. Returns GEMM_OK or
 * GEMM_ERR_BAD_DIM / GEMM_ERR_NULL_POINTER. Intended for tests and tuning.
 */
typedef struct {
  int32_t kernel;       /* 0 = tiled MFMA kernel, 1 = skinny weight-streaming kernel
                           (M <= 16; K split over the waves of a workgroup) */
  int32_t tile_m, tile_n, tile_k;
  int32_t split_k;      /* number of K partitions (1 = none) */
  int32_t waves;        /* wavefronts per workgroup */
  int64_t grid;         /* workgroups launched by the main kernel */
  size_t workspace_bytes;
} gemm_plan_info;

gemm_status gemm_plan(int64_t M, int64_t N, int64_t K, int is_fp8, gemm_plan_info* out);

/* Static, NUL-terminated name of a status code ("GEMM_OK", ...). */
const char* gemm_status_string(gemm_status s);

#ifdef __cplusplus
}
#endif

#endif /* GEMM355_H */
