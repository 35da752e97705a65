/*
 * puro_ops.h -- C ABI of the operators around the blockwise-scaled FP8 linear layer (MI355X / gfx950):
 * the norm in front of it (as a tensor, as the codes and scales its products read, and backward),
 * the product of those codes for any number of rows, and the clipping of its gradients by their
 * global norm.  Same library (libpuro_fp8.so) as puro_fp8.h, whose status codes, output types and
 * conventions hold here too, except where an entry point says otherwise:
 *   - device pointers, row-major matrices, leading dimensions in elements;
 *   - everything is enqueued on the caller's stream `st`, nothing synchronizes or allocates;
 *   - every argument check runs on the host before any HIP call; a failed check launches nothing;
 *   - no state is kept between calls; concurrent calls on different streams are independent when
 *     their outputs and workspaces do not overlap.  A workspace is written before it is read within
 *     each call and needs no initialization; calls that may run at the same time (two streams, two
 *     captured graphs) need one each.
 * Every result is deterministic: no atomics, all sums in a fixed order.
 */
#ifndef PURO_OPS_H
#define PURO_OPS_H

#include "puro_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Kind of norm.  With mu the row's mean and n = C columns,
 *   LAYER: y = (x - mu) / sqrt(sum (x - mu)^2 / n + eps) * weight + bias
 *   RMS:   y = x / sqrt(sum x^2 / n + eps) * weight (+ bias)
 * The pages' model is built on the Qwen3-1.7B configuration, whose blocks have RMS norms in front of
 * their FP8 linear layers; the layer norm is the same kernel with the mean taken out. */
enum { PURO_NORM_LAYER = 0, PURO_NORM_RMS = 1 };

/*
 * Norm of each row.
 *   x      : [T, C] of x_dtype (PURO_OUT_BF16 or PURO_OUT_FP32), row stride ldx; 0 <= T, 0 <= C <= 16384.
 *   weight : [C], bias: [C] or NULL, both of w_dtype (PURO_OUT_BF16 or PURO_OUT_FP32).
 *   eps    : finite, >= 0 (else PURO_ERR_ARG).
 *   y      : [T, C] of x_dtype, row stride ldy.  y may be x (same pointer and stride).
 *   mean, rstd : fp32 [T], the row statistics the backward pass takes; each optional (NULL).  RMS has
 *            no mean: mean must be NULL (else PURO_ERR_ARG).  With C == 0 nothing is written, these included.
 * Mean and variance are taken in fp32 from the row held in registers (variance of the differences
 * from the mean, not of squares), y is rounded once.  Rows need only element alignment (2 or 4
 * bytes, any ldx >= C); 16-byte aligned rows with C % 8 == 0 take the fast path.
 * A NaN or an infinity stays in its row (a layer norm's whole row becomes NaN).  Squares are fp32: beyond about 1e17
 * of |x - mu| their sum leaves its range, rstd is 0 and y is bias; beyond 2e34 of |x| so does a layer norm's sum, and
 * the row is NaN.  C > 16384: PURO_ERR_UNSUPPORTED.
 */
int puro_layer_norm(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                    const void* weight, const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                    hipStream_t st);

/*
 * Norm of each row, written as the 1x128 codes and scales an FP8 product reads (layouts of
 * puro_fp8_quant_act_1x128): q uint8 [T, C] (row stride ldq), s fp32 [C/128][T].  The group maximum,
 * scale and codes come from the fp32 norm (one rounding, to E4M3; the numerics of puro_fp8.h with
 * the fp32 value in place of the bf16 one), so y itself is never written.  A NaN has a NaN code and does not
 * enter its group's scale.  Any T >= 0; C % 128 == 0.
 * x, q and s 16-byte aligned, rows a multiple of 16 bytes apart, as in puro_fp8.h; weight and bias
 * 16-byte aligned.  mean and rstd as in puro_layer_norm.
 */
int puro_layer_norm_quant(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                          const void* weight, const void* bias, float eps, uint8_t* q, int64_t ldq, float* s,
                          float* mean, float* rstd, hipStream_t st);

/*
 * As puro_layer_norm_quant, with the transposed 128x1 codes of the same fp32 norm as well (layouts of
 * puro_fp8_quant_act_dual): qT uint8 [C, T] (row stride ldqT), sT fp32 [T/128][C].  The training form:
 * q feeds FWD, qT feeds WGRAD.  T % 128 == 0, C % 128 == 0.  rstd is required, and so is mean for
 * PURO_NORM_LAYER: the second launch reads them.  q and s are puro_layer_norm_quant's, bit for bit.
 */
int puro_layer_norm_quant_dual(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                               const void* weight, const void* bias, float eps, uint8_t* q, int64_t ldq, float* s,
                               uint8_t* qT, int64_t ldqT, float* sT, float* mean, float* rstd, hipStream_t st);

/*
 * Backward pass of the norm.  With xh = (x - mean) * rstd (RMS: x * rstd) and u = dy * weight:
 *   dx      = rstd * (u - mean_c(u) - xh * mean_c(u * xh))      (RMS: without mean_c(u))
 *   dweight = sum_t dy * xh,   dbias = sum_t dy
 *   dy, x, dx : [T, C] of x_dtype, row strides lddy, ldx, lddx (element alignment, as puro_layer_norm);
 *               dx may be dy or x (same pointer and stride).
 *   mean    : fp32 [T] (NULL for RMS, else PURO_ERR_ARG), rstd: fp32 [T], from the forward pass.
 *   dweight : fp32 [C]; dbias: fp32 [C] or NULL.  accumulate = 0 sets them, 1 adds to them (one fp32
 *             addition per element; for gradients kept over micro-batches).
 *               Both are fp32 sums of short runs (64 rows, 64 of those sums, up to 32 rows at a time): their
 *               error does not grow with T.
 *   workspace : puro_layer_norm_backward_workspace_size(T, C) bytes, 16-byte aligned (NULL when 0).
 * T == 0 (or C == 0) writes no dx; with accumulate = 0 it still sets dweight and dbias to zero.
 */
int puro_layer_norm_backward(int kind, int x_dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                             int64_t T, int64_t C, int w_dtype, const void* weight, const float* mean,
                             const float* rstd, void* dx, int64_t lddx, float* dweight, float* dbias, int accumulate,
                             void* workspace, size_t workspace_bytes, hipStream_t st);
size_t puro_layer_norm_backward_workspace_size(int64_t T, int64_t C);

/*
 * One gradient tensor: n contiguous elements of dtype (PURO_OUT_BF16 or PURO_OUT_FP32) at src, and
 * where its clipped values go (dst: same type; dst == src clips in place).  Element alignment; n >= 0.
 */
typedef struct puro_grad_job {
  const void* src;
  void* dst;      /* ignored by puro_grad_norm */
  int64_t n;
  int dtype;
} puro_grad_job;

/*
 * Global norm of n_jobs tensors: *norm = sqrt(sum of all squares), fp32, on the device.  Squares are
 * taken and summed in 64 bits, so nothing overflows or is lost below the fp32 range of the result.
 *   jobs : host array (read before the call returns; not kept); any n_jobs >= 0 (0: norm is 0).
 *   norm : fp32 [1], on the device.
 *   workspace : puro_grad_norm_workspace_size(jobs, n_jobs) bytes, 16-byte aligned, apart from the tensors
 *          (else PURO_ERR_ARG).
 */
int puro_grad_norm(const puro_grad_job* jobs, int n_jobs, float* norm, void* workspace, size_t workspace_bytes,
                   hipStream_t st);

/*
 * Clipping by the global norm: as puro_grad_norm, then dst = src * c with
 *   c = min(1, max_norm / (norm + 1e-6))
 * in fp32, rounded once to the tensor's type.  max_norm: >= 0, not NaN (else PURO_ERR_ARG).  Where c is
 * 1 and dst == src nothing is written.  A norm that is not finite is not hidden: an infinite one gives
 * c = 0 (infinite elements become NaN; where max_norm is infinite too, c and every element), a NaN makes
 * every element NaN, as the product says.  A dst
 * that overlaps another job's src or dst, or its own src other than being it, is refused (PURO_ERR_ARG):
 * a gradient that is listed twice is one.  So is a norm inside a tensor or inside the part of the workspace
 * that the call uses.
 */
int puro_clip_grad_norm(const puro_grad_job* jobs, int n_jobs, float max_norm, float* norm, void* workspace,
                        size_t workspace_bytes, hipStream_t st);

/*
 * The second half alone: dst = src * min(1, max_norm / (*norm + 1e-6)) with a norm that is already on
 * the device (fp32 [1]), e.g. one joined over several processes.  It lies outside
 * the tensors (else PURO_ERR_ARG).
 */
int puro_scale_by_norm(const puro_grad_job* jobs, int n_jobs, float max_norm, const float* norm, hipStream_t st);

size_t puro_grad_norm_workspace_size(const puro_grad_job* jobs, int n_jobs);

/*
 * The FWD / DGRAD product of puro_fp8_gemm for any number of rows M >= 0 (single tokens, decode
 * batches, ragged prompts):  C[m,n] = sum_kb sA[kb][m] sB[n/128][kb] sum_{k in kb} dec(A[m,k]) dec(B[n,k]).
 *   A : uint8 codes [M, K], row stride lda; sA: fp32 [K/128][M]     (puro_fp8_quant_act_1x128)
 *   B : uint8 codes [N, K], row stride ldb; sB: fp32 [N/128][K/128] (puro_fp8_quant_w_128x128)
 *   C : [M, N] of out_dtype, row stride ldc.  N % 128 == 0, K % 128 == 0.  K == 0 gives zeros.
 *         M, K < 2^31, N < 2^29, lda, ldb <= 2^29 (else PURO_ERR_UNSUPPORTED).
 *   workspace : puro_gemm_rows_workspace_size(M, N, K) bytes, 16-byte aligned (NULL when 0); an fp32 output needs
 *         none.
 * Alignment as puro_fp8_gemm (16-byte pointers and row strides; sA and sB 4-byte).  Codes are decoded exactly to bf16
 * and multiplied by bf16 matrix instructions with fp32 sums, each 128-deep slice scaled into a separate fp32
 * accumulator (measured up to 3e-7 of the sum of magnitudes off).  Of a long bf16 product the leading multiple of 128
 * rows is what puro_fp8_gemm writes for them, with its FP8 matrix instructions' sums (up to 1.6e-4): from 2^33
 * multiplications of at least 256 leading rows, 2^34 of 128 (weights that puro_fp8_gemm's 32-bit offsets do not reach
 * excepted).  An fp32 output has the row kernel's sums throughout.  The last bits of a row depend on M in any case: the
 * order of the sums goes by the tile.
 */
int puro_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B,
                   int64_t ldb, const float* sB, void* C, int64_t ldc, int out_dtype, void* workspace,
                   size_t workspace_bytes, hipStream_t st);
size_t puro_gemm_rows_workspace_size(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* PURO_OPS_H */
