/*
 * puro_ops.h -- C ABI of the operators around the blockwise-scaled FP8 linear layer (MI355X / gfx950):
 * the norm in front of it (as a tensor, as the codes and scales its products read, and backward), alone
 * and together with the residual sum behind the block before, the product of those codes for any number of
 * rows, rotary positions, the clipping of its gradients by their global norm, and the AdamW step.  Same library (libpuro_fp8.so) as puro_fp8.h, whose status codes, output types and
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

/*
 * The residual sum behind a block together with the norm in front of the next one.  With norm() as puro_layer_norm of `kind`
 * without weight and bias, row by row:
 *   p     = x                          (post_weight NULL)
 *         = norm(x) * post_weight      (a norm behind the block)
 *   h_out = h + scale * gate * p       (gate NULL: 1), rounded to x_dtype
 *   y     = norm(h_out) * weight + bias
 * The norm is that of h_out as it is written: y, mean and rstd (or the codes and scales) are those that puro_layer_norm
 * (puro_layer_norm_quant, ..._dual) gives for it, bit for bit.
 * h_out may be h or x (same pointer and stride).  Other than that nothing that is written may share memory with anything else
 * that the call reads or writes (PURO_ERR_ARG); rows of one buffer whose columns lie side by side share none.
 */
typedef struct puro_residual {
  int kind;               /* PURO_NORM_LAYER, PURO_NORM_RMS: of both norms */
  int x_dtype;            /* of h, x, h_out and y: PURO_OUT_BF16, PURO_OUT_FP32 */
  int w_dtype;            /* of weight, bias, gate and post_weight */
  int64_t T, C;           /* 0 <= T, 0 <= C <= 16384 */
  const void* h;          /* [T, C], the residual stream, row stride ldh */
  int64_t ldh;
  const void* x;          /* [T, C], the block's output, row stride ldx */
  int64_t ldx;
  const void* weight;     /* [C] */
  const void* bias;       /* [C] or NULL */
  const void* gate;       /* [C] or NULL */
  const void* post_weight; /* [C] or NULL */
  float scale;            /* finite (else PURO_ERR_ARG) */
  float eps;              /* of both norms: finite, >= 0 (else PURO_ERR_ARG) */
  void* h_out;            /* [T, C], row stride ldh_out */
  int64_t ldh_out;
  float* mean;            /* fp32 [T] or NULL, as puro_layer_norm (an RMS norm has none: NULL) */
  float* rstd;            /* fp32 [T] or NULL */
  float* post_mean;       /* the statistics of the norm of x, likewise; without post_weight NULL (else PURO_ERR_ARG) */
  float* post_rstd;
} puro_residual;

/*
 * The norm as a tensor: y [T, C] of x_dtype, row stride ldy.  As h_out, y may be h or x, but not both the same tensor.  Rows
 * need element alignment, as in puro_layer_norm.
 * The struct is read before the call returns.
 */
int puro_residual_norm(const puro_residual* r, void* y, int64_t ldy, hipStream_t st);

/*
 * The norm as 1x128 codes and scales (layouts and numerics of puro_layer_norm_quant): q uint8 [T, C], s fp32 [C/128][T].
 * Any T >= 0; C % 128 == 0.  Pointers 16-byte aligned, rows a multiple of 16 bytes apart.
 */
int puro_residual_norm_quant(const puro_residual* r, uint8_t* q, int64_t ldq, float* s, hipStream_t st);

/*
 * With the transposed 128x1 codes as well (layouts of puro_layer_norm_quant_dual): the training form.  T % 128 == 0,
 * C % 128 == 0.  rstd is required, and so is mean for PURO_NORM_LAYER.
 */
int puro_residual_norm_quant_dual(const puro_residual* r, uint8_t* q, int64_t ldq, float* s, uint8_t* qT, int64_t ldqT,
                                  float* sT, hipStream_t st);

/*
 * Backward pass.  With D = (backward pass of the norm at h_out, of dy) + dh_out, kept in fp32:
 *   dh      = D
 *   dx      = scale * gate * D                                     (post_weight NULL)
 *           = backward pass of the norm at x, of scale * gate * D * post_weight
 *   dweight = sum_t dy * xh(h_out),  dbias = sum_t dy
 *   dgate   = scale * sum_t D * p,   dpost_weight = scale * gate * sum_t D * xh(x)
 * Every sum over rows in short fp32 runs, as puro_layer_norm_backward's.
 */
typedef struct puro_residual_grad {
  int kind, x_dtype, w_dtype;
  int64_t T, C;
  const void* dy;         /* [T, C] of x_dtype, row stride lddy */
  int64_t lddy;
  const void* h_out;      /* [T, C], from the forward pass */
  int64_t ldh_out;
  const void* dh_out;     /* [T, C], its gradient from behind, or NULL (zero) */
  int64_t lddh_out;
  const void* x;          /* [T, C], the forward pass's; read with a gate or a post_weight alone, else ignored */
  int64_t ldx;
  const void* weight;     /* [C] */
  const void* gate;       /* [C] or NULL */
  const void* post_weight; /* [C] or NULL */
  float scale;
  const float* mean;      /* fp32 [T], from the forward pass (RMS: NULL, else PURO_ERR_ARG) */
  const float* rstd;
  const float* post_mean; /* with post_weight alone (else NULL, or PURO_ERR_ARG) */
  const float* post_rstd;
  void* dh;               /* [T, C] of x_dtype */
  int64_t lddh;
  void* dx;               /* [T, C] of x_dtype.  NULL without gate and post_weight: not written (with scale 1 it equals dh) */
  int64_t lddx;
  float* dweight;         /* fp32 [C] */
  float* dbias;           /* fp32 [C] or NULL */
  float* dgate;           /* fp32 [C] or NULL; without a gate NULL (else PURO_ERR_ARG) */
  float* dpost_weight;    /* fp32 [C] or NULL; without post_weight NULL (else PURO_ERR_ARG) */
  int accumulate;         /* 0 sets the four sums, 1 adds to them */
} puro_residual_grad;

/*
 * workspace: puro_residual_norm_backward_workspace_size(T, C, gated) bytes, gated = 1 with a gate or a post_weight; 16-byte
 * aligned (NULL when 0).  T == 0 (or C == 0) writes no dh and dx; with accumulate = 0 it still sets the sums to zero.
 * dh and dx may each be one of dy, h_out, dh_out and x (same pointer and stride), not both the same.  Other than that nothing that
 * is written, the used part of the workspace included, may share memory with anything else of the call (PURO_ERR_ARG).
 */
int puro_residual_norm_backward(const puro_residual_grad* r, void* workspace, size_t workspace_bytes, hipStream_t st);
size_t puro_residual_norm_backward_workspace_size(int64_t T, int64_t C, int gated);

/* Which columns of a head make a pair: i and i + pairs, or 2 i and 2 i + 1. */
enum { PURO_ROTARY_HALF = 0, PURO_ROTARY_INTERLEAVED = 1 };

/*
 * Rotary positions: each pair (a, b) of a head's leading 2 * pairs columns is turned by the token's angle for it,
 *   angle = position * freqs[i],  a' = scale * (a cos - b sin),  b' = scale * (b cos + a sin)
 * and the columns behind them are copied.  inverse = 1 turns by -angle: with the same scale, the backward pass.
 *   x : [T, H, D] of x_dtype, token stride ld_t, head stride ld_h (elements; unit stride within a head).  Any element
 *       alignment; 16-byte aligned heads with D % 8 == 0 (half layout: pairs % 8 == 0) take the fast path.
 *   positions : int64 [T] on the device, or NULL: token t is at start + t.
 *   freqs : fp64 [pairs] on the device, radians a position; 2 * pairs <= D, pairs <= 2048.
 *   scale : finite (else PURO_ERR_ARG); of the turned columns alone, where a long-context scaling has one.
 *   y : [T, H, D] of x_dtype with its own strides; y may be x, with the same strides; other than that it may not share memory
 *       with x, positions or freqs (PURO_ERR_ARG; heads of one buffer beside each other share none).
 * Angles are formed and reduced in 64 bits: position * freq is off by 2^-53 of itself.  Positions beyond 2^53 are rounded.
 * Strides of y that put two heads over each other are refused (PURO_ERR_LD): tokens lie apart from each other with all their
 * heads, or heads with all their tokens.  x may repeat (stride 0).  T, H < 2^31, D <= 2^30.
 */
int puro_rotary(int x_dtype, int layout, int inverse, const void* x, int64_t ld_t, int64_t ld_h, int64_t T, int64_t H,
                int64_t D, const int64_t* positions, int64_t start, const double* freqs, int64_t pairs, float scale, void* y,
                int64_t ldy_t, int64_t ldy_h, hipStream_t st);

/*
 * One tensor of an AdamW step: n contiguous elements each.  States are fp32 (both scales NULL), or 8-bit: E4M3 codes with one
 * fp32 scale for every 128 consecutive elements (the last of a tensor fewer), of the first moment and of the second one's
 * square root.  A block's scale is its largest magnitude (2^-96 at least) times 1 / 448.  States of zero (codes and scales,
 * or fp32) are the start.
 */
typedef struct puro_adamw_job {
  void* param;            /* of param_dtype; updated */
  float* master;          /* fp32 copy of a bf16 param, updated in its place (param is its rounding), or NULL */
  const void* grad;       /* of grad_dtype */
  void* exp_avg;          /* fp32, or uint8 codes */
  void* exp_avg_sq;       /* fp32 (the second moment), or uint8 codes (its square root) */
  float* avg_scale;       /* [ceil(n / 128)], or NULL */
  float* sq_scale;        /* [ceil(n / 128)], or NULL */
  int64_t n;
  int param_dtype, grad_dtype;   /* PURO_OUT_BF16, PURO_OUT_FP32 */
} puro_adamw_job;

typedef struct puro_adamw_hyper {
  double lr, beta1, beta2, eps, weight_decay;   /* finite; 0 <= betas < 1; eps >= 0 (else PURO_ERR_ARG) */
  int64_t step;           /* counted from 1 (else PURO_ERR_ARG) */
  const float* lr_dev;    /* on the device, read by the kernel in place of lr; or NULL */
  const int64_t* step_dev; /* on the device, read by the kernel in place of step (below 1 its factors are infinite); or NULL */
  const float* norm;      /* on the device: gradients are taken times min(1, max_norm / (*norm + 1e-6)); or NULL */
  float max_norm;         /* >= 0, not NaN (else PURO_ERR_ARG); read with a norm alone */
  uint64_t seed;          /* of the rounding of 8-bit states; the step enters too, so it may stay the same */
} puro_adamw_hyper;

/*
 * AdamW (decoupled weight decay) over all tensors of a list:
 *   g  = grad * min(1, max_norm / (*norm + 1e-6))
 *   m' = beta1 m + (1 - beta1) g,   v' = beta2 v + (1 - beta2) g g
 *   param' = param (1 - lr weight_decay) - lr / (1 - beta1^step) * m' / (sqrt(v' / (1 - beta2^step)) + eps)
 * in fp32, the hyperparameters' factors rounded once from 64 bits; squares are fp32 (gradients beyond 1.8e19 overflow).  With
 * eps = 0 an element whose gradients have all been zero becomes NaN (0 / 0); an eps below 2^-126 counts as 0.  A bf16 param without a master loses what
 * its rounding takes of each step.
 * The step takes m' and v' before they are rounded to 8 bits.  8-bit states are rounded by chance among the two nearest
 * three-bit mantissas, which keeps their expected value (less than 2^-16 of a code's step below it in magnitude), where rounding
 * to the nearest would freeze a state that moves by less than half a code's step; the random bits depend on seed, step, the job's index in the list and the element alone.
 * Values below 2^-6 of a block's codes go to the nearest code, and a root that is not zero never becomes zero.
 * A gradient that is not finite is not hidden: a NaN's element becomes NaN (its codes too), an infinity's too, and with 8-bit
 * states an infinity makes all parameters of its block NaN from the next step on.
 *   jobs : host array (read before the call returns; not kept), any n_jobs >= 0; element alignment.  Nothing that is written
 *          may overlap anything else that the call reads or writes (PURO_ERR_ARG).  One scale without the other, or a
 *          master of an fp32 param: PURO_ERR_ARG.
 */
int puro_adamw(const puro_adamw_job* jobs, int n_jobs, const puro_adamw_hyper* h, hipStream_t st);

#ifdef __cplusplus
}
#endif

#endif /* PURO_OPS_H */
