// Internal launcher declarations of the operators of puro_ops.h, between the C-ABI layer (abi_ops.cpp)
// and the kernels.  Shapes and pointers are validated by the caller before any of these runs.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace puro {

// ---- norm (norm.hip) ------------------------------------------------------------------------------
constexpr int64_t kNormMaxC = 16384;   // the widest row the kernels hold in registers

struct NormArgs {
  const void* x;
  int64_t ldx;
  int64_t T;
  int C;
  const void* gamma;
  const void* beta;      // optional
  bool x_bf16, w_bf16;
  bool layer;            // layer norm; else RMS norm
  float eps;
  float* mean;           // optional
  float* rstd;           // optional
  // outputs of the tensor form
  void* y;
  int64_t ldy;
  // outputs of the quantized forms
  uint8_t* q;
  int64_t ldq;
  float* s;
  uint8_t* qT;
  int64_t ldqT;
  float* sT;
  int rows_per_team;     // filled in by the launcher
};
hipError_t launch_norm(NormArgs a, hipStream_t st);
hipError_t launch_norm_quant(NormArgs a, hipStream_t st);
hipError_t launch_norm_quant_dual(NormArgs a, hipStream_t st);
// Its second launch alone: the codes of both orientations from x and the statistics in mean and rstd.
hipError_t launch_norm_tiles(NormArgs a, hipStream_t st);

struct NormBwdArgs {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  int64_t T;
  int C;
  const void* gamma;
  bool x_bf16, w_bf16;
  bool layer;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t lddx;
  float* dgamma;
  float* dbeta;          // optional
  int accumulate;
  float* partial;        // [blocks][2][C], the workspace
};
// Workgroups of the backward pass: one partial sum of the weight's and bias's gradient each.
int norm_bwd_blocks(int64_t T, int64_t C);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st);

// ---- residual sum and norm (residual.hip, residual_bwd.hip) -------------------------------------------
// Whether a call that moves `passes` times T C elements of es bytes reads past the caches.
bool beyond_cache(int64_t T, int64_t C, int64_t es, int passes);

struct ResidualArgs {
  NormArgs n;              // x: the sum as written (h_out), ldx its row stride; the norm of it, and its outputs
  const void* h;
  int64_t ldh;
  const void* b;           // the block's output
  int64_t ldb;
  void* h_out;             // n.x
  const void* gate;        // optional
  const void* post;        // weight of the norm of b, optional
  float scale;
  float* post_mean;        // optional
  float* post_rstd;        // optional
  bool stream;             // filled in by the launcher: h and b are read past the caches, else (bf16, in one launch) h_out written
};
hipError_t launch_residual(ResidualArgs a, hipStream_t st);
hipError_t launch_residual_quant(ResidualArgs a, hipStream_t st);
hipError_t launch_residual_quant_dual(ResidualArgs a, hipStream_t st);

struct ResidualBwdArgs {
  const void* dy;
  int64_t lddy;
  const void* h;           // the sum as written
  int64_t ldh;
  const void* dho;         // its gradient from behind, optional
  int64_t lddho;
  const void* b;           // the block's output (with a gate or a norm of it)
  int64_t ldb;
  int64_t T;
  int C;
  const void* gamma;
  const void* gate;        // optional
  const void* post;        // optional
  float scale;
  bool x_bf16, w_bf16;
  bool layer;
  const float* mean;
  const float* rstd;
  const float* post_mean;
  const float* post_rstd;
  void* dh;
  int64_t lddh;
  void* dx;                // optional without gate and post
  int64_t lddx;
  float* dgamma;
  float* dbeta;            // optional
  float* dgate;            // with a gate
  float* dpost;            // with post
  int accumulate;
  float* partial;          // [blocks][2 or 3][C], the workspace
  bool stream, past;       // filled in by the launcher: the rows are read past the caches, bf16 ones written past them
};
// Workgroups of the backward pass, and the fp32 vectors of C columns that each leaves in the workspace.
int residual_bwd_blocks(int64_t T, int64_t C, bool gated);
constexpr int residual_bwd_sums(bool gated) { return gated ? 3 : 2; }
hipError_t launch_residual_bwd(ResidualBwdArgs a, hipStream_t st);

// ---- rotary positions (rotary.hip) ------------------------------------------------------------------
constexpr int64_t kRotaryMaxPairs = 2048;   // of a head: its cosines and sines are held in LDS

struct RotaryArgs {
  const void* x;
  int64_t ldt, ldh;
  void* y;
  int64_t ldyt, ldyh;
  int64_t T;
  int H, D, pairs;
  const double* freqs;
  const int64_t* positions;   // optional: start + t
  int64_t start;
  float scale;
  bool bf16, interleaved, inverse;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st);

// ---- AdamW (adamw.hip) ------------------------------------------------------------------------------
struct AdamJob {
  void* param;
  float* master;          // optional, of a bf16 param
  const void* grad;
  void* avg;
  void* sq;
  float* avg_scale;       // of 8-bit states
  float* sq_scale;
  int64_t n;
  uint32_t place;         // in the caller's list
  bool param_bf16, grad_bf16;
};
struct AdamHyper {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const float* lr_dev;          // optional, in place of lr
  const int64_t* step_dev;      // optional, in place of step
  const float* norm;            // optional
  float max_norm;
  uint64_t seed;
};
// Jobs of 32-bit states, or (eight) of 8-bit ones.
hipError_t launch_adamw(const AdamJob* jobs, int n_jobs, bool eight, const AdamHyper& h, hipStream_t st);

// ---- gradient norm and clipping (clip.hip) ----------------------------------------------------------
struct GradJob {
  const void* src;
  void* dst;
  int64_t n;
  bool bf16;
};
// Doubles of workspace: one partial sum of squares per workgroup of every launch.
int64_t grad_partials(const GradJob* jobs, int n_jobs);
hipError_t launch_grad_squares(const GradJob* jobs, int n_jobs, double* partials, hipStream_t st);
hipError_t launch_grad_norm(const double* partials, int64_t n_partials, float* norm, hipStream_t st);
// dst = src * min(1, max_norm / (norm + 1e-6)), with the norm from the partials (which is then also
// written to norm_out), or, where partials is NULL, from norm_in.
hipError_t launch_grad_scale(const GradJob* jobs, int n_jobs, const double* partials, int64_t n_partials,
                             const float* norm_in, float* norm_out, float max_norm, hipStream_t st);

// ---- few-row product (gemm_rows.hip) ----------------------------------------------------------------
// (of a bf16 output; an fp32 one needs none)
size_t gemm_rows_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                            const uint8_t* B, int64_t ldb, const float* sB, void* C, int64_t ldc, bool out_bf16,
                            void* workspace, size_t workspace_bytes, hipStream_t st);

}  // namespace puro
