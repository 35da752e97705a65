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
