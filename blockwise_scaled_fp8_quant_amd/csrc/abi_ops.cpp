// C-ABI layer of puro_ops.h: argument validation on the host, then asynchronous launches on the
// caller's stream.  Every check runs before any HIP call; a failed check launches nothing.
#include "../../include/puro_ops.h"

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "ops_internal.hpp"

namespace {

constexpr int64_t kGroup = 128;
constexpr int64_t kIntMax = 0x7FFFFFFF;
constexpr int64_t kMaxGemmLd = int64_t(1) << 29;   // as puro_fp8_gemm: leading rows may run its kernels

inline bool aligned(const void* p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0; }
inline bool dtype_ok(int d) { return d == PURO_OUT_BF16 || d == PURO_OUT_FP32; }
inline int64_t size_of(int d) { return d == PURO_OUT_BF16 ? 2 : 4; }
inline bool too_many_blocks(int64_t a, int64_t b) { return a > 0 && b > kIntMax / a; }

inline int from_hip(hipError_t e) {
  if (e == hipErrorInvalidConfiguration) return PURO_ERR_UNSUPPORTED;
  return e == hipSuccess ? PURO_OK : PURO_ERR_HIP;
}

// What the three forward forms check alike (x, weight, bias, statistics).  `align`: bytes the rows of
// x have to be aligned to (0: those of an element).
int check_norm(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype, const void* weight,
               const void* bias, float eps, const float* mean, const float* rstd, int64_t align) {
  if (kind != PURO_NORM_LAYER && kind != PURO_NORM_RMS) return PURO_ERR_MODE;
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return PURO_ERR_DTYPE;
  if (T < 0 || C < 0) return PURO_ERR_SHAPE;
  if (!(eps >= 0.f) || std::isinf(eps)) return PURO_ERR_ARG;
  if (kind == PURO_NORM_RMS && mean) return PURO_ERR_ARG;
  if (T == 0 || C == 0) return PURO_OK;
  if (!x || !weight) return PURO_ERR_NULLPTR;
  const int64_t es = size_of(x_dtype), ws = size_of(w_dtype);
  if (!aligned(x, align ? align : es) || !aligned(weight, align ? align : ws) || !aligned(bias, align ? align : ws) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return PURO_ERR_ALIGN;
  if (ldx < C || (align && (ldx * es) % align)) return PURO_ERR_LD;
  if (C > puro::kNormMaxC) return PURO_ERR_UNSUPPORTED;
  return PURO_OK;
}

puro::NormArgs norm_args(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                         const void* weight, const void* bias, float eps, float* mean, float* rstd) {
  puro::NormArgs a = {};
  a.x = x; a.ldx = ldx; a.T = T; a.C = (int)C;
  a.gamma = weight; a.beta = bias;
  a.x_bf16 = x_dtype == PURO_OUT_BF16; a.w_bf16 = w_dtype == PURO_OUT_BF16;
  a.layer = kind == PURO_NORM_LAYER; a.eps = eps;
  a.mean = mean; a.rstd = rstd;
  return a;
}

// Whether a tensor's output range overlaps another job's output, or another job's input that is not its
// own output's: the workgroups of a launch run in no order, so such a call would race.
bool outputs_overlap(const std::vector<puro::GradJob>& jobs) {
  struct Range {
    uintptr_t lo, hi;
    size_t job;
    bool dst;
  };
  std::vector<Range> r;
  r.reserve(2 * jobs.size());
  for (size_t i = 0; i < jobs.size(); ++i) {
    const uintptr_t bytes = (uintptr_t)jobs[i].n * (jobs[i].bf16 ? 2 : 4);
    const uintptr_t d = reinterpret_cast<uintptr_t>(jobs[i].dst), s = reinterpret_cast<uintptr_t>(jobs[i].src);
    r.push_back(Range{d, d + bytes, i, true});
    if (s != d) r.push_back(Range{s, s + bytes, i, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_dst = 0, end_any = 0;   // furthest end of an output, and of any range, so far
  for (const Range& x : r) {
    if (x.lo < end_dst || (x.dst && x.lo < end_any)) return true;
    end_any = std::max(end_any, x.hi);
    if (x.dst) end_dst = std::max(end_dst, x.hi);
  }
  return false;
}

inline bool overlap(const void* a, uintptr_t a_bytes, const void* b, uintptr_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Whether [p, p + bytes) shares memory with a tensor of the jobs: such a norm or workspace would be written while
// other workgroups still read the tensor, or read while they write it.
bool in_tensors(const std::vector<puro::GradJob>& jobs, const void* p, uintptr_t bytes) {
  for (const puro::GradJob& j : jobs) {
    const uintptr_t n = (uintptr_t)j.n * (j.bf16 ? 2 : 4);
    if (overlap(p, bytes, j.src, n) || (j.dst && overlap(p, bytes, j.dst, n))) return true;
  }
  return false;
}

// Checks a job list and translates it (no exception leaves: PURO_ERR_UNSUPPORTED without memory).
int grad_jobs(const puro_grad_job* jobs, int n_jobs, bool with_dst, std::vector<puro::GradJob>& out) {
  if (n_jobs < 0) return PURO_ERR_SHAPE;
  if (n_jobs == 0) return PURO_OK;
  if (!jobs) return PURO_ERR_NULLPTR;
  try {
    out.reserve((size_t)n_jobs);
  } catch (...) {
    return PURO_ERR_UNSUPPORTED;
  }
  // (the pushes below stay within that reservation)
  for (int i = 0; i < n_jobs; ++i) {
    const puro_grad_job& j = jobs[i];
    if (!dtype_ok(j.dtype)) return PURO_ERR_DTYPE;
    if (j.n < 0) return PURO_ERR_SHAPE;
    if (j.n == 0) continue;
    if (!j.src || (with_dst && !j.dst)) return PURO_ERR_NULLPTR;
    const int64_t es = size_of(j.dtype);
    if (!aligned(j.src, es) || (with_dst && !aligned(j.dst, es))) return PURO_ERR_ALIGN;
    if (j.n > (int64_t(1) << 42)) return PURO_ERR_UNSUPPORTED;
    out.push_back(puro::GradJob{j.src, with_dst ? j.dst : nullptr, j.n, j.dtype == PURO_OUT_BF16});
  }
  if (with_dst) {
    try {
      if (outputs_overlap(out)) return PURO_ERR_ARG;
    } catch (...) {
      return PURO_ERR_UNSUPPORTED;
    }
  }
  return PURO_OK;
}

}  // namespace

extern "C" {

int puro_layer_norm(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                    const void* weight, const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                    hipStream_t st) {
  const int rc = check_norm(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd, 0);
  if (rc != PURO_OK || T == 0 || C == 0) return rc;
  if (!y) return PURO_ERR_NULLPTR;
  if (!aligned(y, size_of(x_dtype))) return PURO_ERR_ALIGN;
  if (ldy < C) return PURO_ERR_LD;
  puro::NormArgs a = norm_args(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd);
  a.y = y; a.ldy = ldy;
  return from_hip(puro::launch_norm(a, st));
}

int puro_layer_norm_quant(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                          const void* weight, const void* bias, float eps, uint8_t* q, int64_t ldq, float* s,
                          float* mean, float* rstd, hipStream_t st) {
  if (C % kGroup) return PURO_ERR_SHAPE;
  const int rc = check_norm(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd, 16);
  if (rc != PURO_OK || T == 0 || C == 0) return rc;
  if (!q || !s) return PURO_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(s, 16)) return PURO_ERR_ALIGN;
  if (ldq < C || ldq % 16) return PURO_ERR_LD;
  puro::NormArgs a = norm_args(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd);
  a.q = q; a.ldq = ldq; a.s = s;
  return from_hip(puro::launch_norm_quant(a, st));
}

int puro_layer_norm_quant_dual(int kind, int x_dtype, const void* x, int64_t T, int64_t C, int64_t ldx, int w_dtype,
                               const void* weight, const void* bias, float eps, uint8_t* q, int64_t ldq, float* s,
                               uint8_t* qT, int64_t ldqT, float* sT, float* mean, float* rstd, hipStream_t st) {
  if (T % kGroup || C % kGroup) return PURO_ERR_SHAPE;
  const int rc = check_norm(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd, 16);
  if (rc != PURO_OK || T == 0 || C == 0) return rc;
  if (!q || !s || !qT || !sT || !rstd || (kind == PURO_NORM_LAYER && !mean)) return PURO_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(s, 16) || !aligned(qT, 16) || !aligned(sT, 16)) return PURO_ERR_ALIGN;
  if (ldq < C || ldq % 16 || ldqT < T || ldqT % 16) return PURO_ERR_LD;
  if (too_many_blocks(T / kGroup, C / kGroup)) return PURO_ERR_UNSUPPORTED;
  puro::NormArgs a = norm_args(kind, x_dtype, x, T, C, ldx, w_dtype, weight, bias, eps, mean, rstd);
  a.q = q; a.ldq = ldq; a.s = s;
  a.qT = qT; a.ldqT = ldqT; a.sT = sT;
  return from_hip(puro::launch_norm_quant_dual(a, st));
}

size_t puro_layer_norm_backward_workspace_size(int64_t T, int64_t C) {
  if (T <= 0 || C <= 0 || C > puro::kNormMaxC) return 0;
  const int blocks = puro::norm_bwd_blocks(T, C);
  return blocks <= 1 ? 0 : (size_t)blocks * 2 * (size_t)C * 4;
}

int puro_layer_norm_backward(int kind, int x_dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t T,
                             int64_t C, int w_dtype, const void* weight, const float* mean, const float* rstd, void* dx,
                             int64_t lddx, float* dweight, float* dbias, int accumulate, void* workspace,
                             size_t workspace_bytes, hipStream_t st) {
  if (kind != PURO_NORM_LAYER && kind != PURO_NORM_RMS) return PURO_ERR_MODE;
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return PURO_ERR_DTYPE;
  if (T < 0 || C < 0) return PURO_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return PURO_ERR_ARG;
  if (kind == PURO_NORM_RMS && mean) return PURO_ERR_ARG;
  if (C == 0) return PURO_OK;
  if (!dweight) return PURO_ERR_NULLPTR;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return PURO_ERR_ALIGN;
  if (C > puro::kNormMaxC) return PURO_ERR_UNSUPPORTED;
  if (T > 0) {
    if (!dy || !x || !weight || !rstd || !dx || (kind == PURO_NORM_LAYER && !mean)) return PURO_ERR_NULLPTR;
    const int64_t es = size_of(x_dtype);
    if (!aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) || !aligned(weight, size_of(w_dtype)) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
      return PURO_ERR_ALIGN;
    if (lddy < C || ldx < C || lddx < C) return PURO_ERR_LD;
    const size_t need = puro_layer_norm_backward_workspace_size(T, C);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PURO_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return PURO_ERR_ALIGN;
    if (T / 256 > kIntMax) return PURO_ERR_UNSUPPORTED;
  }
  puro::NormBwdArgs a = {};
  a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx; a.T = T; a.C = (int)C;
  a.gamma = weight;
  a.x_bf16 = x_dtype == PURO_OUT_BF16; a.w_bf16 = w_dtype == PURO_OUT_BF16;
  a.layer = kind == PURO_NORM_LAYER;
  a.mean = mean; a.rstd = rstd; a.dx = dx; a.lddx = lddx;
  a.dgamma = dweight; a.dbeta = dbias; a.accumulate = accumulate;
  a.partial = static_cast<float*>(workspace);
  return from_hip(puro::launch_norm_bwd(a, st));
}

size_t puro_grad_norm_workspace_size(const puro_grad_job* jobs, int n_jobs) {
  std::vector<puro::GradJob> b;
  if (grad_jobs(jobs, n_jobs, false, b) != PURO_OK) return 0;
  return (size_t)puro::grad_partials(b.data(), (int)b.size()) * sizeof(double);
}

static int grad_common(const puro_grad_job* jobs, int n_jobs, bool clip, float max_norm, float* norm, void* workspace,
                       size_t workspace_bytes, hipStream_t st) {
  if (clip && !(max_norm >= 0.f)) return PURO_ERR_ARG;
  std::vector<puro::GradJob> b;
  const int rc = grad_jobs(jobs, n_jobs, clip, b);
  if (rc != PURO_OK) return rc;
  if (!norm) return PURO_ERR_NULLPTR;
  if (!aligned(norm, 4)) return PURO_ERR_ALIGN;
  const int n = (int)b.size();
  const int64_t parts = puro::grad_partials(b.data(), n);
  if (parts > 0 && (workspace == nullptr || workspace_bytes < (size_t)parts * sizeof(double))) return PURO_ERR_WORKSPACE;
  if (parts > 0 && !aligned(workspace, 16)) return PURO_ERR_ALIGN;
  if (clip && in_tensors(b, norm, sizeof(float))) return PURO_ERR_ARG;
  if (parts > 0 && in_tensors(b, workspace, (uintptr_t)parts * sizeof(double))) return PURO_ERR_ARG;
  // (the scaling's first workgroup writes the norm while others read the partial sums; the norm alone is written
  // by the one workgroup that has read them)
  if (clip && overlap(norm, sizeof(float), workspace, (uintptr_t)parts * sizeof(double))) return PURO_ERR_ARG;
  double* w = static_cast<double*>(workspace);
  hipError_t e = puro::launch_grad_squares(b.data(), n, w, st);
  if (e != hipSuccess) return from_hip(e);
  if (!clip || n == 0) return from_hip(puro::launch_grad_norm(w, parts, norm, st));
  return from_hip(puro::launch_grad_scale(b.data(), n, w, parts, nullptr, norm, max_norm, st));
}

int puro_grad_norm(const puro_grad_job* jobs, int n_jobs, float* norm, void* workspace, size_t workspace_bytes,
                   hipStream_t st) {
  return grad_common(jobs, n_jobs, false, 0.f, norm, workspace, workspace_bytes, st);
}

int puro_clip_grad_norm(const puro_grad_job* jobs, int n_jobs, float max_norm, float* norm, void* workspace,
                        size_t workspace_bytes, hipStream_t st) {
  return grad_common(jobs, n_jobs, true, max_norm, norm, workspace, workspace_bytes, st);
}

int puro_scale_by_norm(const puro_grad_job* jobs, int n_jobs, float max_norm, const float* norm, hipStream_t st) {
  if (!(max_norm >= 0.f)) return PURO_ERR_ARG;
  std::vector<puro::GradJob> b;
  const int rc = grad_jobs(jobs, n_jobs, true, b);
  if (rc != PURO_OK) return rc;
  if (!norm) return PURO_ERR_NULLPTR;
  if (!aligned(norm, 4)) return PURO_ERR_ALIGN;
  if (in_tensors(b, norm, sizeof(float))) return PURO_ERR_ARG;
  return from_hip(puro::launch_grad_scale(b.data(), (int)b.size(), nullptr, 0, norm, nullptr, max_norm, st));
}

size_t puro_gemm_rows_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return puro::gemm_rows_workspace_bytes(M, N, K);
}

int puro_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B,
                   int64_t ldb, const float* sB, void* C, int64_t ldc, int out_dtype, void* workspace,
                   size_t workspace_bytes, hipStream_t st) {
  if (!dtype_ok(out_dtype)) return PURO_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0) return PURO_ERR_SHAPE;
  if (N % kGroup || K % kGroup) return PURO_ERR_SHAPE;
  if (M == 0 || N == 0) return PURO_OK;
  if (!C) return PURO_ERR_NULLPTR;
  if (!aligned(C, 16)) return PURO_ERR_ALIGN;
  if (ldc < N || (ldc * size_of(out_dtype)) % 16) return PURO_ERR_LD;
  if (K > 0) {
    if (!A || !B || !sA || !sB) return PURO_ERR_NULLPTR;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 4) || !aligned(sB, 4)) return PURO_ERR_ALIGN;
    if (lda < K || ldb < K || lda % 16 || ldb % 16) return PURO_ERR_LD;
  }
  // (a launch counts its threads, 8 to a column, in 32 bits)
  if (M > kIntMax || N > kIntMax / 4 || K > kIntMax) return PURO_ERR_UNSUPPORTED;
  if (K > 0 && (lda > kMaxGemmLd || ldb > kMaxGemmLd)) return PURO_ERR_UNSUPPORTED;
  const size_t need = out_dtype == PURO_OUT_BF16 ? puro_gemm_rows_workspace_size(M, N, K) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PURO_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return PURO_ERR_ALIGN;
  return from_hip(puro::launch_gemm_rows(M, N, K, A, lda, sA, B, ldb, sB, C, ldc, out_dtype == PURO_OUT_BF16, workspace,
                                         workspace_bytes, st));
}

}  // extern "C"
