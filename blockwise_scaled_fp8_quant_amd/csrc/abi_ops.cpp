// C-ABI layer of puro_ops.h: argument validation on the host, then asynchronous launches on the
// caller's stream.  Every check runs before any HIP call; a failed check launches nothing.
#include "../../include/puro_ops.h"

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "ops_internal.hpp"
#include "overlap.hpp"

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

// A range of memory that a call writes, or reads.
struct Range {
  uintptr_t lo, hi;
  bool written;
};

// Whether a range that is written overlaps any other: the workgroups of a launch run in no order, so such a call would race.
bool written_overlap(std::vector<Range>& r) {
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_written = 0, end_any = 0;   // furthest end of a written range, and of any, so far
  for (const Range& x : r) {
    if (x.lo < end_written || (x.written && x.lo < end_any)) return true;
    end_any = std::max(end_any, x.hi);
    if (x.written) end_written = std::max(end_written, x.hi);
  }
  return false;
}

// ... for a list of gradients: an output over another job's output, or over an input that is not its own.
bool outputs_overlap(const std::vector<puro::GradJob>& jobs) {
  std::vector<Range> r;
  r.reserve(2 * jobs.size());
  for (const puro::GradJob& j : jobs) {
    const uintptr_t bytes = (uintptr_t)j.n * (j.bf16 ? 2 : 4);
    const uintptr_t d = reinterpret_cast<uintptr_t>(j.dst), s = reinterpret_cast<uintptr_t>(j.src);
    r.push_back(Range{d, d + bytes, true});
    if (s != d) r.push_back(Range{s, s + bytes, false});
  }
  return written_overlap(r);
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

// What the three forward forms of the residual sum check beyond the norm's (`align` as there), and their arguments.
int check_residual(const puro_residual* r, int64_t align, puro::ResidualArgs& a) {
  if (!r) return PURO_ERR_NULLPTR;
  // (the norm is that of h_out: its checks are h_out's too)
  const int rc = check_norm(r->kind, r->x_dtype, r->h_out, r->T, r->C, r->ldh_out, r->w_dtype, r->weight, r->bias, r->eps,
                            r->mean, r->rstd, align);
  if (rc != PURO_OK) return rc;
  if (!std::isfinite(r->scale)) return PURO_ERR_ARG;
  if (r->kind == PURO_NORM_RMS && r->post_mean) return PURO_ERR_ARG;
  if (r->T == 0 || r->C == 0) return PURO_OK;   // (a vector of no columns may be NULL)
  if (!r->post_weight && (r->post_mean || r->post_rstd)) return PURO_ERR_ARG;
  if (!r->h || !r->x) return PURO_ERR_NULLPTR;
  const int64_t es = size_of(r->x_dtype), rows = align ? align : es, vec = align ? align : size_of(r->w_dtype);
  if (!aligned(r->h, rows) || !aligned(r->x, rows) || !aligned(r->gate, vec) || !aligned(r->post_weight, vec) ||
      !aligned(r->post_mean, 4) || !aligned(r->post_rstd, 4))
    return PURO_ERR_ALIGN;
  if (r->ldh < r->C || r->ldx < r->C || (align && ((r->ldh * es) % align || (r->ldx * es) % align))) return PURO_ERR_LD;
  a = {};
  a.n = norm_args(r->kind, r->x_dtype, r->h_out, r->T, r->C, r->ldh_out, r->w_dtype, r->weight, r->bias, r->eps, r->mean,
                  r->rstd);
  a.h = r->h; a.ldh = r->ldh; a.b = r->x; a.ldb = r->ldx;
  a.h_out = r->h_out;
  a.gate = r->gate; a.post = r->post_weight; a.scale = r->scale;
  a.post_mean = r->post_mean; a.post_rstd = r->post_rstd;
  return PURO_OK;
}

// What the forward forms read and write but for the norm: h_out may be h or x, and so may another matrix that replaces.
puro::Tensors residual_tensors(const puro_residual& r) {
  using namespace puro;
  const int64_t es = size_of(r.x_dtype), vec = r.C * size_of(r.w_dtype), stat = r.T * 4;
  Tensors t;
  t.reads(r.h, replacing(matrix(r.h, r.T, r.ldh, r.C, es)));
  t.reads(r.x, replacing(matrix(r.x, r.T, r.ldx, r.C, es)));
  for (const void* p : {r.weight, r.bias, r.gate, r.post_weight}) t.reads(p, vector(p, vec));
  t.writes(r.h_out, replacing(matrix(r.h_out, r.T, r.ldh_out, r.C, es)));
  for (const void* p : {r.mean, r.rstd, r.post_mean, r.post_rstd}) t.writes(p, vector(p, stat));
  return t;
}

// Whether the D-wide heads of [T, H, D] with these strides lie apart from each other.
bool heads_apart(int64_t T, int64_t H, int64_t D, int64_t ld_t, int64_t ld_h) {
  if (T <= 1) return H <= 1 || ld_h >= D;
  if (H <= 1) return ld_t >= D;
  typedef __int128 wide;
  return (ld_h >= D && ld_t >= (wide)(H - 1) * ld_h + D) || (ld_t >= D && ld_h >= (wide)(T - 1) * ld_t + D);
}

// Checks an AdamW job list and translates it (no exception leaves: PURO_ERR_UNSUPPORTED without memory).
int adam_jobs(const puro_adamw_job* jobs, int n_jobs, const puro_adamw_hyper& h, std::vector<puro::AdamJob>& out) {
  if (n_jobs < 0) return PURO_ERR_SHAPE;
  if (n_jobs == 0) return PURO_OK;
  if (!jobs) return PURO_ERR_NULLPTR;
  std::vector<Range> r;
  try {
    out.reserve((size_t)n_jobs);
    r.reserve(7 * (size_t)n_jobs + 3);
  } catch (...) {
    return PURO_ERR_UNSUPPORTED;
  }
  // (the pushes below stay within those reservations)
  auto range = [&](const void* p, uintptr_t bytes, bool written) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p) r.push_back(Range{lo, lo + bytes, written});
  };
  for (int i = 0; i < n_jobs; ++i) {
    const puro_adamw_job& j = jobs[i];
    if (!dtype_ok(j.param_dtype) || !dtype_ok(j.grad_dtype)) return PURO_ERR_DTYPE;
    if (j.n < 0) return PURO_ERR_SHAPE;
    if ((j.avg_scale == nullptr) != (j.sq_scale == nullptr)) return PURO_ERR_ARG;
    if (j.master && j.param_dtype != PURO_OUT_BF16) return PURO_ERR_ARG;
    if (j.n == 0) continue;
    if (!j.param || !j.grad || !j.exp_avg || !j.exp_avg_sq) return PURO_ERR_NULLPTR;
    const bool eight = j.avg_scale != nullptr;
    const int64_t ps = size_of(j.param_dtype), gs = size_of(j.grad_dtype), ss = eight ? 1 : 4;
    if (!aligned(j.param, ps) || !aligned(j.grad, gs) || !aligned(j.exp_avg, ss) || !aligned(j.exp_avg_sq, ss) ||
        !aligned(j.master, 4) || !aligned(j.avg_scale, 4) || !aligned(j.sq_scale, 4))
      return PURO_ERR_ALIGN;
    if (j.n > (int64_t(1) << 42)) return PURO_ERR_UNSUPPORTED;
    const uintptr_t n = (uintptr_t)j.n, blocks = (n + kGroup - 1) / kGroup;
    range(j.param, n * ps, true);
    range(j.master, n * 4, true);
    range(j.grad, n * gs, false);
    range(j.exp_avg, n * ss, true);
    range(j.exp_avg_sq, n * ss, true);
    range(j.avg_scale, blocks * 4, true);
    range(j.sq_scale, blocks * 4, true);
    out.push_back(puro::AdamJob{j.param, j.master, j.grad, j.exp_avg, j.exp_avg_sq, j.avg_scale, j.sq_scale, j.n, (uint32_t)i,
                                j.param_dtype == PURO_OUT_BF16, j.grad_dtype == PURO_OUT_BF16});
  }
  range(h.lr_dev, 4, false);
  range(h.step_dev, 8, false);
  range(h.norm, 4, false);
  return written_overlap(r) ? PURO_ERR_ARG : PURO_OK;
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

int puro_residual_norm(const puro_residual* r, void* y, int64_t ldy, hipStream_t st) {
  puro::ResidualArgs a;
  const int rc = check_residual(r, 0, a);
  if (rc != PURO_OK || r->T == 0 || r->C == 0) return rc;
  if (!y) return PURO_ERR_NULLPTR;
  if (!aligned(y, size_of(r->x_dtype))) return PURO_ERR_ALIGN;
  if (ldy < r->C) return PURO_ERR_LD;
  puro::Tensors t = residual_tensors(*r);
  t.writes(y, puro::replacing(puro::matrix(y, r->T, ldy, r->C, size_of(r->x_dtype))));
  if (t.clash()) return PURO_ERR_ARG;
  a.n.y = y; a.n.ldy = ldy;
  return from_hip(puro::launch_residual(a, st));
}

int puro_residual_norm_quant(const puro_residual* r, uint8_t* q, int64_t ldq, float* s, hipStream_t st) {
  if (r && r->C % kGroup) return PURO_ERR_SHAPE;
  puro::ResidualArgs a;
  const int rc = check_residual(r, 16, a);
  if (rc != PURO_OK || r->T == 0 || r->C == 0) return rc;
  if (!q || !s) return PURO_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(s, 16)) return PURO_ERR_ALIGN;
  if (ldq < r->C || ldq % 16) return PURO_ERR_LD;
  puro::Tensors t = residual_tensors(*r);
  t.writes(q, puro::matrix(q, r->T, ldq, r->C, 1));
  t.writes(s, puro::vector(s, r->C / kGroup * r->T * 4));
  if (t.clash()) return PURO_ERR_ARG;
  a.n.q = q; a.n.ldq = ldq; a.n.s = s;
  return from_hip(puro::launch_residual_quant(a, st));
}

int puro_residual_norm_quant_dual(const puro_residual* r, uint8_t* q, int64_t ldq, float* s, uint8_t* qT, int64_t ldqT,
                                  float* sT, hipStream_t st) {
  if (r && (r->T % kGroup || r->C % kGroup)) return PURO_ERR_SHAPE;
  puro::ResidualArgs a;
  const int rc = check_residual(r, 16, a);
  if (rc != PURO_OK || r->T == 0 || r->C == 0) return rc;
  if (!q || !s || !qT || !sT || !r->rstd || (r->kind == PURO_NORM_LAYER && !r->mean)) return PURO_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(s, 16) || !aligned(qT, 16) || !aligned(sT, 16)) return PURO_ERR_ALIGN;
  if (ldq < r->C || ldq % 16 || ldqT < r->T || ldqT % 16) return PURO_ERR_LD;
  if (too_many_blocks(r->T / kGroup, r->C / kGroup)) return PURO_ERR_UNSUPPORTED;
  puro::Tensors t = residual_tensors(*r);
  t.writes(q, puro::matrix(q, r->T, ldq, r->C, 1));
  t.writes(s, puro::vector(s, r->C / kGroup * r->T * 4));
  t.writes(qT, puro::matrix(qT, r->C, ldqT, r->T, 1));
  t.writes(sT, puro::vector(sT, r->T / kGroup * r->C * 4));
  if (t.clash()) return PURO_ERR_ARG;
  a.n.q = q; a.n.ldq = ldq; a.n.s = s;
  a.n.qT = qT; a.n.ldqT = ldqT; a.n.sT = sT;
  return from_hip(puro::launch_residual_quant_dual(a, st));
}

size_t puro_residual_norm_backward_workspace_size(int64_t T, int64_t C, int gated) {
  if (T <= 0 || C <= 0 || C > puro::kNormMaxC) return 0;
  const int blocks = puro::residual_bwd_blocks(T, C, gated != 0);
  return blocks <= 1 ? 0 : (size_t)blocks * puro::residual_bwd_sums(gated != 0) * (size_t)C * 4;
}

int puro_residual_norm_backward(const puro_residual_grad* r, void* workspace, size_t workspace_bytes, hipStream_t st) {
  if (!r) return PURO_ERR_NULLPTR;
  const bool layer = r->kind == PURO_NORM_LAYER, gated = r->gate || r->post_weight;
  if (!layer && r->kind != PURO_NORM_RMS) return PURO_ERR_MODE;
  if (!dtype_ok(r->x_dtype) || !dtype_ok(r->w_dtype)) return PURO_ERR_DTYPE;
  if (r->T < 0 || r->C < 0) return PURO_ERR_SHAPE;
  if (r->accumulate != 0 && r->accumulate != 1) return PURO_ERR_ARG;
  if (!layer && (r->mean || r->post_mean)) return PURO_ERR_ARG;
  if (!std::isfinite(r->scale)) return PURO_ERR_ARG;
  if (r->C == 0) return PURO_OK;                // (a vector of no columns may be NULL)
  if (!r->post_weight && (r->post_mean || r->post_rstd || r->dpost_weight)) return PURO_ERR_ARG;
  if (!r->gate && r->dgate) return PURO_ERR_ARG;
  if (!r->dweight) return PURO_ERR_NULLPTR;
  if (!aligned(r->dweight, 4) || !aligned(r->dbias, 4) || !aligned(r->dgate, 4) || !aligned(r->dpost_weight, 4))
    return PURO_ERR_ALIGN;
  if (r->C > puro::kNormMaxC) return PURO_ERR_UNSUPPORTED;
  if (r->T > 0) {
    if (!r->dy || !r->h_out || !r->weight || !r->rstd || !r->dh || (layer && !r->mean)) return PURO_ERR_NULLPTR;
    if (gated && (!r->x || !r->dx)) return PURO_ERR_NULLPTR;
    if (r->post_weight && (!r->post_rstd || (layer && !r->post_mean))) return PURO_ERR_NULLPTR;
    const int64_t es = size_of(r->x_dtype), ws = size_of(r->w_dtype);
    if (!aligned(r->dy, es) || !aligned(r->h_out, es) || !aligned(r->dh_out, es) || !aligned(r->dh, es) ||
        !aligned(r->dx, es) || (gated && !aligned(r->x, es)) || !aligned(r->weight, ws) || !aligned(r->gate, ws) ||
        !aligned(r->post_weight, ws) || !aligned(r->mean, 4) || !aligned(r->rstd, 4) || !aligned(r->post_mean, 4) ||
        !aligned(r->post_rstd, 4))
      return PURO_ERR_ALIGN;
    if (r->lddy < r->C || r->ldh_out < r->C || r->lddh < r->C || (r->dh_out && r->lddh_out < r->C) ||
        (gated && r->ldx < r->C) || (r->dx && r->lddx < r->C))
      return PURO_ERR_LD;
    const size_t need = puro_residual_norm_backward_workspace_size(r->T, r->C, gated);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PURO_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return PURO_ERR_ALIGN;
    using namespace puro;
    Tensors t;
    t.reads(r->dy, replacing(matrix(r->dy, r->T, r->lddy, r->C, es)));
    t.reads(r->h_out, replacing(matrix(r->h_out, r->T, r->ldh_out, r->C, es)));
    t.reads(r->dh_out, replacing(matrix(r->dh_out, r->T, r->lddh_out, r->C, es)));
    if (gated) t.reads(r->x, replacing(matrix(r->x, r->T, r->ldx, r->C, es)));
    for (const void* p : {r->weight, r->gate, r->post_weight}) t.reads(p, vector(p, r->C * ws));
    for (const void* p : {r->mean, r->rstd, r->post_mean, r->post_rstd}) t.reads(p, vector(p, r->T * 4));
    t.writes(r->dh, replacing(matrix(r->dh, r->T, r->lddh, r->C, es)));
    t.writes(r->dx, replacing(matrix(r->dx, r->T, r->lddx, r->C, es)));
    for (const void* p : {r->dweight, r->dbias, r->dgate, r->dpost_weight}) t.writes(p, vector(p, r->C * 4));
    if (need > 0) t.writes(workspace, vector(workspace, need));
    if (t.clash()) return PURO_ERR_ARG;
  }
  puro::ResidualBwdArgs a = {};
  a.dy = r->dy; a.lddy = r->lddy; a.h = r->h_out; a.ldh = r->ldh_out; a.dho = r->dh_out; a.lddho = r->lddh_out;
  a.b = gated ? r->x : nullptr; a.ldb = r->ldx;
  a.T = r->T; a.C = (int)r->C;
  a.gamma = r->weight; a.gate = r->gate; a.post = r->post_weight; a.scale = r->scale;
  a.x_bf16 = r->x_dtype == PURO_OUT_BF16; a.w_bf16 = r->w_dtype == PURO_OUT_BF16; a.layer = layer;
  a.mean = r->mean; a.rstd = r->rstd; a.post_mean = r->post_mean; a.post_rstd = r->post_rstd;
  a.dh = r->dh; a.lddh = r->lddh; a.dx = r->dx; a.lddx = r->lddx;
  a.dgamma = r->dweight; a.dbeta = r->dbias; a.dgate = r->dgate; a.dpost = r->dpost_weight;
  a.accumulate = r->accumulate;
  a.partial = static_cast<float*>(workspace);
  return from_hip(puro::launch_residual_bwd(a, st));
}

int puro_rotary(int x_dtype, int layout, int inverse, const void* x, int64_t ld_t, int64_t ld_h, int64_t T, int64_t H,
                int64_t D, const int64_t* positions, int64_t start, const double* freqs, int64_t pairs, float scale, void* y,
                int64_t ldy_t, int64_t ldy_h, hipStream_t st) {
  if (layout != PURO_ROTARY_HALF && layout != PURO_ROTARY_INTERLEAVED) return PURO_ERR_MODE;
  if (!dtype_ok(x_dtype)) return PURO_ERR_DTYPE;
  if (T < 0 || H < 0 || D < 0 || pairs < 0 || pairs > D / 2) return PURO_ERR_SHAPE;
  if ((inverse != 0 && inverse != 1) || !std::isfinite(scale)) return PURO_ERR_ARG;
  if (T == 0 || H == 0 || D == 0) return PURO_OK;
  if (!x || !y || (pairs > 0 && !freqs)) return PURO_ERR_NULLPTR;
  const int64_t es = size_of(x_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(freqs, 8) || !aligned(positions, 8)) return PURO_ERR_ALIGN;
  if (ld_t < 0 || ld_h < 0 || !heads_apart(T, H, D, ldy_t, ldy_h)) return PURO_ERR_LD;
  if (T > kIntMax || H > kIntMax || D > (int64_t(1) << 30) || pairs > puro::kRotaryMaxPairs) return PURO_ERR_UNSUPPORTED;
  puro::Tensors t;
  const bool tokens_first = H <= 1 || T <= 1 || ldy_t >= ldy_h;      // (heads_apart: the longer stride is the outer one)
  auto heads = [&](const void* p, int64_t ldt, int64_t ldh) {
    puro::Rows r = puro::matrix(p, tokens_first ? T : H, tokens_first ? ldt : ldh, D, es);
    r.rows = tokens_first ? H : T;
    r.ld_row = (puro::Rows::wide)(tokens_first ? ldh : ldt) * es;
    return puro::replacing(r);
  };
  t.reads(x, heads(x, ld_t, ld_h));
  t.reads(positions, puro::vector(positions, T * 8));
  t.reads(freqs, puro::vector(freqs, pairs * 8));
  t.writes(y, heads(y, ldy_t, ldy_h));
  if (t.clash()) return PURO_ERR_ARG;
  puro::RotaryArgs a = {};
  a.x = x; a.ldt = ld_t; a.ldh = ld_h;
  a.y = y; a.ldyt = ldy_t; a.ldyh = ldy_h;
  a.T = T; a.H = (int)H; a.D = (int)D; a.pairs = (int)pairs;
  a.freqs = freqs; a.positions = positions; a.start = start; a.scale = scale;
  a.bf16 = x_dtype == PURO_OUT_BF16; a.interleaved = layout == PURO_ROTARY_INTERLEAVED; a.inverse = inverse != 0;
  return from_hip(puro::launch_rotary(a, st));
}

int puro_adamw(const puro_adamw_job* jobs, int n_jobs, const puro_adamw_hyper* h, hipStream_t st) {
  if (!h) return PURO_ERR_NULLPTR;
  auto fraction = [](double v) { return v >= 0.0 && v < 1.0; };
  if (!std::isfinite(h->lr) || !fraction(h->beta1) || !fraction(h->beta2) || !(h->eps >= 0.0) || std::isinf(h->eps) ||
      !std::isfinite(h->weight_decay) || (!h->step_dev && h->step < 1) || (h->norm && !(h->max_norm >= 0.f)))
    return PURO_ERR_ARG;
  if (!aligned(h->lr_dev, 4) || !aligned(h->step_dev, 8) || !aligned(h->norm, 4)) return PURO_ERR_ALIGN;
  std::vector<puro::AdamJob> b;
  const int rc = adam_jobs(jobs, n_jobs, *h, b);
  if (rc != PURO_OK) return rc;
  const puro::AdamHyper a = {h->lr, h->beta1, h->beta2, h->eps, h->weight_decay, h->step, h->lr_dev, h->step_dev, h->norm,
                             h->max_norm, h->seed};
  hipError_t e = puro::launch_adamw(b.data(), (int)b.size(), false, a, st);
  if (e == hipSuccess) e = puro::launch_adamw(b.data(), (int)b.size(), true, a, st);
  return from_hip(e);
}

}  // extern "C"
