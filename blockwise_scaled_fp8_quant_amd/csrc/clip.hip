// gfx950 global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over tensors and elements of g^2);  c = min(1, max_norm / (norm + 1e-6));  out = g c
//
// Two passes over the gradients, both bound by HBM: the first reads every element once and leaves one
// partial sum of squares per workgroup, the second reads again and writes.  The tensors are described
// in the kernel's arguments (kMaxJobs per launch): no table is copied to the device, so a captured
// graph holds it.  Squares are formed and summed in 64 bits -- the product of two fp32 values is exact
// there and cannot overflow or vanish -- at a cost that a stream does not notice (one conversion and
// one fp64 FMA per element).  Every workgroup of the second pass adds the partials itself, in the same
// order, so no third launch stands between the passes and no atomic is needed.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"

#include <algorithm>

namespace puro {

namespace {

constexpr int kMaxJobs = 112;              // 112 * 32 + 128 bytes: inside the 4 KB of kernel arguments
constexpr int kThreads = 256;
// 16-byte loads a thread has in flight, and workgroups of a launch (8 per CU).  Measured on 1.6 GB of fp32
// gradients, norm + scaling: 252 + 566 us.  With 8 loads the scaling takes 627 us, with 1024 workgroups 577, with
// 512 742; past-the-cache loads take 23 us off the norm and put 18 to 30 on the scaling.
constexpr int kVecs = 4;
constexpr int kMaxBlocks = 2048;

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

struct JobDesc {
  const uint8_t* src;
  uint8_t* dst;
  int64_t n;          // elements
  uint32_t first;     // first chunk of the job in the launch
  uint32_t bf16;
};
struct JobTable {
  JobDesc job[kMaxJobs];
  int n_jobs;
  uint32_t chunks;    // of the launch
};
static_assert(sizeof(JobTable) + 64 <= 4096, "kernel arguments exceed 4 KB");

// A tensor's 16-byte vectors are those of its address rounded down to 16 bytes: vector v of a job holds
// the elements [v * per - off, ...) with off = elements between that address and the first one.
__host__ __device__ inline int64_t job_vecs(const void* src, int64_t n, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(src) & 15u);
  return (off + n * es + 15) / 16;
}

// chunk -> job: the last job whose first chunk is not behind it (uniform over the workgroup)
__device__ __forceinline__ int find_job(const JobTable& t, uint32_t chunk) {
  int lo = 0, hi = t.n_jobs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.job[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The part of vector v that belongs to the tensor: elements [lo, hi) of the vector's `per`.
struct Part {
  int64_t first;   // element of the tensor that the vector's element 0 is (negative before its start)
  int lo, hi;
};
__device__ __forceinline__ Part part_of(int64_t v, int per, int off, int64_t n) {
  Part p;
  p.first = v * per - off;
  p.lo = p.first < 0 ? (int)-p.first : 0;
  const int64_t left = n - p.first;
  p.hi = left < per ? (int)(left < 0 ? 0 : left) : per;
  return p;
}

template <typename T>
__device__ __forceinline__ T ld_elem(const uint8_t* base, int64_t i) {
  return reinterpret_cast<const T*>(base)[i];
}

__device__ __forceinline__ u32x4 load_part(const JobDesc& j, const Part& p, int per) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if (p.lo == 0 && p.hi == per) {
    w = *reinterpret_cast<const u32x4*>(j.src + p.first * (16 / per));
  } else {
    for (int e = p.lo; e < p.hi; ++e) {
      if (per == 8) {
        const uint32_t h = ld_elem<uint16_t>(j.src, p.first + e);
        const uint32_t x = h << (16 * (e & 1));
        if ((e >> 1) == 0) w.x |= x; else if ((e >> 1) == 1) w.y |= x; else if ((e >> 1) == 2) w.z |= x; else w.w |= x;
      } else {
        const uint32_t x = ld_elem<uint32_t>(j.src, p.first + e);
        if (e == 0) w.x = x; else if (e == 1) w.y = x; else if (e == 2) w.z = x; else w.w = x;
      }
    }
  }
  return w;
}

__device__ __forceinline__ double sq(float v, double acc) {
  const double d = (double)v;
  return __builtin_fma(d, d, acc);
}

// sum over the workgroup, in every thread (fixed order)
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

__global__ __launch_bounds__(kThreads) void grad_squares_kernel(JobTable t, double* __restrict__ partials) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const JobDesc j = t.job[find_job(t, c)];
    const int per = j.bf16 ? 8 : 4;
    const int off = (int)(reinterpret_cast<uintptr_t>(j.src) & 15u) / (16 / per);
    const int64_t v0 = (int64_t)(c - j.first) * (kThreads * kVecs) + threadIdx.x;
    u32x4 w[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) w[k] = load_part(j, part_of(v0 + k * kThreads, per, off, j.n), per);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if (j.bf16) {
          acc = sq(bf16_lo(w[k][d]), acc);
          acc = sq(bf16_hi(w[k][d]), acc);
        } else {
          acc = sq(__uint_as_float(w[k][d]), acc);
        }
      }
  }
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) partials[blockIdx.x] = acc;
}

__device__ __forceinline__ float norm_of(const double* __restrict__ partials, int64_t n, double* red) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) s += partials[i];
  return (float)__builtin_sqrt(block_sum(s, red));
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* __restrict__ partials, int64_t n, float* norm) {
  __shared__ double red[kThreads / 64];
  const float v = norm_of(partials, n, red);
  if (threadIdx.x == 0) *norm = v;
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(JobTable t, const double* __restrict__ partials,
                                                              int64_t n_partials, const float* norm_in,
                                                              float* norm_out, float max_norm) {
  __shared__ double red[kThreads / 64];
  const float norm = partials ? norm_of(partials, n_partials, red) : *norm_in;
  if (partials && norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  float coef = max_norm / (norm + 1e-6f);
  coef = coef > 1.0f ? 1.0f : coef;        // a NaN stays
  const bool unclipped = coef == 1.0f;
  // From the last chunk to the first: what the first pass read last may still be in the memory-side cache.
  for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const uint32_t c = t.chunks - 1 - i;
    const JobDesc j = t.job[find_job(t, c)];
    if (unclipped && j.dst == j.src) continue;
    const int per = j.bf16 ? 8 : 4, es = 16 / per;
    const int off = (int)(reinterpret_cast<uintptr_t>(j.src) & 15u) / es;
    const bool same = ((reinterpret_cast<uintptr_t>(j.src) ^ reinterpret_cast<uintptr_t>(j.dst)) & 15u) == 0;
    const int64_t v0 = (int64_t)(c - j.first) * (kThreads * kVecs) + threadIdx.x;
    u32x4 w[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) w[k] = load_part(j, part_of(v0 + k * kThreads, per, off, j.n), per);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const Part p = part_of(v0 + k * kThreads, per, off, j.n);
      u32x4 o;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[d] = j.bf16 ? bf16x2_rne(bf16_lo(w[k][d]) * coef, bf16_hi(w[k][d]) * coef)
                      : __float_as_uint(__uint_as_float(w[k][d]) * coef);
      if (p.lo == 0 && p.hi == per) {
        uint8_t* d = j.dst + p.first * es;
        if (same)
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(d));
        else   // whole vectors of the input at another alignment: global stores need the element's alone
          *reinterpret_cast<u32x4_a2*>(d) = o;
      } else {
        for (int e = p.lo; e < p.hi; ++e) {
          const int d = per == 8 ? e >> 1 : e;
          const uint32_t x = d == 0 ? o.x : d == 1 ? o.y : d == 2 ? o.z : o.w;
          if (per == 8) reinterpret_cast<uint16_t*>(j.dst)[p.first + e] = (uint16_t)(x >> (16 * (e & 1)));
          else reinterpret_cast<uint32_t*>(j.dst)[p.first + e] = x;
        }
      }
    }
  }
}

// The launches of a list of jobs: up to kMaxJobs non-empty tensors each.  f(table, blocks) launches one.
template <typename F>
hipError_t for_each_launch(const GradJob* jobs, int n_jobs, F f) {
  JobTable t;
  t.n_jobs = 0;
  t.chunks = 0;
  auto flush = [&]() -> hipError_t {
    if (t.n_jobs == 0) return hipSuccess;
    const hipError_t e = f(t, (int)std::min<uint32_t>(t.chunks, kMaxBlocks));
    t.n_jobs = 0;
    t.chunks = 0;
    return e;
  };
  for (int i = 0; i < n_jobs; ++i) {
    if (jobs[i].n == 0) continue;
    const int64_t vecs = job_vecs(jobs[i].src, jobs[i].n, jobs[i].bf16);
    const int64_t chunks = (vecs + kThreads * kVecs - 1) / (kThreads * kVecs);
    if (t.n_jobs == kMaxJobs || (int64_t)t.chunks + chunks > 0x7FFFFFFF) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    t.job[t.n_jobs++] = JobDesc{static_cast<const uint8_t*>(jobs[i].src), static_cast<uint8_t*>(jobs[i].dst), jobs[i].n,
                                t.chunks, jobs[i].bf16 ? 1u : 0u};
    t.chunks += (uint32_t)chunks;
  }
  return flush();
}

}  // namespace

int64_t grad_partials(const GradJob* jobs, int n_jobs) {
  int64_t total = 0;
  (void)for_each_launch(jobs, n_jobs, [&](const JobTable&, int blocks) {
    total += blocks;
    return hipSuccess;
  });
  return total;
}

hipError_t launch_grad_squares(const GradJob* jobs, int n_jobs, double* partials, hipStream_t st) {
  return for_each_launch(jobs, n_jobs, [&](const JobTable& t, int blocks) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3(blocks), dim3(kThreads), 0, st, t, partials);
    partials += blocks;
    return hipGetLastError();
  });
}

hipError_t launch_grad_norm(const double* partials, int64_t n_partials, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, st, partials, n_partials, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradJob* jobs, int n_jobs, const double* partials, int64_t n_partials,
                             const float* norm_in, float* norm_out, float max_norm, hipStream_t st) {
  return for_each_launch(jobs, n_jobs, [&](const JobTable& t, int blocks) {
    hipLaunchKernelGGL(grad_scale_kernel, dim3(blocks), dim3(kThreads), 0, st, t, partials, n_partials, norm_in,
                       norm_out, max_norm);
    norm_out = nullptr;
    return hipGetLastError();
  });
}

}  // namespace puro
