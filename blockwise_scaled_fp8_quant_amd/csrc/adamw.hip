// gfx950 AdamW step over many tensors at once, with fp32 states or 8-bit ones, and the clipping of the gradients folded in.
//
// Mathematics, per element, with c = min(1, max_norm / (norm + 1e-6)) (1 without a norm):
//   g = c grad;  m' = b1 m + (1 - b1) g;  v' = b2 v + (1 - b2) g g;  r = sqrt(v')
//   p' = p (1 - lr decay) - lr / (1 - b1^step) m' / (r / sqrt(1 - b2^step) + eps)
// One pass, bound by HBM: 28 bytes an element with fp32 states, parameters and gradients, 16.1 with 8-bit states.  The
// tensors are described in the kernel's arguments (kMaxJobs per launch), as in clip.hip: no table is copied to the device.
//
// 8-bit states are E4M3 codes with one fp32 scale for 128 consecutive elements: m, and r in place of v, which halves the
// range that the codes have to hold.  With a the block's largest magnitude (at least 2^-96) the scale is a * (1 / 448)
// and a value is coded times 448 * (1 / a), products of one reciprocal each.  Rounding to the nearest code would freeze them: a
// step moves r by a fraction (1 - b2) / 2 of itself at rest, far less than the half step of a code, 3 to 6%.  So
// the three bits of a code's mantissa are rounded by chance: 16 random bits are added behind them, and the sum is cut.
// The expected value is the value itself (to 2^-17 of a code's step); the noise that remains, a random walk held back by the
// decay, is about sqrt(half a step) = 20% of r.  Values below the codes' normal range (2^-6 of 448 under the block's
// largest) go to the nearest code.  A root that is not zero never becomes zero: m / (0 + eps) would be the step then.
// The states' arithmetic is rounded operation by operation (no fused multiply-add), so that the codes are reproducible
// anywhere from the formulas.
//
// The random bits: key = mix(mix(mix(mix(seed low) ^ seed high) ^ step) ^ the tensor's place in the list), with mix the 32-bit
// finalizer of MurmurHash3 (A. Appleby); a group of eight elements, number k, starts a 32-bit xorshift generator
// (G. Marsaglia, 2003; 13, 17, 5) from mix((key ^ k high) + k low * 0x9E3779B9) | 1, whose j-th output belongs to
// element j: its low half to m, its high half to r.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"
#include "rows.hpp"

#include <algorithm>
#include <cmath>

namespace puro {

namespace {

constexpr int kMaxJobs = 48;
constexpr int kThreads = 256;
constexpr int kVecs = 2;                   // groups of eight elements a thread takes of a chunk
constexpr int kChunk = kThreads * kVecs * 8;
constexpr int kMaxBlocks = 2048;

struct Desc {
  uint8_t* param;
  float* master;
  const uint8_t* grad;
  uint8_t* avg;
  uint8_t* sq;
  float* avg_scale;
  float* sq_scale;
  int64_t n;
  uint32_t first;      // first chunk of the job in the launch
  uint32_t place;
  uint32_t param_bf16, grad_bf16;
};
struct Table {
  Desc job[kMaxJobs];
  int n_jobs;
  uint32_t chunks;
};
static_assert(sizeof(Table) + sizeof(AdamHyper) + 64 <= 4096, "kernel arguments exceed 4 KB");

// What the elements' arithmetic takes from the hyperparameters, rounded once from 64 bits.
struct Factors {
  float b1, c1, b2, c2, eps;
  float keep;      // 1 - lr decay
  float rate;      // lr / (1 - b1^step)
  float root;      // 1 / sqrt(1 - b2^step)
};

__host__ __device__ inline double power(double b, int64_t n) {
  double p = 1.0;
  for (uint64_t k = n > 0 ? (uint64_t)n : 0; k; k >>= 1) {
    if (k & 1) p *= b;
    b *= b;
  }
  return p;
}

__host__ __device__ inline Factors factors_of(const AdamHyper& h, double lr, int64_t step) {
  Factors f;
  f.b1 = (float)h.beta1;
  f.c1 = (float)(1.0 - h.beta1);
  f.b2 = (float)h.beta2;
  f.c2 = (float)(1.0 - h.beta2);
  f.eps = (float)h.eps;
  f.keep = (float)(1.0 - lr * h.weight_decay);
  f.rate = (float)(lr / (1.0 - power(h.beta1, step)));
  f.root = (float)(1.0 / __builtin_sqrt(1.0 - power(h.beta2, step)));
  return f;
}

__host__ __device__ inline uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

__device__ __forceinline__ uint32_t shift(uint32_t x) {
  x ^= x << 13;
  x ^= x >> 17;
  return x ^ (x << 5);
}

__device__ __forceinline__ int find_job(const Table& t, uint32_t chunk) {
  int lo = 0, hi = t.n_jobs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.job[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ---- eight consecutive elements, nv of them there, of element alignment ------------------------------
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

__device__ __forceinline__ void load_values(const void* p, bool bf16, int64_t at, int nv, float v[8]) {
  if (bf16)
    unpack8<true, false>(load8<true, false>(p, at, nv), nv, v);
  else
    unpack8<false, false>(load8<false, false>(p, at, nv), nv, v);
}

__device__ __forceinline__ void store_values(void* p, bool bf16, int64_t at, int nv, const float v[8]) {
  if (bf16)
    store8<true, false, false>(p, at, nv, v);
  else
    store8<false, false, false>(p, at, nv, v);
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int nv) {
  if (nv == 8) return *reinterpret_cast<const u32x2_a1*>(p);
  u32x2 w = {0u, 0u};
  for (int e = 0; e < nv; ++e) {
    const uint32_t c = (uint32_t)p[e] << (8 * (e & 3));
    if (e < 4) w.x |= c;
    else w.y |= c;
  }
  return w;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int nv, u32x2 w) {
  if (nv == 8) {
    *reinterpret_cast<u32x2_a1*>(p) = w;
    return;
  }
  for (int e = 0; e < nv; ++e) p[e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}

__device__ __forceinline__ void decode8(u32x2 w, float scale, float v[8]) {
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[d], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[d], true);
    v[4 * d] = lo[0] * scale;
    v[4 * d + 1] = lo[1] * scale;
    v[4 * d + 2] = hi[0] * scale;
    v[4 * d + 3] = hi[1] * scale;
  }
}

// y (at most 448 but for three roundings in magnitude; NaN stays) with its mantissa cut to three bits after `chance`, 16
// bits, is added behind them.  448 and what rounding put above it stay 448: the chance is short of a step by 16 units.
__device__ __forceinline__ float cut(float y, uint32_t chance) {
  const float r = __uint_as_float((__float_as_uint(y) + (chance << 4)) & 0xFFF00000u);
  return y == y ? r : y;
}

// Scale and multiplier of a block from its largest magnitude.
__device__ __forceinline__ void block_scale(float amax, float& s, float& r) {
  const float a = __builtin_fmaxf(amax, __uint_as_float(kAmaxFloorBf16 << 16));
  s = a * (1.0f / kE4M3Max);
  r = kE4M3Max * (1.0f / a);
}

// The new states, operation by operation.
__device__ __forceinline__ void update_states(const Factors& f, float g, float& m, float& v) {
#pragma clang fp contract(off)
  m = f.b1 * m + f.c1 * g;
  v = f.b2 * v + f.c2 * g * g;
}

__device__ __forceinline__ float updated(const Factors& f, float p, float m, float r) {
  // (the quotient by the reciprocal instruction, 1 ulp: 2^-23 of a step that is itself a small part of p)
  return __builtin_fmaf(p, f.keep, -f.rate * (m * __builtin_amdgcn_rcpf(__builtin_fmaf(r, f.root, f.eps))));
}

template <bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table t, AdamHyper h, Factors given) {
  __shared__ Factors made;
  Factors f = given;
  int64_t step = h.step;
  if (h.lr_dev || h.step_dev) {
    if (h.step_dev) step = *h.step_dev;
    if (threadIdx.x == 0) made = factors_of(h, h.lr_dev ? (double)*h.lr_dev : h.lr, step);
    __syncthreads();
    f = made;
  }
  float coef = 1.f;
  if (h.norm) {
    coef = h.max_norm / (*h.norm + 1e-6f);
    coef = coef > 1.0f ? 1.0f : coef;      // a NaN stays
  }
  const uint32_t key = mix(mix(mix((uint32_t)h.seed) ^ (uint32_t)(h.seed >> 32)) ^ (uint32_t)step);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Desc& j = t.job[find_job(t, c)];
    const uint32_t own_key = mix(key ^ j.place);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int64_t group = (int64_t)(c - j.first) * (kChunk / 8) + k * kThreads + threadIdx.x;
      const int64_t at = group * 8;
      const int nv = j.n - at < 0 ? 0 : (j.n - at < 8 ? (int)(j.n - at) : 8);
      float g[8], p[8], m[8], v[8];
      load_values(j.grad, j.grad_bf16, at, nv, g);
      if (j.master)
        load_values(j.master, false, at, nv, p);
      else
        load_values(j.param, j.param_bf16, at, nv, p);
      if constexpr (EIGHT) {
        const int64_t block = at >> 7;
        const float ms = nv > 0 ? j.avg_scale[block] : 0.f, vs = nv > 0 ? j.sq_scale[block] : 0.f;
        decode8(load_codes(j.avg + at, nv), ms, m);
        decode8(load_codes(j.sq + at, nv), vs, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= v[e];
      } else {
        load_values(j.avg, false, at, nv, m);
        load_values(j.sq, false, at, nv, v);
      }
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        update_states(f, g[e] * coef, m[e], v[e]);
        r[e] = __builtin_sqrtf(v[e]);
        p[e] = updated(f, p[e], m[e], r[e]);
      }
      if (j.master) store_values(j.master, false, at, nv, p);
      store_values(j.param, j.param_bf16, at, nv, p);
      if constexpr (EIGHT) {
        const int64_t block = at >> 7;
        // (elements that are not there have a gradient and states of zero)
        float am = 0.f, ar = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          am = max3abs(am, m[e], m[e + 1]);
          ar = max3abs(ar, r[e], r[e + 1]);
        }
        float ms, mr, rs, rr;
        block_scale(row16_maxf(am), ms, mr);
        block_scale(row16_maxf(ar), rs, rr);
        uint32_t x = mix((own_key ^ (uint32_t)(group >> 32)) + (uint32_t)group * 0x9E3779B9u) | 1u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x = shift(x);
          m[e] = cut(m[e] * mr, x & 0xFFFFu);
          const float y = cut(r[e] * rr, x >> 16);
          r[e] = r[e] > 0.f && y < 0x1p-9f ? 0x1p-9f : y;
        }
        store_codes(j.avg + at, nv, u32x2{codes4(m[0], m[1], m[2], m[3]), codes4(m[4], m[5], m[6], m[7])});
        store_codes(j.sq + at, nv, u32x2{codes4(r[0], r[1], r[2], r[3]), codes4(r[4], r[5], r[6], r[7])});
        if ((threadIdx.x & 15) == 0 && nv > 0) {
          j.avg_scale[block] = ms;
          j.sq_scale[block] = rs;
        }
      } else {
        store_values(j.avg, false, at, nv, m);
        store_values(j.sq, false, at, nv, v);
      }
    }
  }
}

}  // namespace

hipError_t launch_adamw(const AdamJob* jobs, int n_jobs, bool eight, const AdamHyper& h, hipStream_t st) {
  const Factors f = factors_of(h, h.lr, h.step);
  Table t;
  t.n_jobs = 0;
  t.chunks = 0;
  auto flush = [&]() -> hipError_t {
    if (t.n_jobs == 0) return hipSuccess;
    const dim3 grid(std::min<uint32_t>(t.chunks, kMaxBlocks));
    if (eight)
      hipLaunchKernelGGL(adamw_kernel<true>, grid, dim3(kThreads), 0, st, t, h, f);
    else
      hipLaunchKernelGGL(adamw_kernel<false>, grid, dim3(kThreads), 0, st, t, h, f);
    t.n_jobs = 0;
    t.chunks = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < n_jobs; ++i) {
    const AdamJob& j = jobs[i];
    if ((j.avg_scale != nullptr) != eight || j.n == 0) continue;
    const int64_t chunks = (j.n + kChunk - 1) / kChunk;
    if (t.n_jobs == kMaxJobs || (int64_t)t.chunks + chunks > 0x7FFFFFFF) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    Desc& d = t.job[t.n_jobs++];
    d.param = static_cast<uint8_t*>(j.param);
    d.master = j.master;
    d.grad = static_cast<const uint8_t*>(j.grad);
    d.avg = static_cast<uint8_t*>(j.avg);
    d.sq = static_cast<uint8_t*>(j.sq);
    d.avg_scale = j.avg_scale;
    d.sq_scale = j.sq_scale;
    d.n = j.n;
    d.first = t.chunks;
    d.place = j.place;
    d.param_bf16 = j.param_bf16 ? 1u : 0u;
    d.grad_bf16 = j.grad_bf16 ? 1u : 0u;
    t.chunks += (uint32_t)chunks;
  }
  return flush();
}

}  // namespace puro
