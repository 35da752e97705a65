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
// Of the 20 bits that are cut the lowest four meet no random ones: the expected magnitude is the value's, less 0 to 15 2^-20 of
// a code's step (2^-17 on average).  The noise that remains, a random walk held back by the decay, is about sqrt(half a
// step) = 20% of r.  Values below the codes' normal range (2^-6 of 448 under the block's
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
// Threads of a workgroup, with fp32 and with 8-bit states.
constexpr int kThreads32 = 128, kThreads8 = 256;
// Elements a thread takes: one round of 16 bytes of fp32, or of 8 codes, so that workgroups come and go in the order of the
// addresses.  A launch has one for every chunk, up to its 2^32 threads.  403 M elements, us, fp32 and 8-bit states, in turn on
// one card (others: 1836 to 1901 and 1164 to 1179): 1894 (5.96 TB/s) and 1159 (5.61); two rounds a thread 2013 and 1223; 2048 workgroups that stay 2120 and 1326; workgroups of
// 256 and 512 threads 1920 and 1970, of 128 and 512 1183 and 1182.
constexpr int kPer32 = 4, kPer8 = 8;
constexpr uint32_t kMaxBlocks = 1u << 23;

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

// ---- a thread's elements: PER consecutive ones, nv of them there, behind a uniform base --------------
// Of element alignment: wide accesses of this target need no more.  (A uniform base and a 32-bit offset are an access
// without address arithmetic.)  Everything goes past the caches (NT), since no step reads it again soon: 403 M elements with
// fp32 states 1919 us, without 2064; with 8-bit states 1178 and 1201.
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <int PER>
__device__ __forceinline__ void load_values(const uint8_t* base, bool bf16, uint32_t at, int nv, float v[PER]) {
  if (bf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base + 2 * at);
    if (nv == PER) {
      uint32_t w[PER / 2];
      if constexpr (PER == 8) {
        const u32x4 r = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
        w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
      } else {
        const u32x2 r = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a2*>(p));
        w[0] = r.x; w[1] = r.y;
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = e < nv ? __uint_as_float((uint32_t)p[e] << 16) : 0.f;
    }
  } else {
    const float* p = reinterpret_cast<const float*>(base + 4 * at);
    if (nv == PER) {
#pragma unroll
      for (int k = 0; k < PER; k += 4) {
        const u32x4 r = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p + k));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = __uint_as_float(r[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = e < nv ? p[e] : 0.f;
    }
  }
}

template <int PER>
__device__ __forceinline__ void store_values(uint8_t* base, bool bf16, uint32_t at, int nv, const float v[PER]) {
  if (bf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base + 2 * at);
    uint32_t w[PER / 2];
#pragma unroll
    for (int e = 0; e < PER; e += 2) w[e >> 1] = bf16x2_rne(v[e], v[e + 1]);
    if (nv == PER) {
      if constexpr (PER == 8)
        __builtin_nontemporal_store((u32x4{w[0], w[1], w[2], w[3]}), reinterpret_cast<u32x4_a2*>(p));
      else
        __builtin_nontemporal_store((u32x2{w[0], w[1]}), reinterpret_cast<u32x2_a2*>(p));
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (e < nv) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(base + 4 * at);
    if (nv == PER) {
#pragma unroll
      for (int k = 0; k < PER; k += 4)
        __builtin_nontemporal_store((u32x4{__float_as_uint(v[k]), __float_as_uint(v[k + 1]),
                                                       __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])}), reinterpret_cast<u32x4_a4*>(p + k));
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (e < nv) p[e] = v[e];
    }
  }
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int nv) {
  if (nv == 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1*>(p));
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
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2_a1*>(p));
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

// y (at most 448 but for three roundings in magnitude, no NaN) with its mantissa cut to three bits after `chance`, 16
// bits, is added behind them.  448 and what rounding put above it stay 448: the chance is short of a step by 16 units.  (What
// rounding put below it stays 448 too, but for a chance of 0, one in 65536.)
__device__ __forceinline__ float cut(float y, uint32_t chance) {
  return __uint_as_float((__float_as_uint(y) + (chance << 4)) & 0xFFF00000u);
}

// Scale and multiplier of a block from its largest magnitude.  One below 2^126 has its reciprocal by the instruction and one
// correction, which is correctly rounded for every mantissa (SHORT; the general quotient takes three times as many
// instructions).
template <bool SHORT>
__device__ __forceinline__ void block_scale(float amax, float& s, float& r) {
  const float a = __builtin_fmaxf(amax, __uint_as_float(kAmaxFloorBf16 << 16));
  s = a * (1.0f / kE4M3Max);
  if constexpr (SHORT) {
    const float y = __builtin_amdgcn_rcpf(a);
    r = kE4M3Max * __builtin_fmaf(__builtin_fmaf(-a, y, 1.0f), y, y);
  } else {
    r = kE4M3Max * (1.0f / a);
  }
}

// Largest value of the 16 lanes of a block (values >= 0).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  // (every lane has a source: the bound control only lets the compiler make one instruction of it)
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float block_max(float v) {
  uint32_t b = __float_as_uint(v);
  b = dpp_max<kDppQuadXor1>(b);
  b = dpp_max<kDppQuadXor2>(b);
  b = dpp_max<kDppRowHalfMirror>(b);
  return __uint_as_float(dpp_max<kDppRowMirror>(b));
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

// The roots of a thread's values, correctly rounded.  Returns whether all of the wave's values are usual ones, finite and at
// least 2^-96; for those a root is the product with the reciprocal root and one correction, exact here for every
// mantissa (8 instruction slots, where the general root, with its scaling and special cases, takes about 20).
template <int PER>
__device__ __forceinline__ bool roots(const float v[PER], float r[PER]) {
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint32_t b = __float_as_uint(v[e]);      // v >= 0 orders as its bits; a NaN is above infinity
    lo = lo < b ? lo : b;
    hi = hi > b ? hi : b;
  }
  const bool usual = __all(lo >= 0x0F800000u && hi < 0x7F800000u);
  if (usual) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const float y = __builtin_amdgcn_rsqf(v[e]), s = v[e] * y;
      r[e] = __builtin_fmaf(__builtin_fmaf(-s, s, v[e]), 0.5f * y, s);
    }
  } else {
#pragma unroll
    for (int e = 0; e < PER; ++e) r[e] = __builtin_sqrtf(v[e]);
  }
  return usual;
}

template <bool EIGHT>
__global__ __launch_bounds__(EIGHT ? kThreads8 : kThreads32) void adamw_kernel(Table t, AdamHyper h, Factors given) {
  constexpr int PER = EIGHT ? kPer8 : kPer32;
  constexpr int kChunk = (EIGHT ? kThreads8 : kThreads32) * PER;
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
  int job = 0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    if (job + 1 < t.n_jobs && t.job[job + 1].first <= c) job = find_job(t, c);
    const Desc& j = t.job[job];
    const int64_t start = (int64_t)(c - j.first) * kChunk;
    const int64_t left = j.n - start;
    const uint8_t* grad = j.grad + start * (j.grad_bf16 ? 2 : 4);
    uint8_t* param = j.param + start * (j.param_bf16 ? 2 : 4);
    uint8_t* held = j.master ? reinterpret_cast<uint8_t*>(j.master + start) : param;
    const bool held_bf16 = !j.master && j.param_bf16;
    uint8_t* avg = j.avg + start * (EIGHT ? 1 : 4);
    uint8_t* sq = j.sq + start * (EIGHT ? 1 : 4);
    const uint32_t at = threadIdx.x * PER;
    auto take = [&](int nv) {
      float g[PER], p[PER], m[PER], v[PER], r[PER];
      load_values<PER>(grad, j.grad_bf16, at, nv, g);
      load_values<PER>(held, held_bf16, at, nv, p);
      if constexpr (EIGHT) {
        const uint32_t block = at >> 7;
        const u32x2 cm = load_codes(avg + at, nv), cv = load_codes(sq + at, nv);
        const float ms = nv > 0 ? (j.avg_scale + (start >> 7))[block] : 0.f;
        const float vs = nv > 0 ? (j.sq_scale + (start >> 7))[block] : 0.f;
        decode8(cm, ms, m);
        decode8(cv, vs, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= v[e];
      } else {
        load_values<PER>(avg, false, at, nv, m);
        load_values<PER>(sq, false, at, nv, v);
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) update_states(f, g[e] * coef, m[e], v[e]);
      const bool usual = roots<PER>(v, r);
#pragma unroll
      for (int e = 0; e < PER; ++e) p[e] = updated(f, p[e], m[e], r[e]);
      store_values<PER>(held, held_bf16, at, nv, p);
      if (j.master) store_values<PER>(param, true, at, nv, p);
      if constexpr (EIGHT) {
        // (elements that are not there have a gradient and states of zero)
        float am = 0.f, ar = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          am = max3abs(am, m[e], m[e + 1]);
          ar = max3abs(ar, r[e], r[e + 1]);
        }
        am = block_max(am);
        ar = block_max(ar);
        float ms, mr, rs, rr;
        const int64_t group = (start >> 3) + threadIdx.x;
        uint32_t x = mix((mix(key ^ j.place) ^ (uint32_t)(group >> 32)) + (uint32_t)group * 0x9E3779B9u) | 1u;
        // a NaN among the moments makes their sum one
        float any = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) any += m[e];
        // (the roots are below 2^64 then)
        if (usual && __all(any == any && am < 0x1p126f)) {
          block_scale<true>(am, ms, mr);
          block_scale<true>(ar, rs, rr);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x = shift(x);
            m[e] = cut(m[e] * mr, x & 0xFFFFu);
            // positive: orders as its bits
            r[e] = __uint_as_float(umax(__float_as_uint(cut(r[e] * rr, x >> 16)), __float_as_uint(0x1p-9f)));
          }
        } else {
          block_scale<false>(am, ms, mr);
          block_scale<false>(ar, rs, rr);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x = shift(x);
            const float ym = m[e] * mr, yr = r[e] * rr;
            m[e] = ym == ym ? cut(ym, x & 0xFFFFu) : ym;
            const float y = yr == yr ? cut(yr, x >> 16) : yr;
            r[e] = r[e] > 0.f && y < 0x1p-9f ? 0x1p-9f : y;
          }
        }
        store_codes(avg + at, nv, u32x2{codes4(m[0], m[1], m[2], m[3]), codes4(m[4], m[5], m[6], m[7])});
        store_codes(sq + at, nv, u32x2{codes4(r[0], r[1], r[2], r[3]), codes4(r[4], r[5], r[6], r[7])});
        if ((threadIdx.x & 15) == 0 && nv > 0) {
          (j.avg_scale + (start >> 7))[at >> 7] = ms;
          (j.sq_scale + (start >> 7))[at >> 7] = rs;
        }
      } else {
        store_values<PER>(avg, false, at, nv, m);
        store_values<PER>(sq, false, at, nv, v);
      }
    };
    // (a whole chunk's elements are known to be there)
    if (left >= kChunk)
      take(PER);
    else
      take(left - at < 0 ? 0 : (left - at < PER ? (int)(left - at) : PER));
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
      hipLaunchKernelGGL(adamw_kernel<true>, grid, dim3(kThreads8), 0, st, t, h, f);
    else
      hipLaunchKernelGGL(adamw_kernel<false>, grid, dim3(kThreads32), 0, st, t, h, f);
    t.n_jobs = 0;
    t.chunks = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < n_jobs; ++i) {
    const AdamJob& j = jobs[i];
    if ((j.avg_scale != nullptr) != eight || j.n == 0) continue;
    const int64_t chunk = eight ? kThreads8 * kPer8 : kThreads32 * kPer32, chunks = (j.n + chunk - 1) / chunk;
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
