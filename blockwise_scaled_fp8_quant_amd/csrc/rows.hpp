// Device-side helpers of the kernels that hold rows in registers (norm.hip, residual.hip): eight consecutive columns of a
// row in any alignment, sums over the lanes and waves that share a row, the norm and the codes of eight columns.
#pragma once

#include "codec.hpp"
#include "gemm_args.hpp"

namespace puro {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---- eight consecutive columns of a row -------------------------------------------------------------
// VEC: 16-byte aligned, either all eight exist or none.  Otherwise a row starts at any element and its last chunk may
// be short.  Whole chunks are moved 16 bytes at a time all the same: global accesses of this target need the
// element's alignment alone.  A short chunk is moved in pieces of 4, 2 and 1 elements, which stay where the loads put
// them until the row is used (unpack8), so that nothing waits for them before.  At 16384 x 2047 bf16, us forward and
// backward: element by element 79 and 179, whole chunks wide 38 and 101, short ones in pieces 34 and 46.
template <bool BF16>
struct Raw8 {
  u32x4 w[BF16 ? 1 : 2];
};

// Makes the compiler take a value for new, so that what it computed from it before does not stay in registers.
template <bool BF16>
__device__ __forceinline__ void forget(Raw8<BF16>& r) {
  asm volatile("" : "+v"(r.w[0]));
  if constexpr (!BF16) asm volatile("" : "+v"(r.w[1]));
}

// memory vectors of element alignment
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

// NT: past the caches, for aligned rows of large calls (beyond_cache, kMemorySideCache).
template <bool BF16, bool VEC, bool NT = false>
__device__ __forceinline__ Raw8<BF16> load8(const void* base, int64_t at, int nv) {
  Raw8<BF16> r;
  r.w[0] = u32x4{0u, 0u, 0u, 0u};
  if constexpr (!BF16) r.w[1] = u32x4{0u, 0u, 0u, 0u};
  if constexpr (VEC) {
    // (hides that the other side of a branch loads the same: the compiler would make one load of both, and no NT; see apart)
    if constexpr (NT) asm("" : "+v"(at));
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + at * (BF16 ? 2 : 4));
    if (nv > 0) {
      if constexpr (NT) {
        r.w[0] = __builtin_nontemporal_load(p);
        if constexpr (!BF16) r.w[1] = __builtin_nontemporal_load(p + 1);
      } else {
        r.w[0] = p[0];
        if constexpr (!BF16) r.w[1] = p[1];
      }
    }
  } else if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (nv == 8) {
      r.w[0] = *reinterpret_cast<const u32x4_a2*>(p);
    } else if (nv > 0) {
      if (nv & 4) {
        const u32x2 v = *reinterpret_cast<const u32x2_a2*>(p);
        r.w[0].x = v.x;
        r.w[0].y = v.y;
      }
      if (nv & 2) r.w[0].z = *reinterpret_cast<const u32_a2*>(p + (nv & 4));
      if (nv & 1) r.w[0].w = p[nv & 6];
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
    if (nv == 8) {
      r.w[0] = *reinterpret_cast<const u32x4_a4*>(p);
      r.w[1] = *reinterpret_cast<const u32x4_a4*>(p + 4);
    } else if (nv > 0) {
      if (nv & 4) r.w[0] = *reinterpret_cast<const u32x4_a4*>(p);
      if (nv & 2) {
        const u32x2 v = *reinterpret_cast<const u32x2_a4*>(p + (nv & 4));
        r.w[1].x = v.x;
        r.w[1].y = v.y;
      }
      if (nv & 1) r.w[1].z = p[nv & 6];
    }
  }
  return r;
}

// A chunk's elements in order, zero where there is no column.
template <bool BF16, bool VEC>
__device__ __forceinline__ Raw8<BF16> settle8(const Raw8<BF16>& r, int nv) {
  Raw8<BF16> o = r;
  if (VEC || nv == 8) return o;
  if constexpr (BF16) {
    const u32x4 w = r.w[0];
    const uint32_t t0 = (nv & 2) ? w.z : w.w, t1 = (nv & 2) ? w.w : 0u;
    o.w[0] = (nv & 4) ? u32x4{w.x, w.y, t0, t1} : u32x4{t0, t1, 0u, 0u};
  } else {
    const u32x4 hi = r.w[1];
    o.w[1] = (nv & 2) ? u32x4{hi.x, hi.y, hi.z, 0u} : u32x4{hi.z, 0u, 0u, 0u};
    if (!(nv & 4)) {
      o.w[0] = o.w[1];
      o.w[1] = u32x4{0u, 0u, 0u, 0u};
    }
  }
  return o;
}

// The eight values, zero where there is no column.
template <bool BF16, bool VEC>
__device__ __forceinline__ void unpack8(const Raw8<BF16>& raw, int nv, float v[8]) {
  const Raw8<BF16> r = settle8<BF16, VEC>(raw, nv);
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? bf16_hi(r.w[0][j >> 1]) : bf16_lo(r.w[0][j >> 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(r.w[0][j]);
      v[j + 4] = __uint_as_float(r.w[1][j]);
    }
  }
}

// At both ends of such a branch, of loads or stores, for the same reason.
__device__ __forceinline__ void apart() { asm volatile(""); }

// The eight values rounded to the row's type.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> pack8(const float v[8]) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.w[0] = u32x4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
  } else {
    r.w[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
    r.w[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
  }
  return r;
}

// NT: past the caches, for aligned bf16 rows (where a store instruction fills whole lines).  Measured at
// 16384 x 2048 bf16 with inputs in rotation: the forward pass 23.2 us with such stores and 25.4 without (they
// leave the memory-side cache to x), the backward pass 42.0 and 38.9 (its inputs exceed that cache).
template <bool BF16, bool VEC, bool NT>
__device__ __forceinline__ void store_raw8(void* base, int64_t at, int nv, const Raw8<BF16>& r) {
  if constexpr (BF16) {
    const u32x4 o = r.w[0];
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (VEC) {
      if (nv > 0) {
        if constexpr (NT)
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(p));
        else
          *reinterpret_cast<u32x4*>(p) = o;
      }
    } else if (nv == 8) {
      *reinterpret_cast<u32x4_a2*>(p) = o;
    } else if (nv > 0) {
      if (nv & 4) *reinterpret_cast<u32x2_a2*>(p) = u32x2{o.x, o.y};
      const uint32_t two = (nv & 4) ? o.z : o.x, three = (nv & 4) ? o.w : o.y;
      if (nv & 2) *reinterpret_cast<u32_a2*>(p + (nv & 4)) = two;
      if (nv & 1) p[nv & 6] = (uint16_t)((nv & 2) ? three : two);
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    const u32x4 lo = r.w[0], hi = r.w[1];
    if constexpr (VEC) {
      if (nv > 0) {
        reinterpret_cast<u32x4*>(p)[0] = lo;
        reinterpret_cast<u32x4*>(p)[1] = hi;
      }
    } else if (nv == 8) {
      *reinterpret_cast<u32x4_a4*>(p) = lo;
      *reinterpret_cast<u32x4_a4*>(p + 4) = hi;
    } else if (nv > 0) {
      if (nv & 4) *reinterpret_cast<u32x4_a4*>(p) = lo;
      const u32x4 t = (nv & 4) ? hi : lo;
      if (nv & 2) *reinterpret_cast<u32x2_a4*>(p + (nv & 4)) = u32x2{t.x, t.y};
      if (nv & 1) p[nv & 6] = __uint_as_float((nv & 2) ? t.z : t.x);
    }
  }
}

template <bool BF16, bool VEC, bool NT>
__device__ __forceinline__ void store8(void* base, int64_t at, int nv, const float v[8]) {
  store_raw8<BF16, VEC, NT>(base, at, nv, pack8<BF16>(v));
}

// Eight values of a weight or bias vector, read once per thread and launch: two 16-byte loads (one for
// bf16) where the vector is aligned and all eight exist, else element by element.
__device__ __forceinline__ void load_vec8(const void* base, bool bf16, bool aligned, int col, int nv, float v[8]) {
  if (aligned && nv == 8) {
    if (bf16)
      unpack8<true, true>(load8<true, true>(base, col, 8), 8, v);
    else
      unpack8<false, true>(load8<false, true>(base, col, 8), 8, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.f;
    if (j < nv)
      v[j] = bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[col + j] << 16)
                  : static_cast<const float*>(base)[col + j];
  }
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---- sums over the lanes of a wave and the waves of a team -------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}

// Sum over the 16, 32 or 64 lanes of a wave that share a row (N; more: over the wave).
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<kDppQuadXor1>(v);
  v = dpp_add<kDppQuadXor2>(v);
  v = dpp_add<kDppRowHalfMirror>(v);
  v = dpp_add<kDppRowMirror>(v);
  if constexpr (N > 16) v += __shfl_xor(v, 16);
  if constexpr (N > 32) v += __shfl_xor(v, 32);
  return v;
}

// Sum over a team of LPR lanes; every lane gets it.  `slot` is one of two LDS rows used in turn, so a
// wave that runs ahead into the next sum does not overwrite what a slower one still reads (the
// barrier of the next sum is between them).
template <int LPR, int WAVES>
__device__ __forceinline__ float team_sum(float v, float (*red)[WAVES], int slot) {
  v = lanes_sum<LPR>(v);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < LPR / 64; ++w) v += red[slot][wave / (LPR / 64) * (LPR / 64) + w];
  }
  return v;
}

// Scale and multiplier of a group from its fp32 maximum, as tile_scale (codec.hpp).
__device__ __forceinline__ void tile_scale32(float amax, float& s, float& r) {
  const float a = __builtin_fmaxf(amax, __uint_as_float(kAmaxFloorBf16 << 16));
  s = a / kE4M3Max;
  r = kE4M3Max / a;
}

// The norm of eight columns: the mean is taken out of x before anything is rounded, so that a row whose values lie far
// from zero and close together keeps its differences (a constant row's are zero).  v: x - mean.
__device__ __forceinline__ void norm8(const float v[8], float rstd, const float g[8], const float b[8], float y[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(v[j] * rstd, g[j], b[j]);
}

// max(m, |a|, |b|): one v_max3_f32.  A NaN does not enter (its code is NaN whatever the scale).
__device__ __forceinline__ float max3abs(float m, float a, float b) {
  return __builtin_fmaxf(__builtin_fmaxf(m, __builtin_fabsf(a)), __builtin_fabsf(b));
}

// Four values to codes.  The convert that writes the low half keeps the other half of its register: one of
// its own operands serves, where a zero would have to be put there first.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt2_hi(c, d, cvt2_lo(a, b, __float_as_uint(a)));
}

__device__ __forceinline__ float row16_maxf(float v) {   // v >= 0
  return __uint_as_float(row16_max(__float_as_uint(v)));
}

// A lane's part of a row's sum of values (missing columns were loaded as zero) and, of differences from the mean, of
// squares, where a missing column holds no zero.
template <int ITER>
__device__ __forceinline__ float lane_sum(const float (&v)[ITER][8]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[i][j];
  return sum;
}

template <bool VEC, int ITER>
__device__ __forceinline__ float lane_squares(const float (&v)[ITER][8], const int (&nv)[ITER]) {
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    float part = 0.f;
    if (VEC || nv[i] == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part = __builtin_fmaf(v[i][j], v[i][j], part);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j) part = j < nv[i] ? __builtin_fmaf(v[i][j], v[i][j], part) : part;
    }
    sq += nv[i] > 0 ? part : 0.f;
  }
  return sq;
}

// Eight columns of a normed row as codes at q, and their group's scale (16 lanes hold a group; the first writes it).
__device__ __forceinline__ void store_codes8(uint8_t* q, float* s, bool ok, bool first, const float y[8]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) m = max3abs(m, y[j], y[j + 1]);
  float sc, r;
  tile_scale32(row16_maxf(m), sc, r);
  if (ok) {
    const u32x2 o = {codes4(y[0] * r, y[1] * r, y[2] * r, y[3] * r), codes4(y[4] * r, y[5] * r, y[6] * r, y[7] * r)};
    __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(q));
    if (first) *s = sc;
  }
}

// Bytes of the memory-side cache.
constexpr int64_t kMemorySideCache = 256 << 20;

inline bool vec_row(const void* p, int64_t ld, int64_t es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0;
}

}  // namespace

}  // namespace puro
