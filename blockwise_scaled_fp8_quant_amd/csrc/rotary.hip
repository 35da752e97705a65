// gfx950 rotary positions: pairs of a head's values turned by an angle that grows with the token's position.
//
// Mathematics, for token t, pair i of a head with values a and b (half: columns i and i + pairs; interleaved: 2i and 2i + 1):
//   angle = position[t] freqs[i],  c = scale cos(angle),  s = scale sin(angle) (inverse: -s)
//   a' = a c - b s,  b' = b c + a s;  columns behind the pairs are copied
// The backward pass is the inverse (the transposed turn).  Bound by HBM: x is read once and y written once.
//
// The angle is formed in 64 bits, in quarter turns: position * freq is off by 2^-53 of itself (1e-9 radians at 10^7), where
// 32 bits would lose the angle of far positions.  What is left of it after the whole quarters, at most half a quarter
// turn, goes on in 32 bits.  A workgroup forms the cosines and sines of its tokens once, in LDS, and all heads use them.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"
#include "rows.hpp"

#include <algorithm>
#include <type_traits>

namespace puro {

namespace {

constexpr int kThreads = 256;
// Chunks of a workgroup's tile.  Measured, us, 16384 x 24 x 128 bf16 half and 8192 x 24 x 128 fp32 interleaved, half of the head:
// 33.6 (6.0 TB/s) and 32.4 (6.2); 512 chunks 32.3 and 37.0, 256 33.9 and 41.1 (a tile's few tokens have as many angles), 2048
// 33.7 and 33.0, and 64 tokens of the latter 4.9 in place of 4.2.  Chunks of eight fp32 columns, where a wave's accesses
// leave gaps, 40.1.
constexpr int kTileChunks = 1024;

struct RotaryPlan {
  int tokens;        // of a workgroup's tile
  int heads;         // of a workgroup's tile
  int splits;        // tiles that share their tokens
  int units;         // chunks of a head: of 16 bytes, or two of them that make pairs (half layout)
  int turned;        // the first of them hold pairs (half layout), the others copied columns
  int64_t tiles;
};

__device__ __forceinline__ float2 cos_sin(double position, double freq, float scale, bool inverse) {
  const double quarters = position * freq * 0.63661977236758134308;   // 2 / pi
  const double n = __builtin_rint(quarters);
  // n modulo 4, exact: n / 4 has the same digits
  const int q = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  float s, c;
  sincospif((float)(quarters - n) * 0.5f, &s, &c);
  const float cq = (q & 1) ? s : c, sq = (q & 1) ? c : s;
  const float co = (q == 1 || q == 2) ? -cq : cq, si = (q & 2) ? -sq : sq;
  return make_float2(scale * co, scale * (inverse ? -si : si));
}

// 16 bytes of a head: eight bf16 columns or four fp32 ones, nv of them there (a whole chunk where VEC), so that a wave's
// accesses fill whole lines.
template <bool BF16>
constexpr int kPer = BF16 ? 8 : 4;

template <bool BF16, bool VEC, bool NT>
__device__ __forceinline__ u32x4 load16(const void* base, int64_t at, int nv) {
  if constexpr (BF16) {
    return settle8<true, VEC>(load8<true, VEC, NT>(base, at, nv), nv).w[0];
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
    if constexpr (VEC) {
      const u32x4* v = reinterpret_cast<const u32x4*>(p);
      if constexpr (NT) return __builtin_nontemporal_load(v);
      return *v;
    }
    if (nv == 4) return *reinterpret_cast<const u32x4_a4*>(p);
    u32x4 w = {0u, 0u, 0u, 0u};
    if (nv > 0) w.x = p[0];
    if (nv > 1) w.y = p[1];
    if (nv > 2) w.z = p[2];
    return w;
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store16(void* base, int64_t at, int nv, u32x4 w) {
  if constexpr (BF16) {
    Raw8<true> r;
    r.w[0] = w;
    store_raw8<true, VEC, VEC>(base, at, nv, r);
  } else {
    uint32_t* p = static_cast<uint32_t*>(base) + at;
    if constexpr (VEC) {
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
    } else if (nv == 4) {
      *reinterpret_cast<u32x4_a4*>(p) = w;
    } else {
      if (nv > 0) p[0] = w.x;
      if (nv > 1) p[1] = w.y;
      if (nv > 2) p[2] = w.z;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack16(u32x4 w, float (&v)[kPer<BF16>]) {
#pragma unroll
  for (int j = 0; j < kPer<BF16>; ++j)
    v[j] = !BF16 ? __uint_as_float(w[j & 3]) : (j & 1) ? bf16_hi(w[(j >> 1) & 3]) : bf16_lo(w[(j >> 1) & 3]);
}

template <bool BF16>
__device__ __forceinline__ u32x4 pack16(const float (&v)[kPer<BF16>]) {
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) w[k] = bf16x2_rne(v[2 * k], v[2 * k + 1]);
    else w[k] = __float_as_uint(v[k]);
  }
  return w;
}

// One tile after the other (one, but for the longest inputs).  A thread takes chunks kThreads apart: chunk u of
// head h of token t.  Consecutive lanes hold consecutive chunks, then heads, then tokens.
template <bool BF16, bool VEC, bool INTERLEAVED, bool STREAM>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryPlan p) {
  constexpr int PER = kPer<BF16>;
  extern __shared__ float2 turn[];       // [tokens][pairs]
  const int per_head = p.units, per_token = p.units * p.heads;
  // where a thread's first chunk is, and how far the next one is
  const int u0 = threadIdx.x % per_head, h0 = threadIdx.x / per_head % p.heads, t0 = threadIdx.x / per_token;
  const int du = kThreads % per_head, dh = kThreads / per_head % p.heads, dt = kThreads / per_token;
  auto load = [&](int64_t at, int nv) { return load16<BF16, VEC, STREAM>(a.x, at, nv); };
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t group = tile / p.splits;
    const int head0 = (int)(tile - group * p.splits) * p.heads;
    const int64_t token0 = group * p.tokens;
    const int tokens = (int)(a.T - token0 < p.tokens ? a.T - token0 : p.tokens);
    const int heads = a.H - head0 < p.heads ? a.H - head0 : p.heads;
    for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
      const int t = i / a.pairs;
      const int64_t at = token0 + t;
      const int64_t position = a.positions ? a.positions[at] : a.start + at;
      turn[i] = cos_sin((double)position, a.freqs[i - t * a.pairs], a.scale, a.inverse);
    }
    __syncthreads();
    int u = u0, h = h0, t = t0;
    while (t < tokens) {
      if (h < heads) {
        const int64_t in = (token0 + t) * a.ldt + (int64_t)(head0 + h) * a.ldh;
        const int64_t out = (token0 + t) * a.ldyt + (int64_t)(head0 + h) * a.ldyh;
        const float2* cs = turn + t * a.pairs;
        if constexpr (INTERLEAVED) {
          const int col = PER * u, nv = a.D - col < PER ? a.D - col : PER;
          u32x4 w = load(in + col, nv);
          if (col < 2 * a.pairs) {
            float v[PER];
            unpack16<BF16>(w, v);
            const int here = a.pairs - PER / 2 * u;      // pairs of the chunk; columns behind them keep their bits
#pragma unroll
            for (int j = 0; j < PER / 2; ++j) {
              const float2 c = cs[PER / 2 * u + (j < here ? j : 0)];
              const float x = v[2 * j], y = v[2 * j + 1];
              v[2 * j] = x * c.x - y * c.y;
              v[2 * j + 1] = y * c.x + x * c.y;
            }
            const u32x4 o = pack16<BF16>(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = (BF16 ? k : k / 2) < here ? o[k] : w[k];
          }
          store16<BF16, VEC>(a.y, out + col, nv, w);
        } else if (u < p.turned) {
          const int col = PER * u, nv = a.pairs - col < PER ? a.pairs - col : PER;
          float x[PER], y[PER];
          const u32x4 wa = load(in + col, nv), wb = load(in + a.pairs + col, nv);
          unpack16<BF16>(wa, x);
          unpack16<BF16>(wb, y);
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const float2 c = cs[j < nv ? col + j : 0];
            const float z = x[j] * c.x - y[j] * c.y;
            y[j] = y[j] * c.x + x[j] * c.y;
            x[j] = z;
          }
          store16<BF16, VEC>(a.y, out + col, nv, pack16<BF16>(x));
          store16<BF16, VEC>(a.y, out + a.pairs + col, nv, pack16<BF16>(y));
        } else {
          const int col = 2 * a.pairs + PER * (u - p.turned), nv = a.D - col < PER ? a.D - col : PER;
          store16<BF16, VEC>(a.y, out + col, nv, load(in + col, nv));
        }
      }
      u += du;
      h += dh;
      t += dt;
      if (u >= per_head) {
        u -= per_head;
        ++h;
      }
      if (h >= p.heads) {
        h -= p.heads;
        ++t;
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st) {
  const int64_t es = a.bf16 ? 2 : 4;
  const bool in_place = a.x == a.y;      // (the strides are then the same: the copied columns are there)
  RotaryPlan p;
  const int per = a.bf16 ? 8 : 4;
  auto chunks = [&](int columns) { return (columns + per - 1) / per; };
  p.turned = chunks(a.interleaved ? (in_place ? 2 * a.pairs : a.D) : a.pairs);
  p.units = p.turned + (a.interleaved || in_place ? 0 : chunks(a.D - 2 * a.pairs));
  if (p.units == 0) return hipSuccess;
  // A tile is about kTileChunks chunks: whole tokens, up to those whose cosines and sines are one a thread, or some heads of one.
  const int64_t token = (int64_t)a.H * p.units;
  p.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kTileChunks / token, a.pairs ? (kThreads + a.pairs - 1) / a.pairs : 64));
  p.heads = (int)std::max<int64_t>(1, std::min<int64_t>(a.H, kTileChunks / ((int64_t)p.tokens * p.units)));
  p.splits = (int)(((int64_t)a.H + p.heads - 1) / p.heads);
  p.heads = (int)(((int64_t)a.H + p.splits - 1) / p.splits);
  p.tiles = (a.T + p.tokens - 1) / p.tokens * p.splits;
  const unsigned blocks = (unsigned)std::min<int64_t>(p.tiles, 1 << 22);
  const size_t lds = (size_t)p.tokens * a.pairs * sizeof(float2);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), lds, st, a, p);
    return hipGetLastError();
  };
  auto rows = [&](const void* q, int64_t t, int64_t h) {
    return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && (a.T == 1 || t * es % 16 == 0) && (a.H == 1 || h * es % 16 == 0);
  };
  const bool vec = a.D % per == 0 && (a.interleaved || a.pairs % per == 0) &&
                   rows(a.x, a.ldt, a.ldh) && rows(a.y, a.ldyt, a.ldyh);
  // y is written past the caches, which leaves x where it is; STREAM: x is read past them too, where the call moves more than
  // the memory-side cache holds.  us, 24 x 128 bf16, three x and two y in turn, without - writing past - both: 4096 rows 9.6 - 9.7 -
  // 12.1, 8192 19.5 - 17.1 - 20.9, 16384 40.1 - 34.0 - 38.1, 32768 76.6 - 73.7 - 72.6; fp32 32768 rows 141 - 137 - 127.5.
  const bool stream = vec && a.T > kMemorySideCache / (2 * es * a.D) / a.H;
  auto pick = [&](auto bf16, auto interleaved) {
    constexpr bool B = decltype(bf16)::value, I = decltype(interleaved)::value;
    return stream ? go(rotary_kernel<B, true, I, true>) : vec ? go(rotary_kernel<B, true, I, false>) : go(rotary_kernel<B, false, I, false>);
  };
  if (a.bf16) return a.interleaved ? pick(std::true_type(), std::true_type()) : pick(std::true_type(), std::false_type());
  return a.interleaved ? pick(std::false_type(), std::true_type()) : pick(std::false_type(), std::false_type());
}

}  // namespace puro
