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

namespace puro {

namespace {

constexpr int kThreads = 256;

struct RotaryPlan {
  int tokens;        // of a workgroup's tile
  int heads;         // of a workgroup's tile
  int splits;        // tiles that share their tokens
  int units;         // chunks of a head: eight pairs, or eight columns
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

// One tile after the other (one, but for the longest inputs).  A thread takes chunks kThreads apart: chunk u of
// head h of token t.  Consecutive lanes hold consecutive chunks, then heads, then tokens.
template <bool BF16, bool VEC, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryPlan p) {
  extern __shared__ float2 turn[];       // [tokens][pairs]
  const int per_head = p.units, per_token = p.units * p.heads;
  // where a thread's first chunk is, and how far the next one is
  const int u0 = threadIdx.x % per_head, h0 = threadIdx.x / per_head % p.heads, t0 = threadIdx.x / per_token;
  const int du = kThreads % per_head, dh = kThreads / per_head % p.heads, dt = kThreads / per_token;
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
          const int col = 8 * u, nv = a.D - col < 8 ? a.D - col : 8;
          const Raw8<BF16> r = load8<BF16, VEC>(a.x, in + col, nv);
          float v[8];
          unpack8<BF16, VEC>(r, nv, v);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int i = 4 * u + j / 2;
            if (i < a.pairs) {
              const float2 w = cs[i];
              const float x = v[j], y = v[j + 1];
              v[j] = x * w.x - y * w.y;
              v[j + 1] = y * w.x + x * w.y;
            }
          }
          store8<BF16, VEC, false>(a.y, out + col, nv, v);
        } else if (u < p.turned) {
          const int col = 8 * u, nv = a.pairs - col < 8 ? a.pairs - col : 8;
          const Raw8<BF16> ra = load8<BF16, VEC>(a.x, in + col, nv), rb = load8<BF16, VEC>(a.x, in + a.pairs + col, nv);
          float x[8], y[8];
          unpack8<BF16, VEC>(ra, nv, x);
          unpack8<BF16, VEC>(rb, nv, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 w = cs[j < nv ? col + j : 0];
            const float z = x[j] * w.x - y[j] * w.y;
            y[j] = y[j] * w.x + x[j] * w.y;
            x[j] = z;
          }
          store8<BF16, VEC, false>(a.y, out + col, nv, x);
          store8<BF16, VEC, false>(a.y, out + a.pairs + col, nv, y);
        } else {
          const int col = 2 * a.pairs + 8 * (u - p.turned), nv = a.D - col < 8 ? a.D - col : 8;
          store_raw8<BF16, VEC, false>(a.y, out + col, nv, settle8<BF16, VEC>(load8<BF16, VEC>(a.x, in + col, nv), nv));
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
  if (a.interleaved) {
    p.turned = p.units = (int)(((in_place ? 2 * a.pairs : a.D) + 7) / 8);
  } else {
    p.turned = (a.pairs + 7) / 8;
    p.units = p.turned + (in_place ? 0 : (a.D - 2 * a.pairs + 7) / 8);
  }
  if (p.units == 0) return hipSuccess;
  // Tokens whose cosines and sines a workgroup forms together: one a thread, or more where a token has more.
  p.tokens = std::max(1, std::min(a.pairs ? (kThreads + a.pairs - 1) / a.pairs : 16, 64));
  // Heads of a tile: about 8 chunks a thread.
  p.heads = std::max(1, std::min(a.H, 8 * kThreads / (p.tokens * p.units)));
  p.splits = (a.H + p.heads - 1) / p.heads;
  p.heads = (a.H + p.splits - 1) / p.splits;
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
  const bool vec = a.D % 8 == 0 && (a.interleaved || a.pairs % 8 == 0) &&
                   rows(a.x, a.ldt, a.ldh) && rows(a.y, a.ldyt, a.ldyh);
  if (a.bf16) {
    if (a.interleaved) return vec ? go(rotary_kernel<true, true, true>) : go(rotary_kernel<true, false, true>);
    return vec ? go(rotary_kernel<true, true, false>) : go(rotary_kernel<true, false, false>);
  }
  if (a.interleaved) return vec ? go(rotary_kernel<false, true, true>) : go(rotary_kernel<false, false, true>);
  return vec ? go(rotary_kernel<false, true, false>) : go(rotary_kernel<false, false, false>);
}

}  // namespace puro
