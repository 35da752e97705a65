// gfx950 residual sum behind a block and the norm in front of the next one, in one pass: forward (the norm as a tensor, as
// 1x128 FP8 codes, as 1x128 and transposed 128x1 codes) and backward.
//
// Mathematics, for a row h of the residual stream and a row b of the block's output, C columns each (norm: as norm.hip,
// layer or RMS, without weight and bias):
//   p = b, or norm(b) w_post;   h' = h + scale gate p  (rounded to its type);   y = norm(h') w + bias
//   backward, from dy and the gradient dh' that the residual stream brings:
//   D = (the norm's backward pass of dy at h') + dh';  dh = D;  dw = sum_t dy xh,  dbias = sum_t dy
//   u = D scale gate w_post:  db = u, or the backward pass of u at b
//   With q = b or norm(b), one column sum S = sum_t D q serves both vectors:  dgate = scale w_post S,  dw_post = scale gate S.
// The norm is that of h' as it is stored, so y is what the norm alone gives for it, bit for bit, and the backward pass, which
// reads h', sees the same numbers.  All of it is bound by HBM: each input is read once and each output written once, a row
// stays in registers between its statistics and its use, a thread keeps the same columns for all its rows.
// Statistics and sums are fp32, as in norm.hip; D stays fp32 on its way into db.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"
#include "rows.hpp"

#include <algorithm>
#include <type_traits>

namespace puro {

namespace {

// ---------------------------------------------------------------------------------------------------
// Forward.  Teams, columns and rows as in norm_kernel, and the sums over h' in its order.
// WHAT: 0 y, 1 codes and scales, 2 h' and the statistics alone (first launch of the dual form).
// FULL: with a gate or a norm of b (their product with the scale is one vector); else the scale alone.
// Measured, bf16 RMS, us: 16384 x 2048 y 44.5 (6.0 TB/s; three sets of inputs and two of outputs in turn), h' and statistics
// 33 and the codes of both orientations 23 more; one row 4 in a graph: two sums' chains and one trip to memory; 4000 x 8192
// 59, 2000 x 16384 66 with gate and norm.  1027 x 1000 fp32 with gate and both norms, layer, 7.7: load_vec8 chooses type,
// alignment and end at run time, and each of its branches waits for what was loaded before, so that four vectors of two chunks
// are eight trips to memory, one behind the other.
// ---------------------------------------------------------------------------------------------------
template <bool BF16, bool VEC, int LPR, int ITER, int WHAT, bool FULL>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void residual_kernel(ResidualArgs a) {
  constexpr int kThreads = LPR > 256 ? LPR : 256;
  constexpr int kWaves = kThreads / 64;
  constexpr int kTeams = kThreads / LPR;
  __shared__ float red[2][kWaves];
  const NormArgs& n = a.n;
  const int team = threadIdx.x / LPR;
  const int tt = threadIdx.x % LPR;
  const int64_t row0 = ((int64_t)blockIdx.x * kTeams + team) * n.rows_per_team;
  const bool post = FULL && a.post != nullptr;

  int col[ITER], nv[ITER];
  float g[ITER][8], b[ITER][8], f[FULL ? ITER : 1][8];
  Raw8<BF16> nb[ITER], nh[ITER];
  auto load = [&](int64_t row, auto past) {
    constexpr bool NT = decltype(past)::value;
    const bool ok = row < n.T;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      nb[i] = load8<BF16, VEC, NT>(a.b, row * a.ldb + col[i], ok ? nv[i] : 0);
      nh[i] = load8<BF16, VEC, NT>(a.h, row * a.ldh + col[i], ok ? nv[i] : 0);
    }
  };
  auto fetch = [&](int64_t row) {
    if (VEC && a.stream) {
      apart();
      load(row, std::integral_constant<bool, VEC>());
      apart();
    } else {
      load(row, std::false_type());
    }
  };
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = n.C - col[i] < 0 ? 0 : (n.C - col[i] > 8 ? 8 : n.C - col[i]);
  }
  // (the widest class has no registers for a row ahead)
  constexpr bool kAhead = ITER < 4;
  if (kAhead) fetch(row0);
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if constexpr (WHAT != 2) {
      load_vec8(n.gamma, n.w_bf16, aligned16(n.gamma), col[i], nv[i], g[i]);
      load_vec8(n.beta, n.w_bf16, aligned16(n.beta), col[i], n.beta ? nv[i] : 0, b[i]);
    }
    if constexpr (FULL) {
      // a column that does not exist has the factor 0
      float w[8];
      load_vec8(a.gate, n.w_bf16, aligned16(a.gate), col[i], a.gate ? nv[i] : 0, f[i]);
      load_vec8(a.post, n.w_bf16, aligned16(a.post), col[i], a.post ? nv[i] : 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float one = j < nv[i] ? 1.f : 0.f;
        f[i][j] = a.scale * (a.gate ? f[i][j] : one) * (a.post ? w[j] : one);
      }
    }
  }
  const float inv_c = 1.0f / (float)n.C;
  int slot = 0;   // the LDS rows of the sums are taken in turn
  auto sum_of = [&](float v) {
    const float s = team_sum<LPR, kWaves>(v, red, slot);
    slot ^= 1;
    return s;
  };

  for (int k = 0; k < n.rows_per_team; ++k) {
    const int64_t row = row0 + k;
    const bool ok = row < n.T;
    float v[ITER][8];
    Raw8<BF16> hh[ITER];
    if (!kAhead) fetch(row);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      unpack8<BF16, VEC>(nb[i], nv[i], v[i]);
      hh[i] = nh[i];
    }
    if (kAhead && k + 1 < n.rows_per_team) fetch(row + 1);
    if (post) {
      float mean = 0.f;
      if (n.layer) mean = sum_of(lane_sum(v)) * inv_c;
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] -= mean;
      const float rstd = 1.0f / __builtin_sqrtf(sum_of(lane_squares<VEC>(v, nv)) * inv_c + n.eps);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
      if (ok && tt == 0) {
        if (a.post_mean) a.post_mean[row] = mean;
        if (a.post_rstd) a.post_rstd[row] = rstd;
      }
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float h[8];
      unpack8<BF16, VEC>(hh[i], nv[i], h);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = __builtin_fmaf(FULL ? f[FULL ? i : 0][j] : a.scale, v[i][j], h[j]);
      const Raw8<BF16> o = pack8<BF16>(h);
      if (BF16 && VEC && WHAT != 2 && !a.stream) {
        apart();
        store_raw8<BF16, VEC, VEC>(a.h_out, row * n.ldx + col[i], ok ? nv[i] : 0, o);
        apart();
      } else {
        store_raw8<BF16, VEC, false>(a.h_out, row * n.ldx + col[i], ok ? nv[i] : 0, o);
      }
      unpack8<BF16, true>(o, 8, v[i]);
    }
    float mean = 0.f;
    if (n.layer) mean = sum_of(lane_sum(v)) * inv_c;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] -= mean;
    const float rstd = 1.0f / __builtin_sqrtf(sum_of(lane_squares<VEC>(v, nv)) * inv_c + n.eps);
    if (ok && tt == 0) {
      if (n.mean) n.mean[row] = mean;
      if (n.rstd) n.rstd[row] = rstd;
    }
    if constexpr (WHAT != 2) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float y[8];
        norm8(v[i], rstd, g[i], b[i], y);
        if constexpr (WHAT == 0)
          store8<BF16, VEC, true>(n.y, row * n.ldy + col[i], ok ? nv[i] : 0, y);
        else if constexpr (VEC)
          store_codes8(n.q + row * n.ldq + col[i], n.s + (int64_t)(col[i] >> 7) * n.T + row, ok && nv[i] > 0, (tt & 15) == 0, y);
      }
    }
  }
}

template <bool BF16, bool VEC, int WHAT, bool FULL>
hipError_t launch_fwd(ResidualArgs a, hipStream_t st) {
  // lanes and rows per team by the rules of norm.hip's launch_fwd (its sums' order is this one's)
  auto go = [&](auto kernel, int lpr) {
    const int threads = lpr > 256 ? lpr : 256, teams = threads / lpr;
    int64_t r = std::max<int64_t>(1, std::min<int64_t>(4, a.n.T / (131072 / lpr)));
    const int64_t most = 0xFFFFFFFFll / threads * teams;
    r = std::max(r, (a.n.T + most - 1) / most);
    if (r > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    a.n.rows_per_team = (int)r;
    const int64_t blocks = (a.n.T + teams * r - 1) / (teams * r);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
    return hipGetLastError();
  };
  const int C = a.n.C;
  if (C <= 128) return go(residual_kernel<BF16, VEC, 16, 1, WHAT, FULL>, 16);
  if (C <= 256) return go(residual_kernel<BF16, VEC, 32, 1, WHAT, FULL>, 32);
  if (C <= 512) return go(residual_kernel<BF16, VEC, 64, 1, WHAT, FULL>, 64);
  if (C <= 1024) return go(residual_kernel<BF16, VEC, 64, 2, WHAT, FULL>, 64);
  if (C <= 2048) return go(residual_kernel<BF16, VEC, 128, 2, WHAT, FULL>, 128);
  if (C <= 4096) return go(residual_kernel<BF16, VEC, 256, 2, WHAT, FULL>, 256);
  if (C <= 8192) return go(residual_kernel<BF16, VEC, 512, 2, WHAT, FULL>, 512);
  return go(residual_kernel<BF16, VEC, 512, 4, WHAT, FULL>, 512);
}

template <bool BF16, bool VEC, int WHAT>
hipError_t launch_fwd(const ResidualArgs& a, hipStream_t st) {
  return a.gate || a.post ? launch_fwd<BF16, VEC, WHAT, true>(a, st) : launch_fwd<BF16, VEC, WHAT, false>(a, st);
}

}  // namespace

// Whether a call that moves `passes` times T C elements reads past the caches and leaves them to what it writes; the
// others write past them (bf16; fp32 rows are written through them at any size), which leaves what they read where it is.  The
// border, half the memory-side cache, is where the sides meet: us, 2048 columns bf16, three sets of inputs and two of outputs in turn, without - writing past - reading past:
//   forward (4 passes)       4096 rows 12.6 - 12.5 - 15.5, 8192 26.1 - 22.1 - 24.2, 12288 38.2 - 39.6 - 36.4, 16384 54.3 - 53.7 - 44.5
//   backward (4)             4096 rows 16.4 - 16.0 - 19.2, 8192 28.3 - 28.4 - 29.9, 12288 41.8 - 40.8 - 40.2, 16384 52.6 - 51.5 - 50.5
//   with gate and norm (6)   4096 rows 27.1 - 25.7 - 29.5, 8192 47.4 - 45.9 - 44.5, 12288 65.3 - 63.6 - 59.1, 16384 84.6 - 81.1 - 74.5
// fp32, which only reads past them, without - reading past: forward 4096 rows 26.0 - 28.1, 6144 41.7 - 38.5, 8192 53.8 - 49.7, 16384
// 100.9 - 105.8; backward 29.1 - 31.6, 42.9 - 43.1, 54.2 - 54.6, 103.9 - 99.6; with gate and norm 44.3 - 48.7, 62.2 - 67.3, 85.0 - 85.5,
// 158.0 - 155.4: there the sides meet at twice the border.
// Outputs that alone fill the cache go past it too (bf16): 32768 rows with gate and norm 157 - 153 - 151, both 145.
bool beyond_cache(int64_t T, int64_t C, int64_t es, int passes) {
  return T > kMemorySideCache / 2 / (C * es * passes);
}

hipError_t launch_residual(ResidualArgs a, hipStream_t st) {
  const int64_t es = a.n.x_bf16 ? 2 : 4;
  a.stream = beyond_cache(a.n.T, a.n.C, es, 4);
  const bool vec = a.n.C % 8 == 0 && vec_row(a.h, a.ldh, es) && vec_row(a.b, a.ldb, es) && vec_row(a.h_out, a.n.ldx, es) &&
                   vec_row(a.n.y, a.n.ldy, es);
  if (a.n.x_bf16) return vec ? launch_fwd<true, true, 0>(a, st) : launch_fwd<true, false, 0>(a, st);
  return vec ? launch_fwd<false, true, 0>(a, st) : launch_fwd<false, false, 0>(a, st);
}

hipError_t launch_residual_quant(ResidualArgs a, hipStream_t st) {
  a.stream = beyond_cache(a.n.T, a.n.C, a.n.x_bf16 ? 2 : 4, 4);
  return a.n.x_bf16 ? launch_fwd<true, true, 1>(a, st) : launch_fwd<false, true, 1>(a, st);
}

hipError_t launch_residual_quant_dual(ResidualArgs a, hipStream_t st) {
  a.stream = beyond_cache(a.n.T, a.n.C, a.n.x_bf16 ? 2 : 4, 5);   // (read again, and the codes)
  const hipError_t e = a.n.x_bf16 ? launch_fwd<true, true, 2>(a, st) : launch_fwd<false, true, 2>(a, st);
  return e != hipSuccess ? e : launch_norm_tiles(a.n, st);
}

}  // namespace puro
