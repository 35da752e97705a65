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

namespace puro {

namespace {

// ---------------------------------------------------------------------------------------------------
// Forward.  Teams, columns and rows as in norm_kernel, and the sums over h' in its order.
// WHAT: 0 y, 1 codes and scales, 2 h' and the statistics alone (first launch of the dual form).
// FULL: with a gate or a norm of b (their product with the scale is one vector); else the scale alone.
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
  auto fetch = [&](int64_t row) {
    const bool ok = row < n.T;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      nb[i] = load8<BF16, VEC>(a.b, row * a.ldb + col[i], ok ? nv[i] : 0);
      nh[i] = load8<BF16, VEC>(a.h, row * a.ldh + col[i], ok ? nv[i] : 0);
    }
  };
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = n.C - col[i] < 0 ? 0 : (n.C - col[i] > 8 ? 8 : n.C - col[i]);
  }
  fetch(row0);
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
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      unpack8<BF16, VEC>(nb[i], nv[i], v[i]);
      hh[i] = nh[i];
    }
    if (k + 1 < n.rows_per_team) fetch(row + 1);
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
      store_raw8<BF16, VEC, false>(a.h_out, row * n.ldx + col[i], ok ? nv[i] : 0, o);
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

// ---------------------------------------------------------------------------------------------------
// Backward.  As norm_bwd_kernel: eight waves per workgroup, teams of LPR lanes with a row each, the column sums of a
// thread's columns in registers over the team's rows (in runs of 64, added up in LDS), then over the teams, then written as
// the workgroup's partial sums and joined in order by a second launch.  FULL: with a gate or a norm of b: one more input and
// output, a second pair of row sums (b's norm) and the column sum S.
// The widest class (ITER 4) of FULL has no room in LDS for its runs: its launches have a workgroup for every 64 rows.
// ---------------------------------------------------------------------------------------------------
constexpr int kBwdThreads = 512;
constexpr int kRun = 64;               // rows a thread adds in order, and sums of such runs
constexpr int kBwdWaves = kBwdThreads / 64;

// An output of column c from its sum: the weight's gradient, the bias's, or S for the gate's and w_post's.
__device__ __forceinline__ void finish_sum(const ResidualBwdArgs& a, int which, int c, float s) {
  auto put = [&](float* out, float v) { out[c] = a.accumulate ? out[c] + v : v; };
  auto at = [&](const void* w) {
    return a.w_bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(w)[c] << 16) : static_cast<const float*>(w)[c];
  };
  if (which == 0) put(a.dgamma, s);
  if (which == 1 && a.dbeta) put(a.dbeta, s);
  if (which == 2) {
    if (a.dgate) put(a.dgate, a.scale * (a.post ? at(a.post) * s : s));
    if (a.dpost) put(a.dpost, a.scale * (a.gate ? at(a.gate) * s : s));
  }
}

template <bool BF16, bool VEC, int LPR, int ITER, bool FULL>
__global__ __launch_bounds__(kBwdThreads) void residual_bwd_kernel(ResidualBwdArgs a, int rows_per_team, bool direct) {
  constexpr int kTeams = kBwdThreads / LPR;
  constexpr int kWidth = 8 * LPR * ITER;
  constexpr int kSums = residual_bwd_sums(FULL);
  constexpr bool kRuns = !FULL || ITER < 4;
  __shared__ float red[2][2][kBwdWaves];
  __shared__ __attribute__((aligned(16))) float join[kSums][kRuns ? kTeams * kWidth : 4];
  const int team = threadIdx.x / LPR;
  const int tt = threadIdx.x % LPR;
  const int64_t stride = (int64_t)gridDim.x * kTeams;
  const bool post = FULL && a.post != nullptr;

  int col[ITER], nv[ITER];
  float g[ITER][8], f[FULL ? ITER : 1][8], sum[kSums][ITER][8];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = a.C - col[i] < 0 ? 0 : (a.C - col[i] > 8 ? 8 : a.C - col[i]);
    load_vec8(a.gamma, a.w_bf16, aligned16(a.gamma), col[i], nv[i], g[i]);
    if constexpr (FULL) {
      float w[8];
      load_vec8(a.gate, a.w_bf16, aligned16(a.gate), col[i], a.gate ? nv[i] : 0, f[i]);
      load_vec8(a.post, a.w_bf16, aligned16(a.post), col[i], a.post ? nv[i] : 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float one = j < nv[i] ? 1.f : 0.f;
        f[i][j] = a.scale * (a.gate ? f[i][j] : one) * (a.post ? w[j] : one);
      }
    }
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[s][i][j] = 0.f;
  }
  const float inv_c = 1.0f / (float)a.C;
  int64_t row = (int64_t)blockIdx.x * kTeams + team;

  struct Fetched {
    Raw8<BF16> y[ITER], h[ITER], o[ITER], b[FULL ? ITER : 1];
    float mean, rstd, pmean, prstd;
  } nx;
  auto fetch = [&](int64_t r) {
    const bool ok = r < a.T;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      nx.y[i] = load8<BF16, VEC>(a.dy, r * a.lddy + col[i], ok ? nv[i] : 0);
      nx.h[i] = load8<BF16, VEC>(a.h, r * a.ldh + col[i], ok ? nv[i] : 0);
      nx.o[i] = load8<BF16, VEC>(a.dho, r * a.lddho + col[i], ok && a.dho ? nv[i] : 0);
      if constexpr (FULL) nx.b[i] = load8<BF16, VEC>(a.b, r * a.ldb + col[i], ok ? nv[i] : 0);
    }
    nx.mean = ok && a.layer ? a.mean[r] : 0.f;
    nx.rstd = ok ? a.rstd[r] : 0.f;
    nx.pmean = ok && post && a.layer ? a.post_mean[r] : 0.f;
    nx.prstd = ok && post ? a.post_rstd[r] : 0.f;
  };
  // a thread's eight sums at its place in LDS, set or added to (no other thread touches it before the join)
  auto put = [&](int which, int i, const float (&v)[8], bool add) {
    f32x4* p = reinterpret_cast<f32x4*>(join[which] + team * kWidth + col[i]);
    const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    p[0] = add ? p[0] + lo : lo;
    p[1] = add ? p[1] + hi : hi;
  };
  int slot = 0;
  // both sums of a norm's backward pass over the team
  auto sums_of = [&](float& s1, float& s2) {
    s1 = lanes_sum<LPR>(s1);
    s2 = lanes_sum<LPR>(s2);
    if constexpr (LPR > 64) {
      constexpr int kTeamWaves = LPR / 64;
      if ((threadIdx.x & 63) == 0) {
        red[slot][0][threadIdx.x >> 6] = s1;
        red[slot][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < kTeamWaves; ++w) {
        s1 += red[slot][0][team * kTeamWaves + w];
        s2 += red[slot][1][team * kTeamWaves + w];
      }
      slot ^= 1;
    }
    s1 = a.layer ? s1 * inv_c : 0.f;
    s2 *= inv_c;
  };

  constexpr bool kAhead = ITER < 4;    // (the widest class has no registers for a row ahead)
  if (kAhead) fetch(row);
  for (int k = 0; k < rows_per_team; ++k, row += stride) {
    if (!kAhead) fetch(row);
    const bool ok = row < a.T;
    const Fetched cur = nx;
    if (kAhead && k + 1 < rows_per_team) fetch(row + stride);
    float d[ITER][8], xh[ITER][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      unpack8<BF16, VEC>(cur.h[i], nv[i], xh[i]);
      unpack8<BF16, VEC>(cur.y[i], nv[i], d[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // a column that does not exist has dy = 0 and weight 0: it adds nothing to any sum
        xh[i][j] = (xh[i][j] - cur.mean) * cur.rstd;
        sum[0][i][j] = __builtin_fmaf(d[i][j], xh[i][j], sum[0][i][j]);
        sum[1][i][j] += d[i][j];
        d[i][j] *= g[i][j];
        s1 += d[i][j];
        s2 = __builtin_fmaf(d[i][j], xh[i][j], s2);
      }
    }
    sums_of(s1, s2);
    float t1 = 0.f, t2 = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float o[8];
      unpack8<BF16, VEC>(cur.o[i], nv[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[i][j] = __builtin_fmaf(__builtin_fmaf(-xh[i][j], s2, d[i][j]) - s1, cur.rstd, o[j]);
      store8<BF16, VEC, false>(a.dh, row * a.lddh + col[i], ok ? nv[i] : 0, d[i]);
      if constexpr (FULL) {
        unpack8<BF16, VEC>(cur.b[i], nv[i], xh[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (post) xh[i][j] = (xh[i][j] - cur.pmean) * cur.prstd;
          // (behind the last column D holds -s1 rstd: its place of S is never written, and its factor is 0)
          sum[2][i][j] = __builtin_fmaf(d[i][j], xh[i][j], sum[2][i][j]);
          d[i][j] *= f[i][j];
          t1 += d[i][j];
          t2 = __builtin_fmaf(d[i][j], xh[i][j], t2);
        }
      } else if (a.dx) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a.scale * d[i][j];
        store8<BF16, VEC, false>(a.dx, row * a.lddx + col[i], ok ? nv[i] : 0, v);
      }
    }
    if constexpr (FULL) {
      if (post) sums_of(t1, t2);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (post) {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[i][j] = (__builtin_fmaf(-xh[i][j], t2, d[i][j]) - t1) * cur.prstd;
        }
        store8<BF16, VEC, false>(a.dx, row * a.lddx + col[i], ok ? nv[i] : 0, d[i]);
      }
    }
    if constexpr (kRuns) {
      if (k % kRun == kRun - 1 && k + 1 < rows_per_team) {   // a run is full, and another one follows
#pragma unroll
        for (int s = 0; s < kSums; ++s)
#pragma unroll
          for (int i = 0; i < ITER; ++i) {
            put(s, i, sum[s][i], k >= kRun);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[s][i][j] = 0.f;
          }
      }
    }
  }

  // the workgroup's sums
  const bool runs = kRuns && rows_per_team > kRun;
  auto out = [&](int which, int c, float s) {
    if (direct)
      finish_sum(a, which, c, s);
    else
      a.partial[((int64_t)blockIdx.x * kSums + which) * a.C + c] = s;
  };
#pragma unroll
  for (int which = 0; which < kSums; ++which) {
    if (which == 1 && a.dbeta == nullptr) continue;
    if constexpr (kTeams > 1) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) put(which, i, sum[which][i], runs);
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += kBwdThreads) {
        float s = join[which][c];
#pragma unroll
        for (int w = 1; w < kTeams; ++w) s += join[which][w * kWidth + c];
        out(which, c, s);
      }
    } else {
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float s = sum[which][i][j];
          if constexpr (kRuns) {
            if (runs) s += join[which][col[i] + j];
          }
          if (j < nv[i]) out(which, col[i] + j, s);
        }
    }
  }
}

// The column sums over the workgroups' partials: 16 columns x 16 runs of workgroups per workgroup, the runs joined in
// order.  (More than 256 partials are added in 64 bits 16 at a time.)
__global__ __launch_bounds__(256) void residual_bwd_reduce_kernel(ResidualBwdArgs a, int blocks, int sums) {
  __shared__ float part[16][17];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cx;
  const int which = blockIdx.y;
  if (which == 1 && a.dbeta == nullptr) return;
  double sum = 0.0;
  if (c < a.C)
    for (int b0 = ry; b0 < blocks; b0 += 256) {
      float v[16], s = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        v[k] = b0 + 16 * k < blocks ? a.partial[((int64_t)(b0 + 16 * k) * sums + which) * a.C + c] : 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += v[k];
      sum += (double)s;
    }
  float s = (float)sum;
  part[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < a.C) {
#pragma unroll
    for (int r = 1; r < 16; ++r) s += part[r][cx];
    finish_sum(a, which, c, s);
  }
}

__global__ __launch_bounds__(256) void residual_zero_kernel(float* dgamma, float* dbeta, float* dgate, float* dpost, int C) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  dgamma[c] = 0.f;
  if (dbeta) dbeta[c] = 0.f;
  if (dgate) dgate[c] = 0.f;
  if (dpost) dpost[c] = 0.f;
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

// lanes per row of the backward kernel; it takes kBwdThreads / this rows per workgroup and step
int bwd_lpr(int64_t C) {
  return C <= 128 ? 16 : C <= 256 ? 32 : C <= 1024 ? 64 : C <= 2048 ? 128 : C <= 4096 ? 256 : 512;
}

template <bool BF16, bool VEC, bool FULL>
hipError_t launch_bwd(const ResidualBwdArgs& a, hipStream_t st) {
  const int blocks = residual_bwd_blocks(a.T, a.C, FULL);
  const int teams = kBwdThreads / bwd_lpr(a.C);
  const int64_t rows = (a.T + (int64_t)blocks * teams - 1) / ((int64_t)blocks * teams);
  if (rows > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBwdThreads), 0, st, a, (int)rows, blocks == 1);
    return hipGetLastError();
  };
  hipError_t e;
  if (a.C <= 128) e = go(residual_bwd_kernel<BF16, VEC, 16, 1, FULL>);
  else if (a.C <= 256) e = go(residual_bwd_kernel<BF16, VEC, 32, 1, FULL>);
  else if (a.C <= 512) e = go(residual_bwd_kernel<BF16, VEC, 64, 1, FULL>);
  else if (a.C <= 1024) e = go(residual_bwd_kernel<BF16, VEC, 64, 2, FULL>);
  else if (a.C <= 2048) e = go(residual_bwd_kernel<BF16, VEC, 128, 2, FULL>);
  else if (a.C <= 4096) e = go(residual_bwd_kernel<BF16, VEC, 256, 2, FULL>);
  else if (a.C <= 8192) e = go(residual_bwd_kernel<BF16, VEC, 512, 2, FULL>);
  else e = go(residual_bwd_kernel<BF16, VEC, 512, 4, FULL>);
  if (e != hipSuccess || blocks == 1) return e;
  constexpr int kSums = residual_bwd_sums(FULL);
  const int used = FULL ? kSums : a.dbeta ? 2 : 1;
  hipLaunchKernelGGL(residual_bwd_reduce_kernel, dim3((unsigned)((a.C + 15) / 16), used), dim3(256), 0, st, a, blocks, kSums);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_residual(ResidualArgs a, hipStream_t st) {
  const int64_t es = a.n.x_bf16 ? 2 : 4;
  const bool vec = a.n.C % 8 == 0 && vec_row(a.h, a.ldh, es) && vec_row(a.b, a.ldb, es) && vec_row(a.h_out, a.n.ldx, es) &&
                   vec_row(a.n.y, a.n.ldy, es);
  if (a.n.x_bf16) return vec ? launch_fwd<true, true, 0>(a, st) : launch_fwd<true, false, 0>(a, st);
  return vec ? launch_fwd<false, true, 0>(a, st) : launch_fwd<false, false, 0>(a, st);
}

hipError_t launch_residual_quant(ResidualArgs a, hipStream_t st) {
  return a.n.x_bf16 ? launch_fwd<true, true, 1>(a, st) : launch_fwd<false, true, 1>(a, st);
}

hipError_t launch_residual_quant_dual(ResidualArgs a, hipStream_t st) {
  const hipError_t e = a.n.x_bf16 ? launch_fwd<true, true, 2>(a, st) : launch_fwd<false, true, 2>(a, st);
  return e != hipSuccess ? e : launch_norm_tiles(a.n, st);
}

// As norm_bwd_blocks, with a workgroup for every 64 rows at least where the kernel has no runs.
int residual_bwd_blocks(int64_t T, int64_t C, bool gated) {
  if (T <= 0 || C <= 0) return 0;
  const int64_t teams = kBwdThreads / bwd_lpr(C);
  constexpr int64_t kMost = (int64_t(1) << 32) / kBwdThreads - 1;
  if (T <= 2 * teams) return 1;
  if (gated && C > 8192 && T > 256 * kRun) return (int)std::min<int64_t>((T + kRun - 1) / kRun, kMost);
  const int64_t round = (int64_t)kRun * kRun * 256 * teams;
  if (T > round) return (int)(256 * std::min<int64_t>((T + round - 1) / round, kMost / 256));
  return (int)std::min<int64_t>(std::min<int64_t>(256, (T + teams - 1) / teams), std::max<int64_t>(64, (T + 7) / 8));
}

hipError_t launch_residual_bwd(const ResidualBwdArgs& a, hipStream_t st) {
  if (a.T == 0 || a.C == 0) {
    if (a.accumulate || a.C == 0) return hipSuccess;
    hipLaunchKernelGGL(residual_zero_kernel, dim3((unsigned)((a.C + 255) / 256)), dim3(256), 0, st, a.dgamma, a.dbeta, a.dgate,
                       a.dpost, a.C);
    return hipGetLastError();
  }
  const int64_t es = a.x_bf16 ? 2 : 4;
  const bool full = a.gate || a.post;
  const bool vec = a.C % 8 == 0 && vec_row(a.dy, a.lddy, es) && vec_row(a.h, a.ldh, es) &&
                   (!a.dho || vec_row(a.dho, a.lddho, es)) && (!full || vec_row(a.b, a.ldb, es)) &&
                   vec_row(a.dh, a.lddh, es) && (!a.dx || vec_row(a.dx, a.lddx, es));
  if (a.x_bf16) {
    if (full) return vec ? launch_bwd<true, true, true>(a, st) : launch_bwd<true, false, true>(a, st);
    return vec ? launch_bwd<true, true, false>(a, st) : launch_bwd<true, false, false>(a, st);
  }
  if (full) return vec ? launch_bwd<false, true, true>(a, st) : launch_bwd<false, false, true>(a, st);
  return vec ? launch_bwd<false, true, false>(a, st) : launch_bwd<false, false, false>(a, st);
}

}  // namespace puro
