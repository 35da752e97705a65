// gfx950 residual sum and norm: the backward pass (mathematics at the head of residual.hip).
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"
#include "rows.hpp"

#include <algorithm>
#include <type_traits>

namespace puro {

namespace {

// ---------------------------------------------------------------------------------------------------
// Backward.  As norm_bwd_kernel: eight waves per workgroup, teams of LPR lanes with a row each, the column sums of a
// thread's columns in registers over the team's rows (in runs of 64, added up in LDS), then over the teams, then written as
// the workgroup's partial sums and joined in order by a second launch.  FULL: with a gate or a norm of b: one more input and
// output, a second pair of row sums (b's norm) and the column sum S.
// Measured, 16384 x 2048 bf16 RMS, three sets of inputs and two of outputs in turn: 50.7 us with the joining (4 of them; 5.3
// TB/s), FULL 74.5 (5.4 TB/s): 565 vector instructions a row and wave keep the vector units 43% busy at two waves per SIMD,
// which meet at the sums' barriers.
// FULL of 4097 to 8192 columns (a workgroup to a row) keeps the weight and b's factor in LDS, so that nothing spills: a spilled
// register's reload waits for the row that is loaded ahead.  4000 x 8192: 85 us.
// Beyond 8192 columns the first and the last column sum stay in LDS and take a row at a time (128 KB at 16384 columns; up to
// 12288 the weight too), and no row is loaded ahead (loading ahead: 2667 x 12288 bf16 70.5 us, FULL 111.6).  With every sum in
// registers, which spilled, and without in turn, with a scale (dx is one output more): 2667 x 12288 bf16 91.0 and 70.4 us, FULL 199.2 and 101.5; 2000 x 16384 92.5
// and 73.2, FULL 186.5 and 154.2 (fp32 294 and 291: FULL at that width still spills 60 to 280 bytes a lane).
// Both have no room for runs: their launches have a workgroup for every 64 rows.
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
  constexpr bool kWide = ITER > 2;                                // sums in LDS
  constexpr bool kLds = FULL && LPR == kBwdThreads && !kWide;     // vectors in LDS
  constexpr bool kRuns = !kLds && !kWide;
  constexpr bool kWeightAgain = FULL && ITER > 3;                 // the weight is read again for each row
  constexpr bool kWeightLds = kLds || (kWide && ITER < 4);
  __shared__ float red[2][2][kBwdWaves];
  __shared__ __attribute__((aligned(16))) float join[kSums][kRuns ? kTeams * kWidth : 4];
  __shared__ __attribute__((aligned(16))) float weights[kWeightLds ? kWidth : 4];
  __shared__ __attribute__((aligned(16))) float factors[kLds ? kWidth : 4];       // of b
  __shared__ __attribute__((aligned(16))) float held[2][kWide ? kWidth : 4];      // the first sum, the last
  const int team = threadIdx.x / LPR;
  const int tt = threadIdx.x % LPR;
  const int64_t stride = (int64_t)gridDim.x * kTeams;
  const bool post = FULL && a.post != nullptr;

  int col[ITER], nv[ITER];
  float g[kWeightLds || kWeightAgain ? 1 : ITER][8], f[FULL && !kLds ? ITER : 1][8], sum[kSums][ITER][8];
  auto in_lds = [](int which) { return kWide && (which == 0 || which == kSums - 1); };
  // eight values at a thread's place in LDS (no other thread touches them)
  auto to_lds = [&](float* base, const float (&v)[8]) {
    reinterpret_cast<f32x4*>(base)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(base)[1] = f32x4{v[4], v[5], v[6], v[7]};
  };
  auto from_lds = [&](const float* base, float (&v)[8]) {
    const f32x4* p = reinterpret_cast<const f32x4*>(base);
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = lo[j];
      v[j + 4] = hi[j];
    }
  };
  auto vector_of = [&](int which, int i, float (&v)[8]) {
    if (which == 0 && kWeightAgain) {
      int c = col[i];
      asm volatile("" : "+v"(c));   // or the load moves before the loop, and its registers are spilled
      load_vec8(a.gamma, a.w_bf16, aligned16(a.gamma), c, nv[i], v);
    } else if (which == 0 ? kWeightLds : kLds) {
      from_lds((which == 0 ? weights : factors) + col[i], v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = which == 0 ? g[kWeightLds || kWeightAgain ? 0 : i][j] : f[FULL && !kLds ? i : 0][j];
    }
  };
  // a sum of a thread's eight columns, to be added to and put back
  auto sum_of = [&](int which, int i, float (&v)[8]) {
    if (in_lds(which)) {
      from_lds(held[which != 0] + col[i], v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sum[which][i][j];
    }
  };
  auto keep_sum = [&](int which, int i, const float (&v)[8]) {
    if (in_lds(which)) {
      to_lds(held[which != 0] + col[i], v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[which][i][j] = v[j];
    }
  };
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = a.C - col[i] < 0 ? 0 : (a.C - col[i] > 8 ? 8 : a.C - col[i]);
    if constexpr (!kWeightAgain) {
      float (&gi)[8] = g[kWeightLds ? 0 : i];
      load_vec8(a.gamma, a.w_bf16, aligned16(a.gamma), col[i], nv[i], gi);
      if constexpr (kWeightLds) to_lds(weights + col[i], gi);
    }
    if constexpr (FULL) {
      float (&fi)[8] = f[kLds ? 0 : i];
      float w[8];
      load_vec8(a.gate, a.w_bf16, aligned16(a.gate), col[i], a.gate ? nv[i] : 0, fi);
      load_vec8(a.post, a.w_bf16, aligned16(a.post), col[i], a.post ? nv[i] : 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float one = j < nv[i] ? 1.f : 0.f;
        fi[j] = a.scale * (a.gate ? fi[j] : one) * (a.post ? w[j] : one);
      }
      if constexpr (kLds) to_lds(factors + col[i], fi);
    }
    const float none[8] = {};
#pragma unroll
    for (int s = 0; s < kSums; ++s) keep_sum(s, i, none);
  }
  const float inv_c = 1.0f / (float)a.C;
  int64_t row = (int64_t)blockIdx.x * kTeams + team;

  // what a row needs first, and what it needs behind its first sums
  struct First {
    Raw8<BF16> y[ITER], h[ITER];
    float mean, rstd;
  } n1;
  struct Second {
    Raw8<BF16> o[ITER], b[FULL ? ITER : 1];
    float mean, rstd;
  } n2;
  auto load1 = [&](int64_t r, auto past) {
    constexpr bool NT = decltype(past)::value;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      n1.y[i] = load8<BF16, VEC, NT>(a.dy, r * a.lddy + col[i], r < a.T ? nv[i] : 0);
      n1.h[i] = load8<BF16, VEC, NT>(a.h, r * a.ldh + col[i], r < a.T ? nv[i] : 0);
    }
  };
  auto load2 = [&](int64_t r, auto past) {
    constexpr bool NT = decltype(past)::value;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      n2.o[i] = load8<BF16, VEC, NT>(a.dho, r * a.lddho + col[i], r < a.T && a.dho ? nv[i] : 0);
      if constexpr (FULL) n2.b[i] = load8<BF16, VEC, NT>(a.b, r * a.ldb + col[i], r < a.T ? nv[i] : 0);
    }
  };
  auto fetch = [&](int64_t r, auto load) {
    if (VEC && a.stream) {
      apart();
      load(r, std::integral_constant<bool, VEC>());
      apart();
    } else {
      load(r, std::false_type());
    }
  };
  auto fetch1 = [&](int64_t r) {
    fetch(r, load1);
    n1.mean = r < a.T && a.layer ? a.mean[r] : 0.f;
    n1.rstd = r < a.T ? a.rstd[r] : 0.f;
  };
  auto fetch2 = [&](int64_t r) {
    fetch(r, load2);
    n2.mean = r < a.T && post && a.layer ? a.post_mean[r] : 0.f;
    n2.rstd = r < a.T && post ? a.post_rstd[r] : 0.f;
  };
  // a thread's eight sums at its place in LDS, set or added to (no other thread touches it before the join)
  auto put = [&](int which, int i, const float (&v)[8], bool add) {
    f32x4* p = reinterpret_cast<f32x4*>(join[which] + team * kWidth + col[i]);
    const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    p[0] = add ? p[0] + lo : lo;
    p[1] = add ? p[1] + hi : hi;
  };
  auto store = [&](void* base, int64_t at, int n, const float (&v)[8]) {
    if (BF16 && VEC && a.past) {
      apart();
      store8<BF16, VEC, VEC>(base, at, n, v);
      apart();
    } else {
      store8<BF16, VEC, false>(base, at, n, v);
    }
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

  // The next row is loaded ahead, as far as there are registers: none beyond 8192 columns; of four fp32 or unaligned rows the
  // two needed first (8192 x 2047 bf16 56.0 us, 59.9 with all; aligned 16384 x 2048 bf16 77.0 and 73.6 with all), the
  // others while those are worked on.
  constexpr bool kAhead1 = ITER < 3, kAhead2 = kAhead1 && ((BF16 && VEC) || !FULL);
  if (kAhead1) fetch1(row);
  if (kAhead2) fetch2(row);
  for (int k = 0; k < rows_per_team; ++k, row += stride) {
    const bool ok = row < a.T, more = k + 1 < rows_per_team;
    if (!kAhead1) fetch1(row);
    const First c1 = n1;
    Second c2;
    if (kAhead2) c2 = n2;
    // (loads return in order: this row's before the next one's)
    if (kAhead1 && !kAhead2) fetch2(row);
    if (kAhead1 && more) fetch1(row + stride);
    if (kAhead2 && more) fetch2(row + stride);
    float d[ITER][8], xh[ITER][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float w[8], q0[8], q1[8];
      vector_of(0, i, w);
      sum_of(0, i, q0);
      sum_of(1, i, q1);
      unpack8<BF16, VEC>(c1.h[i], nv[i], xh[i]);
      unpack8<BF16, VEC>(c1.y[i], nv[i], d[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // a column that does not exist has dy = 0 and weight 0: it adds nothing to any sum
        xh[i][j] = (xh[i][j] - c1.mean) * c1.rstd;
        q0[j] = __builtin_fmaf(d[i][j], xh[i][j], q0[j]);
        q1[j] += d[i][j];
        d[i][j] *= w[j];
        s1 += d[i][j];
        s2 = __builtin_fmaf(d[i][j], xh[i][j], s2);
      }
      keep_sum(0, i, q0);
      keep_sum(1, i, q1);
    }
    if (!kAhead1) fetch2(row);
    sums_of(s1, s2);
    if (!kAhead2) c2 = n2;
    float t1 = 0.f, t2 = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float o[8];
      unpack8<BF16, VEC>(c2.o[i], nv[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[i][j] = __builtin_fmaf(__builtin_fmaf(-xh[i][j], s2, d[i][j]) - s1, c1.rstd, o[j]);
      store(a.dh, row * a.lddh + col[i], ok ? nv[i] : 0, d[i]);
      if constexpr (FULL) {
        float w[8], q2[8];
        vector_of(1, i, w);
        sum_of(2, i, q2);
        unpack8<BF16, VEC>(c2.b[i], nv[i], xh[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (post) xh[i][j] = (xh[i][j] - c2.mean) * c2.rstd;
          // (behind the last column D holds -s1 rstd: its place of S is never written, and its factor is 0)
          q2[j] = __builtin_fmaf(d[i][j], xh[i][j], q2[j]);
          d[i][j] *= w[j];
          t1 += d[i][j];
          t2 = __builtin_fmaf(d[i][j], xh[i][j], t2);
        }
        keep_sum(2, i, q2);
      } else if (a.dx) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a.scale * d[i][j];
        store(a.dx, row * a.lddx + col[i], ok ? nv[i] : 0, v);
      }
    }
    if constexpr (FULL) {
      if (post) sums_of(t1, t2);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (post) {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[i][j] = (__builtin_fmaf(-xh[i][j], t2, d[i][j]) - t1) * c2.rstd;
        }
        store(a.dx, row * a.lddx + col[i], ok ? nv[i] : 0, d[i]);
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
      for (int i = 0; i < ITER; ++i) {
        float v[8];
        sum_of(which, i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float s = v[j];
          if constexpr (kRuns) {
            if (runs) s += join[which][col[i] + j];
          }
          if (j < nv[i]) out(which, col[i] + j, s);
        }
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
  else if (a.C <= 12288) e = go(residual_bwd_kernel<BF16, VEC, 512, 3, FULL>);
  else e = go(residual_bwd_kernel<BF16, VEC, 512, 4, FULL>);
  if (e != hipSuccess || blocks == 1) return e;
  constexpr int kSums = residual_bwd_sums(FULL);
  const int used = FULL ? kSums : a.dbeta ? 2 : 1;
  hipLaunchKernelGGL(residual_bwd_reduce_kernel, dim3((unsigned)((a.C + 15) / 16), used), dim3(256), 0, st, a, blocks, kSums);
  return hipGetLastError();
}

}  // namespace

// As norm_bwd_blocks, with a workgroup for every 64 rows at least where the kernel has no runs.
int residual_bwd_blocks(int64_t T, int64_t C, bool gated) {
  if (T <= 0 || C <= 0) return 0;
  const int64_t teams = kBwdThreads / bwd_lpr(C);
  constexpr int64_t kMost = (int64_t(1) << 32) / kBwdThreads - 1;
  if (T <= 2 * teams) return 1;
  if (C > (gated ? 4096 : 8192) && T > 256 * kRun) return (int)std::min<int64_t>((T + kRun - 1) / kRun, kMost);
  const int64_t round = (int64_t)kRun * kRun * 256 * teams;
  if (T > round) return (int)(256 * std::min<int64_t>((T + round - 1) / round, kMost / 256));
  return (int)std::min<int64_t>(std::min<int64_t>(256, (T + teams - 1) / teams), std::max<int64_t>(64, (T + 7) / 8));
}

hipError_t launch_residual_bwd(ResidualBwdArgs a, hipStream_t st) {
  if (a.T == 0 || a.C == 0) {
    if (a.accumulate || a.C == 0) return hipSuccess;
    hipLaunchKernelGGL(residual_zero_kernel, dim3((unsigned)((a.C + 255) / 256)), dim3(256), 0, st, a.dgamma, a.dbeta, a.dgate,
                       a.dpost, a.C);
    return hipGetLastError();
  }
  const int64_t es = a.x_bf16 ? 2 : 4;
  const bool full = a.gate || a.post;
  a.stream = beyond_cache(a.T, a.C, es, full ? 6 : a.dx ? 5 : 4);
  a.past = !a.stream || a.T >= kMemorySideCache / (a.C * es * (a.dx ? 2 : 1));
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
