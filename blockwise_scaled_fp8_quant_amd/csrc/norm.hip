// gfx950 layer / RMS norm: forward (as a tensor, as 1x128 FP8 codes, as 1x128 and transposed 128x1
// codes) and backward with the reduction of the weight's and bias's gradient.
//
// Mathematics, for a row x of C columns:
//   mu = mean(x) (RMS: 0),  r = 1 / sqrt(mean((x - mu)^2) + eps),  xh = (x - mu) r,  y = xh g + b
//   u = dy g:  dx = r (u - mean(u) - xh mean(u xh)) (RMS: without mean(u));  dg = sum_t dy xh;  db = sum_t dy
// All of it is bound by HBM: one read of x (and dy) and one write.  A row is therefore held in
// registers between its statistics and its use, and a thread keeps the same columns for every row it
// takes, so the weight, the bias and the weight gradient's sums stay in registers too.
//
// Statistics are fp32: a thread adds its at most 32 values of the row in order, then the lanes and waves are joined
// in a tree; the variance is the mean square of the differences from the mean.  y, dx are rounded
// once.  dg and db are summed in fp32 in short runs: at most 64 rows in order per thread, at most 64 such sums, then
// teams and workgroups in a fixed order (norm_bwd_kernel): the error does not grow with T.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"
#include "rows.hpp"

#include <algorithm>

namespace puro {

namespace {

// ---------------------------------------------------------------------------------------------------
// Forward.  A team of LPR lanes takes a row (16 lanes, so that a wave takes four short rows, up to eight waves), each
// lane ITER chunks of eight columns, chunk i of team lane t at column 8 (LPR i + t): 16-byte loads that are
// contiguous over a team, and 16 lanes hold one 128-column group.  A team takes rows_per_team consecutive rows and loads the
// next one before it works on the present one.
// WHAT: 0 y, 1 codes and scales, 2 the statistics alone (first launch of the dual form).
// Measured, 16384 x 2048 bf16: y 23.0 us (5.8 TB/s, a copy's rate), the statistics 12.0 (5.6 TB/s read); one row 2.9 us, its
// two sums' chains and one trip to memory.  Two chunks per lane: with four (64 lanes a row) 168 registers leave three waves
// per SIMD, 24.4 us.
// ---------------------------------------------------------------------------------------------------
template <bool BF16, bool VEC, int LPR, int ITER, int WHAT>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void norm_kernel(NormArgs a) {
  constexpr int kThreads = LPR > 256 ? LPR : 256;
  constexpr int kWaves = kThreads / 64;
  constexpr int kTeams = kThreads / LPR;
  __shared__ float red[2][kWaves];
  const int team = threadIdx.x / LPR;
  const int tt = threadIdx.x % LPR;
  const int64_t row0 = ((int64_t)blockIdx.x * kTeams + team) * a.rows_per_team;

  int col[ITER], nv[ITER];
  float g[ITER][8], b[ITER][8];
  Raw8<BF16> next[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = a.C - col[i] < 0 ? 0 : (a.C - col[i] > 8 ? 8 : a.C - col[i]);
    next[i] = load8<BF16, VEC>(a.x, row0 * a.ldx + col[i], row0 < a.T ? nv[i] : 0);
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if constexpr (WHAT != 2) {
      load_vec8(a.gamma, a.w_bf16, aligned16(a.gamma), col[i], nv[i], g[i]);
      load_vec8(a.beta, a.w_bf16, aligned16(a.beta), col[i], a.beta ? nv[i] : 0, b[i]);
    }
  }
  const float inv_c = 1.0f / (float)a.C;

  for (int k = 0; k < a.rows_per_team; ++k) {
    const int64_t row = row0 + k;
    const bool ok = row < a.T;
    float v[ITER][8];
#pragma unroll
    for (int i = 0; i < ITER; ++i) unpack8<BF16, VEC>(next[i], nv[i], v[i]);
    if (k + 1 < a.rows_per_team) {
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        next[i] = load8<BF16, VEC>(a.x, (row + 1) * a.ldx + col[i], row + 1 < a.T ? nv[i] : 0);
    }
    float mean = 0.f;
    if (a.layer) mean = team_sum<LPR, kWaves>(lane_sum(v), red, 0) * inv_c;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] -= mean;
    const float sq = lane_squares<VEC>(v, nv);
    // (an RMS norm has this sum alone, so it takes the LDS rows in turn from row to row)
    const float rstd =
        1.0f / __builtin_sqrtf(team_sum<LPR, kWaves>(sq, red, a.layer ? 1 : (k & 1)) * inv_c + a.eps);
    if (ok && tt == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if constexpr (WHAT != 2) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float y[8];
        norm8(v[i], rstd, g[i], b[i], y);
        if constexpr (WHAT == 0) {
          store8<BF16, VEC, true>(a.y, row * a.ldy + col[i], ok ? nv[i] : 0, y);
        } else if constexpr (VEC) {
          store_codes8(a.q + row * a.ldq + col[i], a.s + (int64_t)(col[i] >> 7) * a.T + row, ok && nv[i] > 0, (tt & 15) == 0, y);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------------
// Second launch of the dual form: a 128-row x 128-column tile per workgroup, as quant_dual_kernel
// (quant.hip) on the norm formed in registers from x and the statistics of the first launch.  x is
// read twice (once per launch): keeping 128 whole rows on one CU for a single read does not fit
// beyond a few hundred columns.
// Measured at 16384 x 2048 bf16: 23.5 us (5.6 TB/s of reads and writes together, as a copy).  It was bound by
// vector instructions first (18 us with neither loads nor stores): three-operand maxima on magnitudes, converts
// without a register to clear and a norm of two instructions (three with a mean) took it from 27.6 us.
// ---------------------------------------------------------------------------------------------------
constexpr int kDualThreads = 256;

template <bool BF16, bool LAYER>
__global__ __launch_bounds__(kDualThreads) void norm_dual_kernel(NormArgs a, int bt_log2) {
  constexpr int kWaves = kDualThreads / 64;
  constexpr int kRows = 128 * 16 / kDualThreads;   // tokens per thread: 8 (x 8 columns)
  __shared__ float rowmax[128];
  __shared__ float colred[kWaves][128];
  __shared__ float rrow[128], rcol[128];
  __shared__ uint32_t stage[128 * 33];

  const int t = threadIdx.x;
  const int lane = t & 63, wave = t >> 6;
  const int tc = t & 15, tr = t >> 4;
  // tile order of tile_order (quant.hip), in 32 bits: runs of 2^bt_log2 token blocks of one column block
  const uint32_t run = blockIdx.x >> bt_log2, ncb = (uint32_t)a.C / 128u;
  const uint32_t run_row = run / ncb;
  const int64_t tb = ((int64_t)run_row << bt_log2) + (blockIdx.x & ((1u << bt_log2) - 1u));
  const int64_t gcol = run - run_row * ncb;
  const int64_t tok0 = tb * 128 + tr * kRows;
  const int col0 = (int)gcol * 128 + tc * 8;

  Raw8<BF16> raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) raw[i] = load8<BF16, true>(a.x, (tok0 + i) * a.ldx + col0, 8);
  float g[8], be[8];
  load_vec8(a.gamma, a.w_bf16, true, col0, 8, g);
  load_vec8(a.beta, a.w_bf16, true, col0, a.beta ? 8 : 0, be);

  float y[kRows][8];
  float cm[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    unpack8<BF16, true>(raw[i], 8, y[i]);
    if constexpr (LAYER) {
      const float mean = a.mean[tok0 + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] -= mean;
    }
    norm8(y[i], a.rstd[tok0 + i], g, be, y[i]);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) m = max3abs(m, y[i][j], y[i][j + 1]);
    m = row16_maxf(m);
    if (tc == 0) rowmax[tr * kRows + i] = m;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int i = 0; i < kRows; i += 2) cm[j] = max3abs(cm[j], y[i][j], y[i + 1][j]);
    // (magnitudes compare as their bits)
    uint32_t m = __float_as_uint(cm[j]);
    m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
    cm[j] = __uint_as_float(umax(m, (uint32_t)__shfl_xor((int)m, 32)));
  }
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) colred[wave][tc * 8 + j] = cm[j];
  }
  __syncthreads();
  if (t < 128) {
    float sc, r;
    tile_scale32(rowmax[t], sc, r);
    rrow[t] = r;
    a.s[gcol * a.T + tb * 128 + t] = sc;
  } else if (t < 256) {
    const int c = t - 128;
    uint32_t m = __float_as_uint(colred[0][c]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = umax(m, __float_as_uint(colred[w][c]));
    float sc, r;
    tile_scale32(__uint_as_float(m), sc, r);
    rcol[c] = r;
    a.sT[tb * a.C + gcol * 128 + c] = sc;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float r = rrow[tr * kRows + i];
    const u32x2 o = {codes4(y[i][0] * r, y[i][1] * r, y[i][2] * r, y[i][3] * r),
                     codes4(y[i][4] * r, y[i][5] * r, y[i][6] * r, y[i][7] * r)};
    __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(a.q + (tok0 + i) * a.ldq + col0));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r = rcol[tc * 8 + j];
#pragma unroll
    for (int h = 0; h < kRows / 4; ++h)
      stage[(tc * 8 + j) * 33 + kRows / 4 * tr + h] =
          codes4(y[4 * h][j] * r, y[4 * h + 1][j] * r, y[4 * h + 2][j] * r, y[4 * h + 3][j] * r);
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 1024 / kDualThreads; ++it) {
    const int cl = (t >> 3) + kDualThreads / 8 * it;
    const int part = t & 7;
    const uint32_t* sp = stage + cl * 33 + part * 4;
    const u32x4 o = {sp[0], sp[1], sp[2], sp[3]};
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(a.qT + (gcol * 128 + cl) * a.ldqT + tb * 128 + part * 16));
  }
}

// ---------------------------------------------------------------------------------------------------
// Backward.  Eight waves per workgroup, teams of LPR lanes with a row each; a lane's columns as in the
// forward kernel.  The weight's and bias's gradient of a thread's columns are summed in registers
// over the team's rows, then over the workgroup's teams through LDS, and written as the workgroup's
// partial sums; norm_bwd_reduce_kernel adds those in order.  After every 64 rows a thread adds its sums to a place of
// its own in LDS and starts anew: in one run of T / 256 rows the error would grow with T (1024 rows of equal terms
// 256 half steps of fp32 off).  Inputs of up to 64 rows per team, 16384 at 4097 columns and more, have a single run.
// Measured, 16384 x 2048 bf16: 35.3 us (5.7 TB/s) + 4.7 for the joining; with four chunks per lane 40.4.
// ---------------------------------------------------------------------------------------------------
constexpr int kBwdThreads = 512;
constexpr int kRun = 64;               // rows a thread adds in order, and sums of such runs
constexpr int kBwdWaves = kBwdThreads / 64;

template <bool BF16, bool VEC, int LPR, int ITER>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormBwdArgs a, int rows_per_team, bool direct) {
  constexpr int kTeams = kBwdThreads / LPR;
  constexpr int kWidth = 8 * LPR * ITER;
  __shared__ float red[2][2][kBwdWaves];
  __shared__ __attribute__((aligned(16))) float join[2][kTeams * kWidth];   // the weight's sums, the bias's
  const int team = threadIdx.x / LPR;
  const int tt = threadIdx.x % LPR;
  const int64_t stride = (int64_t)gridDim.x * kTeams;

  int col[ITER], nv[ITER];
  float g[ITER][8], dg[ITER][8], db[ITER][8];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    col[i] = 8 * (LPR * i + tt);
    nv[i] = a.C - col[i] < 0 ? 0 : (a.C - col[i] > 8 ? 8 : a.C - col[i]);
    load_vec8(a.gamma, a.w_bf16, aligned16(a.gamma), col[i], nv[i], g[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.f;
  }
  const float inv_c = 1.0f / (float)a.C;
  int64_t row = (int64_t)blockIdx.x * kTeams + team;
  Raw8<BF16> nx[ITER], ny[ITER];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t r) {
    const bool ok = r < a.T;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      nx[i] = load8<BF16, VEC>(a.x, r * a.ldx + col[i], ok ? nv[i] : 0);
      ny[i] = load8<BF16, VEC>(a.dy, r * a.lddy + col[i], ok ? nv[i] : 0);
    }
    nmean = ok && a.layer ? a.mean[r] : 0.f;
    nrstd = ok ? a.rstd[r] : 0.f;
  };
  // a thread's eight sums at its place in LDS, set or added to (no other thread touches it before the join)
  auto put = [&](int which, int i, const float (&v)[8], bool add) {
    f32x4* p = reinterpret_cast<f32x4*>(join[which] + team * kWidth + col[i]);
    const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    p[0] = add ? p[0] + lo : lo;
    p[1] = add ? p[1] + hi : hi;
  };
  // The widest class has no registers for a row ahead nor for a row's differences between their two uses: it keeps the row
  // as loaded and takes them again (2000 x 16384: bf16 65 us, fp32 110; 88 and 201 as the others do it, spilling).  Of its
  // instances the one of unaligned fp32 rows still spills, 136 bytes a lane.
  constexpr bool kAhead = ITER < 4;
  if (kAhead) fetch(row);
  for (int k = 0; k < rows_per_team; ++k, row += stride) {
    if (!kAhead) fetch(row);
    const bool ok = row < a.T;
    const float mean = nmean, rstd = nrstd;
    float xh[kAhead ? ITER : 1][8], d[kAhead ? ITER : 1][8];
    float s1 = 0.f, s2 = 0.f;
    auto take = [&](int i, float (&x)[8], float (&v)[8]) {
      unpack8<BF16, VEC>(nx[i], nv[i], x);
      unpack8<BF16, VEC>(ny[i], nv[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (x[j] - mean) * rstd;
    };
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float (&x)[8] = xh[kAhead ? i : 0], (&v)[8] = d[kAhead ? i : 0];
      take(i, x, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // a column that does not exist has dy = 0 and weight 0: it adds nothing to any sum
        dg[i][j] = __builtin_fmaf(v[j], x[j], dg[i][j]);
        db[i][j] += v[j];
        v[j] *= g[i][j];
        s1 += v[j];
        s2 = __builtin_fmaf(v[j], x[j], s2);
      }
    }
    if (kAhead && k + 1 < rows_per_team) fetch(row + stride);
    s1 = lanes_sum<LPR>(s1);
    s2 = lanes_sum<LPR>(s2);
    if constexpr (LPR > 64) {
      constexpr int kTeamWaves = LPR / 64;
      const int slot = k & 1;
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
    }
    s1 = a.layer ? s1 * inv_c : 0.f;
    s2 *= inv_c;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float o[8];
      float (&x)[8] = xh[kAhead ? i : 0], (&v)[8] = d[kAhead ? i : 0];
      if constexpr (!kAhead) {
        forget(nx[i]);
        forget(ny[i]);
        take(i, x, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g[i][j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (__builtin_fmaf(-x[j], s2, v[j]) - s1) * rstd;
      store8<BF16, VEC, false>(a.dx, row * a.lddx + col[i], ok ? nv[i] : 0, o);
    }
    if (k % kRun == kRun - 1 && k + 1 < rows_per_team) {   // a run is full, and another one follows
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        put(0, i, dg[i], k >= kRun);
        put(1, i, db[i], k >= kRun);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.f;
      }
    }
  }

  // the workgroup's sums: the weight's gradient, then the bias's
  float* out_g = direct ? a.dgamma : a.partial + (int64_t)blockIdx.x * 2 * a.C;
  float* out_b = direct ? a.dbeta : a.partial + ((int64_t)blockIdx.x * 2 + 1) * a.C;
  const bool add = direct && a.accumulate;
  const bool runs = rows_per_team > kRun;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? out_g : out_b;
    if (which == 1 && a.dbeta == nullptr) break;
    if constexpr (kTeams > 1) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) put(which, i, which == 0 ? dg[i] : db[i], runs);
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += kBwdThreads) {
        float s = join[which][c];
#pragma unroll
        for (int w = 1; w < kTeams; ++w) s += join[which][w * kWidth + c];
        out[c] = add ? out[c] + s : s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float s = which == 0 ? dg[i][j] : db[i][j];
          if (runs) s += join[which][col[i] + j];
          if (j < nv[i]) out[col[i] + j] = add ? out[col[i] + j] + s : s;
        }
    }
  }
}

// dgamma[c], dbeta[c] = sum over workgroups of their partials: 16 columns x 16 runs of workgroups per
// workgroup, the runs joined in order.  (More than 256 partials, of more than 10^6 rows, are added in 64 bits 16 at a time.)
__global__ __launch_bounds__(256) void norm_bwd_reduce_kernel(const float* __restrict__ partial, int blocks, int C,
                                                              float* dgamma, float* dbeta, int accumulate) {
  __shared__ float part[16][17];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cx;
  const int which = blockIdx.y;
  double sum = 0.0;
  if (c < C)
    for (int b0 = ry; b0 < blocks; b0 += 256) {
      float v[16], s = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = b0 + 16 * k < blocks ? partial[((int64_t)(b0 + 16 * k) * 2 + which) * C + c] : 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += v[k];
      sum += (double)s;
    }
  float s = (float)sum;
  part[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < C) {
#pragma unroll
    for (int r = 1; r < 16; ++r) s += part[r][cx];
    float* out = which == 0 ? dgamma : dbeta;
    out[c] = accumulate ? out[c] + s : s;
  }
}

__global__ __launch_bounds__(256) void norm_zero_kernel(float* dgamma, float* dbeta, int C) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  dgamma[c] = 0.f;
  if (dbeta) dbeta[c] = 0.f;
}

template <bool BF16, bool VEC, int WHAT>
hipError_t launch_fwd(NormArgs a, hipStream_t st) {
  // The layout over threads goes by C alone, so every form sums a row in the same order.
  auto go = [&](auto kernel, int lpr) {
    const int threads = lpr > 256 ? lpr : 256, teams = threads / lpr;
    // rows per team: 4 for long inputs, so that the next row's loads hide behind this one and a workgroup's rows are runs of
    // the row-wise arrays; one row where the input would not give the card 2048 waves otherwise.  (8 rows leave
    // too few workgroups to share evenly: 16384 x 1024 bf16 15.3 us, 12.2 with 4; 3000 x 3000 10.2 and 9.2; 16384 x 2048
    // 23.5 and 23.2.  2 rows: 36.0 us at 16384 x 2047, 32.4 with 4.)
    int64_t r = std::max<int64_t>(1, std::min<int64_t>(4, a.T / (131072 / lpr)));
    // (a launch counts its threads in 32 bits: past 2^30 of the shortest rows a team takes more)
    const int64_t most = 0xFFFFFFFFll / threads * teams;
    r = std::max(r, (a.T + most - 1) / most);
    if (r > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    a.rows_per_team = (int)r;
    const int64_t blocks = (a.T + teams * r - 1) / (teams * r);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
    return hipGetLastError();
  };
  if (a.C <= 128) return go(norm_kernel<BF16, VEC, 16, 1, WHAT>, 16);
  if (a.C <= 256) return go(norm_kernel<BF16, VEC, 32, 1, WHAT>, 32);
  if (a.C <= 512) return go(norm_kernel<BF16, VEC, 64, 1, WHAT>, 64);
  if (a.C <= 1024) return go(norm_kernel<BF16, VEC, 64, 2, WHAT>, 64);
  if (a.C <= 2048) return go(norm_kernel<BF16, VEC, 128, 2, WHAT>, 128);
  if (a.C <= 4096) return go(norm_kernel<BF16, VEC, 256, 2, WHAT>, 256);
  if (a.C <= 8192) return go(norm_kernel<BF16, VEC, 512, 2, WHAT>, 512);
  return go(norm_kernel<BF16, VEC, 512, 4, WHAT>, 512);
}

// lanes per row of the backward kernel; it takes kBwdThreads / this rows per workgroup and step
int bwd_lpr(int64_t C) {
  return C <= 128 ? 16 : C <= 256 ? 32 : C <= 1024 ? 64 : C <= 2048 ? 128 : C <= 4096 ? 256 : 512;
}

template <bool BF16, bool VEC>
hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t st) {
  const int blocks = norm_bwd_blocks(a.T, a.C);
  const int teams = kBwdThreads / bwd_lpr(a.C);
  const int rows = (int)((a.T + (int64_t)blocks * teams - 1) / ((int64_t)blocks * teams));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBwdThreads), 0, st, a, rows, blocks == 1);
    return hipGetLastError();
  };
  hipError_t e;
  if (a.C <= 128) e = go(norm_bwd_kernel<BF16, VEC, 16, 1>);
  else if (a.C <= 256) e = go(norm_bwd_kernel<BF16, VEC, 32, 1>);
  else if (a.C <= 512) e = go(norm_bwd_kernel<BF16, VEC, 64, 1>);
  else if (a.C <= 1024) e = go(norm_bwd_kernel<BF16, VEC, 64, 2>);
  else if (a.C <= 2048) e = go(norm_bwd_kernel<BF16, VEC, 128, 2>);
  else if (a.C <= 4096) e = go(norm_bwd_kernel<BF16, VEC, 256, 2>);
  else if (a.C <= 8192) e = go(norm_bwd_kernel<BF16, VEC, 512, 2>);
  else e = go(norm_bwd_kernel<BF16, VEC, 512, 4>);
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(norm_bwd_reduce_kernel, dim3((unsigned)((a.C + 15) / 16), a.dbeta ? 2 : 1), dim3(256), 0, st,
                     a.partial, blocks, a.C, a.dgamma, a.dbeta, a.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(NormArgs a, hipStream_t st) {
  const int64_t es = a.x_bf16 ? 2 : 4;
  const bool vec = a.C % 8 == 0 && vec_row(a.x, a.ldx, es) && vec_row(a.y, a.ldy, es);
  if (a.x_bf16) return vec ? launch_fwd<true, true, 0>(a, st) : launch_fwd<true, false, 0>(a, st);
  return vec ? launch_fwd<false, true, 0>(a, st) : launch_fwd<false, false, 0>(a, st);
}

hipError_t launch_norm_quant(NormArgs a, hipStream_t st) {
  return a.x_bf16 ? launch_fwd<true, true, 1>(a, st) : launch_fwd<false, true, 1>(a, st);
}

hipError_t launch_norm_quant_dual(NormArgs a, hipStream_t st) {
  const hipError_t e = a.x_bf16 ? launch_fwd<true, true, 2>(a, st) : launch_fwd<false, true, 2>(a, st);
  return e != hipSuccess ? e : launch_norm_tiles(a, st);
}

hipError_t launch_norm_tiles(NormArgs a, hipStream_t st) {
  const int64_t nb = a.T / 128;
  int bt = 5;   // up to 32 token blocks per run of workgroups: transposed rows are written in 4 KB runs
  while (nb & ((int64_t(1) << bt) - 1)) --bt;
  const dim3 grid((unsigned)(nb * (a.C / 128)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kDualThreads), 0, st, a, bt);
    return hipGetLastError();
  };
  if (a.x_bf16) return a.layer ? go(norm_dual_kernel<true, true>) : go(norm_dual_kernel<true, false>);
  return a.layer ? go(norm_dual_kernel<false, true>) : go(norm_dual_kernel<false, false>);
}

// One workgroup per CU, but no more than there are rows for its teams, and beyond 64 no more than one for 8 rows:
// every workgroup writes and the second launch reads 8 bytes per column, which at 8 rows (6 bytes per element and
// row in bf16) is a third of the pass.  A single one, without a second launch, up to two rows per team.  Measured, us:
// 64 x 2048 7.1 (7.9 with two rows per team at least); 1027 x 4096 14.6 with 128 workgroups, 18.0 with 256; 16 x 1000
// 5.1 alone, 6.7 in two.
// Beyond 64 runs of 64 rows for each of 256 workgroups there are more, whole rounds of 256, up to the 2^32 threads of a
// launch.
int norm_bwd_blocks(int64_t T, int64_t C) {
  if (T <= 0 || C <= 0) return 0;
  const int64_t teams = kBwdThreads / bwd_lpr(C);
  if (T <= 2 * teams) return 1;
  const int64_t round = (int64_t)kRun * kRun * 256 * teams;
  if (T > round) return (int)(256 * std::min<int64_t>((T + round - 1) / round, (int64_t(1) << 32) / (256 * kBwdThreads) - 1));
  return (int)std::min<int64_t>(std::min<int64_t>(256, (T + teams - 1) / teams), std::max<int64_t>(64, (T + 7) / 8));
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
  if (a.T == 0 || a.C == 0) {
    if (a.accumulate || a.C == 0) return hipSuccess;
    hipLaunchKernelGGL(norm_zero_kernel, dim3((unsigned)((a.C + 255) / 256)), dim3(256), 0, st, a.dgamma, a.dbeta, a.C);
    return hipGetLastError();
  }
  const int64_t es = a.x_bf16 ? 2 : 4;
  const bool vec = a.C % 8 == 0 && vec_row(a.x, a.ldx, es) && vec_row(a.dy, a.lddy, es) && vec_row(a.dx, a.lddx, es);
  if (a.x_bf16) return vec ? launch_bwd<true, true>(a, st) : launch_bwd<true, false>(a, st);
  return vec ? launch_bwd<false, true>(a, st) : launch_bwd<false, false>(a, st);
}

}  // namespace puro
