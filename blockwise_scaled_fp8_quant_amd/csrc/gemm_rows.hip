// gfx950 blockwise-scaled FP8 product for any number of rows: single tokens, decode batches, ragged
// prompts.
//
//   C[m,n] = sum_kb sA(kb,m) sB(n/128,kb) P_kb[m,n],   P_kb[m,n] = sum_{k in slice kb} dec(A[m,k]) dec(B[n,k])
//
// With few rows the product is bound by reading the weight codes once (N K bytes), and a CU takes at most about
// 25 bytes per ns of them from HBM (measured: 256 CUs stream 6.4 TB/s), so every CU has to have its share.  A workgroup owns
// NT strips of 16 columns for 16 MT rows, chosen by what a CU then loads (by_tile), and splits the contraction over its
// waves, a run of 128-deep slices each: it has as many weight lines in flight as it has waves, without a second launch
// to join the parts.  The waves' fp32 sums are joined through LDS in order.
//
// A slice of a 16-row fragment is two 16-byte loads per lane, eight lanes to a row's 128-byte line, that go straight into
// the wave's own piece of LDS, and is read from there in the matrix instruction's order (lane l: row l % 16, 16-byte
// chunks l / 16 and l / 16 + 4).  Loading that order directly costs 77 cycles per load instruction (each lane a request of
// its own) against 16.  Chunk c of row r is kept in slot c ^ (r / 2 % 8), which spreads a read's 16 rows over all
// banks; a load fills the slots in order, so the lanes take their row's chunks in that order.  Both operands use the same
// order of the contraction, so the order itself does not matter.
// The next slice is on its way as soon as this one has left LDS for registers.  Loads through registers left none
// for a slice ahead beyond 32 rows and 3 strips (200 x 6144 deep x 2048, same tile: 14.3 us so, 12.9 as it is).
//
// The codes are converted, exactly, to bf16, whose matrix instruction keeps a full fp32 sum (1e-7 off, relative); the
// FP8 one's sum of 128 products is 1.4e-5 off (normal data; 5e-5 for codes of every magnitude, a single sum up to 1.6e-4
// of its magnitudes), which an fp32 output shows and a sum that cancels shows in bf16 too.  The leading rows of a long
// bf16 product, which the FP8 ones take (leading_rows), are as far off as the blockwise GEMM's, and up to three times as
// fast.  The conversion costs 2 to 9% up to 64 rows and 6 to 11% at 200, where matrix work shows.  (The FP8 one's
// 16 x 16 x 32 form is 9e-5 off.)
// The weight is the first operand: a lane then holds four consecutive columns of one output row, and
// its row scale is one value.
#include <algorithm>

#include "codec.hpp"
#include "gemm_args.hpp"
#include "internal.hpp"
#include "ops_internal.hpp"

namespace puro {

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct RowsArgs {
  int M, N, K;
  const uint8_t* A;
  int64_t lda;
  const float* sA;
  int64_t lds;       // elements between consecutive slices of sA
  const uint8_t* B;
  int64_t ldb;
  const float* sB;
  void* C;
  int64_t ldc;
};

// Eight E4M3 codes (two dwords) -> bf16, exact.
__device__ __forceinline__ bf16x8_t decode8(uint32_t lo, uint32_t hi) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

struct Frag {
  u32x4 w[2];
};

// A fragment as the matrix instruction takes it, in four parts of the slice.
struct Operand {
  bf16x8_t v[4];
  __device__ __forceinline__ explicit Operand(const Frag& f)
      : v{decode8(f.w[0].x, f.w[0].y), decode8(f.w[0].z, f.w[0].w), decode8(f.w[1].x, f.w[1].y), decode8(f.w[1].z, f.w[1].w)} {}
};

// MT x NT tiles of 16 x 16, the contraction over WK waves.
template <int MT, int NT, int WK, bool OUT_BF16>
__global__ __launch_bounds__(64 * WK) void gemm_rows_kernel(RowsArgs p) {
  constexpr int kTiles = MT * NT;
  constexpr int kStage = (MT + NT) * 2048;
  constexpr int kJoin = WK * kTiles * 64 * 16, kStages = WK * kStage;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kJoin > kStages ? kJoin : kStages];
  f32x4_t (*join)[kTiles][64] = reinterpret_cast<f32x4_t (*)[kTiles][64]>(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT;
  const int m0 = blockIdx.y * 16 * MT;
  const int nk = p.K >> 7;
  uint8_t* stage = smem + wave * kStage;

  // loads: lane l fills slot l % 8 of row l / 8 (and of row l / 8 + 8)
  const int lr = lane >> 3, lc = lane & 7;
  const int c0 = 16 * (lc ^ (lr >> 1)), c1 = c0 ^ 64;
  const uint8_t* bp[NT][2];
  const float* sb[NT];
  const uint8_t* ap[MT][2];
  int mrow[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = n0 + 16 * j < p.N ? n0 + 16 * j : p.N - 16;   // strips past N repeat the last one, likewise
    bp[j][0] = p.B + (int64_t)(n + lr) * p.ldb + c0;
    bp[j][1] = p.B + (int64_t)(n + lr + 8) * p.ldb + c1;
    sb[j] = p.sB + (int64_t)(n >> 7) * nk;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + l16;
    mrow[i] = m < p.M ? m : p.M - 1;       // rows past M repeat the last one and are not written
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int mm = m0 + 16 * i + 8 * h + lr;
      ap[i][h] = p.A + (int64_t)(mm < p.M ? mm : p.M - 1) * p.lda + (h ? c1 : c0);
    }
  }
  const uint8_t* rd0 = stage + l16 * 128 + ((g ^ ((l16 >> 1) & 7)) * 16);
  const uint8_t* rd1 = stage + l16 * 128 + (((g + 4) ^ ((l16 >> 1) & 7)) * 16);

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int per = (nk + WK - 1) / WK, kbeg = wave * per, kend = kbeg + per < nk ? kbeg + per : nk;
  float sa[MT];
  auto fetch = [&](int kb) {
#pragma unroll
    for (int f = 0; f < NT + MT; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* src = (f < NT ? bp[f < NT ? f : 0][h] : ap[f < NT ? 0 : f - NT][h]) + (int64_t)kb * 128;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                         (__attribute__((address_space(3))) void*)(stage + f * 2048 + h * 1024), 16, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = p.sA[(int64_t)kb * p.lds + mrow[i]];
  };
  if (kbeg < kend) fetch(kbeg);
  for (int kb = kbeg; kb < kend; ++kb) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the slice is in LDS
    __builtin_amdgcn_sched_barrier(0);
    Frag raw[NT + MT];
    float sc[MT];
#pragma unroll
    for (int f = 0; f < NT + MT; ++f) {
      raw[f].w[0] = *reinterpret_cast<const u32x4*>(rd0 + f * 2048);
      raw[f].w[1] = *reinterpret_cast<const u32x4*>(rd1 + f * 2048);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sc[i] = sa[i];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // and read: the next one may overwrite it
    __builtin_amdgcn_sched_barrier(0);
    if (kb + 1 < kend) fetch(kb + 1);
    auto fragment = [&](int f) { return Operand(raw[f]); };
    bf16x8_t bv[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const Operand b = fragment(j);
#pragma unroll
      for (int h = 0; h < 4; ++h) bv[j][h] = b.v[h];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const Operand a = fragment(NT + i);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j][h], a.v[h], v, 0, 0, 0);
        const float s = sc[i] * sb[j][kb];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(v[r], s, acc[i][j][r]);
      }
    }
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) join[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < kTiles * 64; t += 64 * WK) {
    const int tile = t >> 6, l = t & 63;
    f32x4_t v = join[0][tile][l];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += join[w][tile][l];
    const int m = m0 + 16 * (tile / NT) + (l & 15);
    const int n = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    if (m >= p.M || n >= p.N) continue;
    if constexpr (OUT_BF16) {
      const u32x2 o = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.C) + (int64_t)m * p.ldc + n) = o;
    } else {
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.C) + (int64_t)m * p.ldc + n) = v;
    }
  }
}

template <int MT, int NT, int WK>
hipError_t go(const RowsArgs& a, bool out_bf16, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 16 * NT - 1) / (16 * NT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  if (out_bf16)
    hipLaunchKernelGGL((gemm_rows_kernel<MT, NT, WK, true>), grid, dim3(64 * WK), 0, st, a);
  else
    hipLaunchKernelGGL((gemm_rows_kernel<MT, NT, WK, false>), grid, dim3(64 * WK), 0, st, a);
  return hipGetLastError();
}

// Waves of a workgroup, all on the same tile.  A lone strip has 16 where each gets more than one slice (1 x 6144 deep x
// 2048: 6.4 us, 7.0 with 8; 1 x 2048 deep x 4096: 4.05 us with 16, 3.86 with 8).  Where the card is filled more than
// once and a CU's LDS holds one workgroup of 8, two of 4 work while the other starts or ends (256 x 2048 deep x
// 12288: 24.0 us, 27.3 with 8); a single round has 8 (200 x 6144 deep x 2048: 13.7 us, 18.1 with 4).
template <int MT, int NT>
hipError_t by_waves(const RowsArgs& a, bool out_bf16, hipStream_t st, int64_t workgroups) {
  if constexpr (NT == 1) {
    if (a.K > 16 * 128) return go<MT, NT, 16>(a, out_bf16, st);
  }
  if constexpr (NT > 2 && MT + NT > 5) {
    if (workgroups > 256) return go<MT, NT, 4>(a, out_bf16, st);
  }
  return go<MT, NT, 8>(a, out_bf16, st);
}

// The tile: the one with which a CU loads least, rounds of 256 workgroups times MT + NT fragments a slice; among equals the
// one with most workgroups, then fewest rows.  (64 x 6144 deep x 2048: 8.4 us as 16 x 32 tiles, 12.4 as 64 x 16, which
// leave half the CUs idle; 64 x 2048 deep x 4096: 4.9 as 32 x 32, 6.3 as 64 x 16; 37 x 2048 deep x 12288: 9.2 as
// 48 x 48, which makes 256 workgroups.)
template <int MT>
hipError_t by_strips(const RowsArgs& a, bool out_bf16, hipStream_t st, int nt, int64_t workgroups) {
  if constexpr (MT < 4) {   // (4 x 1 never is that: 2 x 2 covers as much)
    if (nt == 1) return by_waves<MT, 1>(a, out_bf16, st, workgroups);
  }
  if (nt == 2) return by_waves<MT, 2>(a, out_bf16, st, workgroups);
  if (nt == 3) return by_waves<MT, 3>(a, out_bf16, st, workgroups);
  return by_waves<MT, 4>(a, out_bf16, st, workgroups);
}

hipError_t by_tile(const RowsArgs& a, bool out_bf16, hipStream_t st) {
  const uint32_t M = (uint32_t)a.M, strips = (uint32_t)a.N / 16;
  const int64_t row_blocks[4] = {(M + 15) / 16, (M + 31) / 32, (M + 47) / 48, (M + 63) / 64};
  const int64_t col_blocks[4] = {strips, (strips + 1) / 2, (strips + 2) / 3, (strips + 3) / 4};
  int mt = 4, nt = 4;
  int64_t best = INT64_MAX, workgroups = 0;
  for (int m = 1; m <= 4; ++m) {
    if (row_blocks[m - 1] > 65535) continue;   // the launch's second dimension
    for (int n = m < 4 ? 1 : 2; n <= 4; ++n) {
      const int64_t w = row_blocks[m - 1] * col_blocks[n - 1], cost = (w + 255) / 256 * (m + n);
      if (cost < best || (cost == best && w > workgroups)) {
        best = cost;
        workgroups = w;
        mt = m;
        nt = n;
      }
    }
  }
  if (mt == 1) return by_strips<1>(a, out_bf16, st, nt, workgroups);
  if (mt == 2) return by_strips<2>(a, out_bf16, st, nt, workgroups);
  if (mt == 3) return by_strips<3>(a, out_bf16, st, nt, workgroups);
  return by_strips<4>(a, out_bf16, st, nt, workgroups);
}

// Leading rows (a multiple of 128) that go through the 256 x 256 tiles of the blockwise GEMM: all there are, where their
// product is long enough to fill it.  The rows left over then read the weight once more, and 128 leading rows fill half a
// row of tiles, so those need twice the product.  Both sides, us (all rows here; leading rows there and the rest here):
//   256 rows and more: 512 x 12288 x 2048 42.2, 25.8; 500 41.4, 41.5; 1024 x 4096 x 2048 27.8, 27.4; 1025 31.0, 31.0;
//   300 x 32768 x 2048 73, 45; 257 x 8192 x 8192 60.8, 55.6; below 2^33: 256 x 12288 x 2048 22.5, 25.2; 257 28.0, 30.9;
//   640 x 2048 x 6144 27, 29; 2048 x 1024 x 1024 10, 15
//   128 to 255 rows: 128 x 151936 x 2048 172, 95; 200 310, 216; 255 318, 240; below 2^34: 130 x 8192 x 8192 37.8, 44.1; 255
//   48.7, 57.6; 130 x 32768 x 2048 43.3, 45.6; 128 x 12288 x 6144 36.6, 36.0; 255 60.5, 64.1
int64_t leading_rows(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = M - M % 128;
  return (double)rows * (double)N * (double)K >= (double)(int64_t(1) << (rows < 256 ? 34 : 33)) ? rows : 0;
}

// Whether the blockwise GEMM can read the row scales where they are.  Its four-wave kernel takes them a value at a time; where
// its 32-bit offsets do not reach, the eight-wave one copies four at once and needs every slice on 16 bytes, which an M
// that is no multiple of 4, or an sA on 4 bytes, does not give.  (Those calls run here: 2 GiB of weight rows and more.)
bool scales_reachable(int64_t M, int64_t K, int64_t lda, const float* sA, int64_t ldb) {
  if (M % 4 == 0 && (reinterpret_cast<uintptr_t>(sA) & 15u) == 0) return true;
  GemmArgs a = {};
  a.K = (int)K;
  a.lda = lda;
  a.ldb = ldb;
  a.ldsa = M;
  return kUseW4 && w4_supported(a);
}

}  // namespace

size_t gemm_rows_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = leading_rows(M, N, K);
  return rows ? gemm_workspace_bytes(0, rows, N, K) : 0;
}

hipError_t launch_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                            const uint8_t* B, int64_t ldb, const float* sB, void* C, int64_t ldc, bool out_bf16,
                            void* workspace, size_t workspace_bytes, hipStream_t st) {
  int64_t lead = out_bf16 ? leading_rows(M, N, K) : 0;
  if (lead && !scales_reachable(M, K, lda, sA, ldb)) lead = 0;
  if (lead) {
    const hipError_t e = launch_gemm(0, lead, N, K, A, lda, sA, B, ldb, sB, C, ldc, true, false, nullptr, 0, nullptr,
                                     workspace, workspace_bytes, st, M);
    if (e != hipSuccess || lead == M) return e;
  }
  constexpr int64_t kMost = 65535 * 64;   // rows that a launch's second dimension holds (fp32 outputs may have more)
  for (int64_t m = lead; m < M; m += kMost) {
    const int64_t rows = std::min(M - m, kMost);
    const RowsArgs a = {(int)rows, (int)N, (int)K, A + m * lda, lda, sA + m, M, B, ldb, sB,
                        static_cast<uint8_t*>(C) + m * ldc * (out_bf16 ? 2 : 4), ldc};
    const hipError_t e = by_tile(a, out_bf16, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace puro
