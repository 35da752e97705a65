// gfx950 blockwise-scaled FP8 product for any number of rows: single tokens, decode batches, ragged
// prompts.
//
//   C[m,n] = sum_kb sA(kb,m) sB(n/128,kb) P_kb[m,n],   P_kb[m,n] = sum_{k in slice kb} dec(A[m,k]) dec(B[n,k])
//
// With few rows the product is bound by reading the weight codes once (N K bytes), and a CU takes at most about
// 25 bytes per ns of them from HBM (measured: 256 CUs stream 6.4 TB/s), so every CU has to have its share.  A workgroup owns
// NT strips of 16 columns for 16 MT rows, with NT chosen so that about one workgroup per CU is left (launch_gemm_rows),
// and splits the contraction over its waves, a run of 128-deep slices each: it has as many weight lines in flight as
// it has waves, without a second launch to join the parts.  The waves' fp32 sums are joined through LDS in order.
//
// A slice of a 16-row fragment is two 16-byte loads per lane, eight lanes to a row's 128-byte line, and is
// turned into the matrix instruction's order (lane l: row l % 16, 16-byte chunks l / 16 and l / 16 + 4) through
// the wave's own piece of LDS.  Loading that order directly costs 77 cycles per load instruction (each lane a request of its
// own) against 16; 64 rows x 6144 deep x 2048 columns took 17.4 us so and take 12.2.  Chunk c of row r is kept
// at c ^ (r / 2 % 8), which spreads a read's 16 rows over all banks.  Both operands use the same order of
// the contraction, so the order itself does not matter.
//
// The codes are converted, exactly, to bf16, whose matrix instruction keeps a full fp32 sum (1e-7 off, relative); the
// FP8 one's sum of 128 products is about 1.4e-5 off, which an fp32 output shows and a sum that cancels shows in
// bf16 too.  The conversion costs 4 to 9% up to 64 rows and 10 to 30% at 200, where matrix work shows.
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

// Keeps the compiler from moving one lane's LDS reads over another's writes; the hardware does a wave's in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT;
  const int m0 = blockIdx.y * 16 * MT;
  const int nk = p.K >> 7;
  uint8_t* stage = smem + wave * kStage;

  // loads: lane l takes 16 bytes of row l / 8 (and l / 8 + 8)
  const int lr = lane >> 3, lc = lane & 7;
  const uint8_t* bp[NT];
  const float* sb[NT];
  const uint8_t* ap[MT][2];
  int mrow[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = n0 + 16 * j < p.N ? n0 + 16 * j : p.N - 16;   // strips past N repeat the last one, likewise
    bp[j] = p.B + (int64_t)(n + lr) * p.ldb + 16 * lc;
    sb[j] = p.sB + (int64_t)(n >> 7) * nk;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + l16;
    mrow[i] = m < p.M ? m : p.M - 1;       // rows past M repeat the last one and are not written
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int mm = m0 + 16 * i + 8 * h + lr;
      ap[i][h] = p.A + (int64_t)(mm < p.M ? mm : p.M - 1) * p.lda + 16 * lc;
    }
  }
  uint8_t* wr0 = stage + lr * 128 + ((lc ^ ((lr >> 1) & 7)) * 16);
  uint8_t* wr1 = stage + (lr + 8) * 128 + ((lc ^ (((lr + 8) >> 1) & 7)) * 16);
  const uint8_t* rd0 = stage + l16 * 128 + ((g ^ ((l16 >> 1) & 7)) * 16);
  const uint8_t* rd1 = stage + l16 * 128 + (((g + 4) ^ ((l16 >> 1) & 7)) * 16);

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int per = (nk + WK - 1) / WK, kbeg = wave * per, kend = kbeg + per < nk ? kbeg + per : nk;
  // Up to 32 rows and 3 strips the next slice is loaded as soon as this one is in LDS (1 x 6144 deep x 2048: 6.2 us, 7.4
  // without).  Larger tiles lack the registers: 64 x 2048 deep x 4096 takes 9.8 us so and 5.7 as it is, one row with 4 strips
  // (151936 columns) 69.7 and 59.1.
  constexpr bool kAhead = MT <= 2 && NT <= 3;
  u32x4 bl[NT][2], al[MT][2];
  float sa[MT];
  auto fetch = [&](int kb) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      bl[j][0] = *reinterpret_cast<const u32x4*>(bp[j] + (int64_t)kb * 128);
      bl[j][1] = *reinterpret_cast<const u32x4*>(bp[j] + 8 * p.ldb + (int64_t)kb * 128);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) al[i][h] = *reinterpret_cast<const u32x4*>(ap[i][h] + (int64_t)kb * 128);
      sa[i] = p.sA[(int64_t)kb * p.lds + mrow[i]];
    }
  };
  if (kAhead && kbeg < kend) fetch(kbeg);
  for (int kb = kbeg; kb < kend; ++kb) {
    if (!kAhead) fetch(kb);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<u32x4*>(wr0 + j * 2048) = bl[j][0];
      *reinterpret_cast<u32x4*>(wr1 + j * 2048) = bl[j][1];
    }
    float sc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      *reinterpret_cast<u32x4*>(wr0 + (NT + i) * 2048) = al[i][0];
      *reinterpret_cast<u32x4*>(wr1 + (NT + i) * 2048) = al[i][1];
      sc[i] = sa[i];
    }
    if (kAhead && kb + 1 < kend) fetch(kb + 1);
    wave_order();   // the LDS piece is the wave's own: its instructions reach it in order
    auto fragment = [&](int f) {
      return Operand(Frag{*reinterpret_cast<const u32x4*>(rd0 + f * 2048), *reinterpret_cast<const u32x4*>(rd1 + f * 2048)});
    };
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
    wave_order();
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

// Strips per workgroup: the fewest that leave at most one workgroup per CU (256).  Fewer would give some CUs two and others one
// (N = 12288, M <= 16: 7.0 us with 3 strips, 8.6 with 1), more would leave CUs idle (N = 4096: 4.1 us with 1,
// 4.5 with 2).  A lone strip gets 16 waves (K = 6144: 6.5 us, 7.2 with 8).
template <int MT>
hipError_t by_strips(const RowsArgs& a, bool out_bf16, hipStream_t st) {
  const int64_t strips = a.N / 16, row_blocks = (a.M + 16 * MT - 1) / (16 * MT);
  auto fits = [&](int64_t nt) { return (strips + nt - 1) / nt * row_blocks <= 256; };
  if (fits(1)) return go<MT, 1, 16>(a, out_bf16, st);
  if (fits(2)) return go<MT, 2, 8>(a, out_bf16, st);
  if (fits(3)) return go<MT, 3, 8>(a, out_bf16, st);
  return go<MT, 4, 8>(a, out_bf16, st);
}

// Leading rows (a multiple of 128) that go through the 256 x 256 tiles of the blockwise GEMM: all there are, where their
// product is long enough to fill it.  Both sides, us: 512 x 12288 x 2048 51 here, 26 there; 1024 x 4096 x 2048 32 and
// 27; 256 x 12288 x 2048 28 and 27; 512 x 2048 x 6144 22 and 30; 2048 x 1024 x 1024 12 and 15.
int64_t leading_rows(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = M - M % 128;
  return (double)rows * (double)N * (double)K >= (double)(int64_t(1) << 33) ? rows : 0;
}

}  // namespace

size_t gemm_rows_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = leading_rows(M, N, K);
  return rows ? gemm_workspace_bytes(0, rows, N, K) : 0;
}

hipError_t launch_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                            const uint8_t* B, int64_t ldb, const float* sB, void* C, int64_t ldc, bool out_bf16,
                            void* workspace, size_t workspace_bytes, hipStream_t st) {
  const int64_t lead = out_bf16 ? leading_rows(M, N, K) : 0;
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
    hipError_t e;
    if (rows <= 16) e = by_strips<1>(a, out_bf16, st);
    else if (rows <= 32) e = by_strips<2>(a, out_bf16, st);
    else if (rows <= 48) e = by_strips<3>(a, out_bf16, st);   // (37 x 4096 x 2048: 4.9 us, 5.4 as 64 rows)
    else e = by_strips<4>(a, out_bf16, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace puro
