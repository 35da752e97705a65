// gfx950 blockwise-scaled FP8 product for any number of rows: single tokens, decode batches, ragged
// prompts.
//
//   C[m,n] = sum_kb sA(kb,m) sB(n/128,kb) P_kb[m,n],   P_kb[m,n] = sum_{k in slice kb} dec(A[m,k]) dec(B[n,k])
//
// With few rows the product is bound by reading the weight codes once (N K bytes).  A workgroup owns
// 16 NT output columns for 16 MT rows and splits the contraction over its waves: wave w takes the
// 128-deep slices w, w + waves, ..., so one workgroup has as many whole weight lines in flight as it
// has waves, and a narrow output still keeps the card busy.  The waves' fp32 sums are joined through
// LDS in a fixed order.
//
// A slice of a 16-row fragment is two 16-byte loads per lane, straight to registers (lane l: row
// l % 16, bytes 16 (l / 16) .. +15 and 64 + 16 (l / 16) .. +15: each load instruction reads 16
// contiguous 64-byte pieces).  E4M3 codes are converted exactly to bf16 and multiplied by
// v_mfma_f32_16x16x32_bf16; both operands use the same order of the contraction, so the order itself
// does not matter.  The bf16 matrix instruction keeps a full fp32 sum; the FP8 one's sum of 128
// products is about 1.4e-5 off (relative, measured), which an fp32 output would show.
// The weight is the first operand: a lane then holds four consecutive columns of one output row, and
// its row scale is one value.
#include "codec.hpp"
#include "gemm_args.hpp"
#include "ops_internal.hpp"

namespace puro {

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;

struct RowsArgs {
  int M, N, K;
  const uint8_t* A;
  int64_t lda;
  const float* sA;
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
__device__ __forceinline__ Frag load_frag(const uint8_t* p) {
  return Frag{*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + 64)};
}

template <int MT, int NT, bool OUT_BF16>
__global__ __launch_bounds__(64 * kWaves) void gemm_rows_kernel(RowsArgs p) {
  __shared__ f32x4_t join[kWaves][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT;
  const int m0 = blockIdx.y * 16 * MT;
  const int nk = p.K >> 7;

  const uint8_t* bp[NT];
  const uint8_t* ap[MT];
  int mrow[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) bp[j] = p.B + (int64_t)(n0 + 16 * j + l16) * p.ldb + 16 * g;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + l16;
    mrow[i] = m < p.M ? m : p.M - 1;       // rows past M repeat the last one and are not written
    ap[i] = p.A + (int64_t)mrow[i] * p.lda + 16 * g;
  }
  const float* sb = p.sB + (int64_t)(n0 >> 7) * nk;

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll 2
  for (int kb = wave; kb < nk; kb += kWaves) {
    Frag bf[NT], af[MT];
    float s[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) bf[j] = load_frag(bp[j] + (int64_t)kb * 128);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      af[i] = load_frag(ap[i] + (int64_t)kb * 128);
      s[i] = p.sA[(int64_t)kb * p.M + mrow[i]] * sb[kb];
    }
    bf16x8_t bd[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bd[j][2 * h] = decode8(bf[j].w[h].x, bf[j].w[h].y);
        bd[j][2 * h + 1] = decode8(bf[j].w[h].z, bf[j].w[h].w);
      }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      bf16x8_t ad[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ad[2 * h] = decode8(af[i].w[h].x, af[i].w[h].y);
        ad[2 * h + 1] = decode8(af[i].w[h].z, af[i].w[h].w);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bd[j][h], ad[h], d, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s[i], acc[i][j][r]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) join[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < MT * NT * 64; t += 64 * kWaves) {
    const int tile = t >> 6, l = t & 63;
    f32x4_t v = join[0][tile][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += join[w][tile][l];
    const int m = m0 + 16 * (tile / NT) + (l & 15);
    const int n = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    if (m >= p.M) continue;
    if constexpr (OUT_BF16) {
      const u32x2 o = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.C) + (int64_t)m * p.ldc + n) = o;
    } else {
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.C) + (int64_t)m * p.ldc + n) = v;
    }
  }
}

template <int MT, int NT>
hipError_t go(const RowsArgs& a, bool out_bf16, hipStream_t st) {
  const dim3 grid((unsigned)(a.N / (16 * NT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  if (grid.y > 65535u) return hipErrorInvalidConfiguration;
  if (out_bf16)
    hipLaunchKernelGGL((gemm_rows_kernel<MT, NT, true>), grid, dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((gemm_rows_kernel<MT, NT, false>), grid, dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t gemm_rows_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_rows(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                            const uint8_t* B, int64_t ldb, const float* sB, void* C, int64_t ldc, bool out_bf16,
                            void*, hipStream_t st) {
  const RowsArgs a = {(int)M, (int)N, (int)K, A, lda, sA, B, ldb, sB, C, ldc};
  if (M <= 16) return go<1, 1>(a, out_bf16, st);
  if (M <= 32) return go<2, 1>(a, out_bf16, st);
  return go<4, 2>(a, out_bf16, st);
}

}  // namespace puro
