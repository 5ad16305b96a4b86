// mxfp4_gemm.hip -- products with an MXFP4 (E2M1, one E8M0 scale per 32 of K)
// right operand on CDNA4 matrix cores (gfx950):
//
//   C[m][n] = sum over 32-wide K blocks j of
//             2^(sa[m][j] - 127) * 2^(sb[n][j] - 127) * sum_{k in j} A[m][k] * B[n][k]
//
// A in E2M1, E4M3 or E5M2, fp32 accumulation, fp32 or bf16 out.  The scaled
// matrix instructions take the element formats and the blocks' scales as they
// are, so nothing is decoded.
#include "mx_common.hpp"
#include "mx_launch.hpp"

namespace mxfp8 {

namespace mxfp4_detail {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Element format as the matrix instructions number them.
template <int FMT> constexpr int kMfmaFmt = FMT == kE2M1 ? 4 : FMT;

__device__ __forceinline__ void mfma_retire_pad() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

__device__ __forceinline__ void store4(float* p, v4f v, int64_t left) {
  if (left >= 4) {
    *reinterpret_cast<v4f*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, v4f v, int64_t left) {
  const uint32_t lo = mx_bf16x2(v[0], v[1]), hi = mx_bf16x2(v[2], v[3]);
  if (left >= 4) {
    *reinterpret_cast<nt_u32x2*>(p) = nt_u32x2{lo, hi};
  } else {
    if (left > 0) p[0] = (uint16_t)lo;
    if (left > 1) p[1] = (uint16_t)(lo >> 16);
    if (left > 2) p[2] = (uint16_t)hi;
  }
}

// ---------------------------------------------------------------------------
// Few rows of A.  A workgroup owns 16 MT rows of A x 16 NT rows of B; its
// waves split K in contiguous runs of 128-wide chunks and add up their
// accumulators through LDS at the end, in a fixed order.  B goes from memory
// to the matrix cores' registers without LDS: each of its bytes is used by
// one wave only.  v_mfma_scale_f32_16x16x128: lane l holds row l & 15 of both
// operands and, with g = l >> 4, the 32 E2M1 elements 32 g .. +31 of the
// chunk (16 bytes), or of FP8 the bytes 16 g .. +15 and 64 + 16 g .. +15; the
// scale of the chunk's 32-wide block g is taken from the lanes of group g.
// Operands are swapped (B first), so a lane's four results are four
// consecutive columns of C.
// ---------------------------------------------------------------------------
template <int AFMT, int MT, int NT, int WAVES, typename OutT>
__global__ __launch_bounds__(WAVES * 64) void few_rows_kernel(int M, int N, int K, const uint8_t* __restrict__ A,
                                                              int64_t lda, const uint8_t* __restrict__ SA,
                                                              const uint8_t* __restrict__ B, int64_t ldb,
                                                              const uint8_t* __restrict__ SB, OutT* __restrict__ C,
                                                              int64_t ldc) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ v4f red[WAVES > 1 ? (WAVES - 1) * MT * NT * 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int chunks = K >> 7, sk = K >> 5;
  const int c0 = (int)((int64_t)chunks * wave / WAVES), c1 = (int)((int64_t)chunks * (wave + 1) / WAVES);
  const uint8_t *bp[NT], *sbp[NT], *ap[MT], *sap[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = min(n0 + 16 * t + r, N - 1);  // rows past the end: results dropped
    bp[t] = B + row * ldb + 16 * g;
    sbp[t] = SB + row * sk;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t row = min(m0 + 16 * t + r, M - 1);
    ap[t] = A + row * lda + 16 * g;
    sap[t] = SA + row * sk;
  }
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = c0; c < c1; ++c) {
    v8i bf[NT], af[MT];
    int bs[NT], as[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const v4i v = *reinterpret_cast<const v4i*>(bp[t] + c * 64);
      bf[t] = v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      bs[t] = *reinterpret_cast<const int*>(sbp[t] + c * 4) >> (8 * g);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if constexpr (AFMT == kE2M1) {
        const v4i v = *reinterpret_cast<const v4i*>(ap[t] + c * 64);
        af[t] = v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      } else {
        const v4i v = *reinterpret_cast<const v4i*>(ap[t] + c * 128);
        const v4i u = *reinterpret_cast<const v4i*>(ap[t] + c * 128 + 64);
        af[t] = v8i{v[0], v[1], v[2], v[3], u[0], u[1], u[2], u[3]};
      }
      as[t] = *reinterpret_cast<const int*>(sap[t] + c * 4) >> (8 * g);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af[i], acc[i][j], kMfmaFmt<kE2M1>,
                                                                    kMfmaFmt<AFMT>, 0, bs[j], 0, as[i]);
  }
  mfma_retire_pad();
  if constexpr (WAVES > 1) {
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[(((wave - 1) * MT + i) * NT + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
    for (int w = 0; w < WAVES - 1; ++w) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] += red[((w * MT + i) * NT + j) * 64 + lane];
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + r;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + 16 * j + 4 * g;
      store4(C + (int64_t)m * ldc + n, acc[i][j], N - n);
    }
  }
#endif
}

template <int AFMT, int MT, int NT, int WAVES>
void few_rows(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
              int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, hipStream_t stream) {
  const dim3 grid((uint32_t)((N + 16 * NT - 1) / (16 * NT)), (uint32_t)((M + 16 * MT - 1) / (16 * MT)));
  if (c_dtype == 0)
    hipLaunchKernelGGL((few_rows_kernel<AFMT, MT, NT, WAVES, float>), grid, dim3(WAVES * 64), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, static_cast<float*>(c), ldc);
  else
    hipLaunchKernelGGL((few_rows_kernel<AFMT, MT, NT, WAVES, uint16_t>), grid, dim3(WAVES * 64), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, static_cast<uint16_t*>(c), ldc);
}

template <int AFMT>
void gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
          int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, hipStream_t stream) {
  if (M <= 16) few_rows<AFMT, 1, 1, 4>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, stream);
  else few_rows<AFMT, 4, 4, 4>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, stream);
}

}  // namespace mxfp4_detail

void launch_mxfp4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                       const uint8_t* b, int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype,
                       hipStream_t stream) {
  using namespace mxfp4_detail;
  if (a_fmt == 0) gemm<0>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, stream);
  else if (a_fmt == 1) gemm<1>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, stream);
  else gemm<kE2M1>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, stream);
}

}  // namespace mxfp8
