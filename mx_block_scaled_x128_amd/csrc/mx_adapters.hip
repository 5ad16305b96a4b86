// mx_adapters.hip -- low-rank adapters of many requests on MX codes (gfx950):
// the projection p[t] = alpha[a] * down[a] x[t], a = ids[t], and the adapters'
// gradients sum over the rows t of a of p[t] (x) z[t].  The second half of the
// forward pass, c[t] += up[a] p[t], is part of the product (mxfp4_gemm.hip).
//
// x and z are MX codes, the adapters bf16, p and the sums fp32.  A code times
// its scale is a bf16 value, so the projection's products are exact; p enters
// the gradients' products as three bf16 parts, all 24 bits.
#include "mx_common.hpp"
#include "mx_launch.hpp"

namespace mxfp8 {

namespace mx_adapters_detail {

#if defined(__HIP_DEVICE_COMPILE__)
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ nt_u32x4 get16(mx_rsrc r, uint32_t lane, uint32_t at) {
  return __builtin_bit_cast(nt_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, at, 0));
}
#endif

// ---------------------------------------------------------------------------
// Projection, a row at a time: a workgroup takes JT ranks of one row, its 256
// threads 8 elements of K each, step after step.  Each row reads its adapter for
// itself, which costs nothing where the rows are few or their adapters differ.
// ---------------------------------------------------------------------------
template <int FMT, int JT>
__global__ __launch_bounds__(256) void project_rows_kernel(int K, const uint8_t* __restrict__ A, int64_t lda,
                                                           const uint8_t* __restrict__ SA,
                                                           const int32_t* __restrict__ ids, int adapters, int rank,
                                                           const uint16_t* __restrict__ down, int64_t ldd,
                                                           int64_t stride, const float* __restrict__ alpha,
                                                           float* __restrict__ p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float red[4][JT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int groups = rank / JT, t = blockIdx.x / groups, j0 = (int)(blockIdx.x % groups) * JT;
  float* to = p + (int64_t)t * rank + j0;
  const int a = ids[t];
  if ((uint32_t)a >= (uint32_t)adapters) {
    if (tid < JT) to[tid] = 0.0f;
    return;
  }
  const mx_rsrc rx = mx_run(A + (int64_t)t * lda), rs = mx_run(SA + (int64_t)t * (K >> 5));
  const mx_rsrc rd = mx_run(down + a * stride + j0 * ldd);
  struct In {
    uint2 x;
    uint32_t s;
    nt_u32x4 d[JT];
  };
  auto load = [&](int k, In& v) __attribute__((always_inline)) {
    const bool in = k < K;
    if constexpr (FMT == kE2M1) v.x = make_uint2(__builtin_amdgcn_raw_buffer_load_b32(rx, in ? k >> 1 : kNowhere, 0, 0), 0);
    else v.x = mx_get_codes(rx, in ? k : kNowhere, 0);
    v.s = mx_get_byte(rs, in ? k >> 5 : kNowhere, 0);
#pragma unroll
    for (int j = 0; j < JT; ++j) v.d[j] = get16(rd, in ? k * 2 : kNowhere, (uint32_t)(j * ldd * 2));
  };
  float sum[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) sum[j] = 0.0f;
  auto add = [&](const In& v) __attribute__((always_inline)) {
    float x[8];
    mx_decode8<FMT>(v.x, mx_factor(v.s), x);
#pragma unroll
    for (int j = 0; j < JT; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sum[j] = __builtin_fmaf(x[2 * q], bf16_lo(v.d[j][q]), sum[j]);
        sum[j] = __builtin_fmaf(x[2 * q + 1], bf16_hi(v.d[j][q]), sum[j]);
      }
    }
  };
  constexpr int STEP = 256 * 8;
  In v0, v1;
  load(tid * 8, v0);
  load(tid * 8 + STEP, v1);
  for (int k = tid * 8; k - tid * 8 < K; k += 2 * STEP) {
    In n0, n1;
    load(k + 2 * STEP, n0);
    load(k + 3 * STEP, n1);
    add(v0);
    add(v1);
    v0 = n0;
    v1 = n1;
  }
#pragma unroll
  for (int j = 0; j < JT; ++j) sum[j] = sum64(sum[j]);
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < JT; ++j) red[wave][j] = sum[j];
  }
  __syncthreads();
  if (tid < JT) to[tid] = (alpha ? alpha[a] : 1.0f) * ((red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]));
#endif
}

// ---------------------------------------------------------------------------
// Projection of many rows.  A workgroup takes 16 TG rows and 16 JC ranks; its
// eight waves split K into runs of 128-wide chunks and add up through LDS in a
// fixed order.  v_mfma_f32_16x16x32_bf16 with the adapter first: lane l holds
// rank, or row, l & 15 and, with g = l >> 4, eight of 32 k.  Which k these are
// is free as long as both sides agree, so a lane takes 16 (E2M1: 32) of a row in
// one load: FP8 k = 64 s + 16 g + 8 h + i of the chunk, E2M1 32 g + 8 h + i.
//
// The rows of a tile may name several adapters: one pass over K for each, of
// which only its own rows are stored.  Other rows' values, infinities and NaN
// among them, stay in columns that are dropped.
// ---------------------------------------------------------------------------
constexpr int kProjectWaves = 8;
template <int FMT, int JC, int TG>
__global__ __launch_bounds__(64 * kProjectWaves) void project_tile_kernel(
    int M, int K, const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ SA,
    const int32_t* __restrict__ ids, int adapters, int rank, const uint16_t* __restrict__ down, int64_t ldd,
    int64_t stride, const float* __restrict__ alpha, float* __restrict__ p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int W = kProjectWaves, ROWS = 16 * TG, XL = FMT == kE2M1 ? 1 : 2;
  __shared__ v4f red[W][JC * TG][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int t0 = (int)blockIdx.x * ROWS, j0 = (int)blockIdx.y * (16 * JC), rows = min(ROWS, M - t0);
  const int chunks = K >> 7, sk = K >> 5;
  const int c0 = (int)((int64_t)chunks * wave / W), c1 = (int)((int64_t)chunks * (wave + 1) / W);
  int id = lane < rows ? ids[t0 + lane] : -1;
  if ((uint32_t)id >= (uint32_t)adapters) id = -1;
  // Rows without an adapter: zeros.
  for (int i = threadIdx.x; i < ROWS * 16 * JC; i += 64 * W) {
    const int t = i / (16 * JC), j = j0 + i % (16 * JC);
    if (t < rows && j < rank && (uint32_t)ids[t0 + t] >= (uint32_t)adapters) p[(int64_t)(t0 + t) * rank + j] = 0.0f;
  }
  const mx_rsrc rx = mx_run(A + (int64_t)t0 * lda), rs = mx_run(SA + (int64_t)t0 * sk);
  uint32_t xo[TG], so[TG], dof[JC];
#pragma unroll
  for (int t = 0; t < TG; ++t) {
    const bool in = 16 * t + r < rows;
    xo[t] = in ? (uint32_t)((16 * t + r) * lda) + 16 * g : kNowhere;
    so[t] = in ? (uint32_t)((16 * t + r) * sk) : kNowhere;
  }
#pragma unroll
  for (int j = 0; j < JC; ++j)
    dof[j] = j0 + 16 * j + r < rank ? (uint32_t)((16 * j + r) * ldd * 2) + (FMT == kE2M1 ? 64 : 32) * g : kNowhere;
  struct In {
    nt_u32x4 x[TG][XL], d[JC][4];
    uint32_t s[TG];
  };
  for (uint64_t todo = __ballot(id >= 0); todo;) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == a);
    const mx_rsrc rd = mx_run(down + a * stride + j0 * ldd);
    auto load = [&](int c, In& v) __attribute__((always_inline)) {
      const bool in = c < c1;
#pragma unroll
      for (int t = 0; t < TG; ++t) {
        v.s[t] = __builtin_amdgcn_raw_buffer_load_b32(rs, in ? so[t] : kNowhere, c * 4, 0);
#pragma unroll
        for (int s = 0; s < XL; ++s) v.x[t][s] = get16(rx, in ? xo[t] : kNowhere, c * (64 * XL) + 64 * s);
      }
#pragma unroll
      for (int j = 0; j < JC; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v.d[j][q] = get16(rd, in ? dof[j] : kNowhere, c * 256 + (FMT == kE2M1 ? 16 * q : 128 * (q >> 1) + 16 * (q & 1)));
    };
    v4f acc[JC][TG];
#pragma unroll
    for (int j = 0; j < JC; ++j)
#pragma unroll
      for (int t = 0; t < TG; ++t) acc[j][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    In v;
    load(c0, v);
    for (int c = c0; c < c1; ++c) {
      In next;
      load(c + 1, next);
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t byte = (v.s[t] >> (FMT == kE2M1 ? 8 * g : 16 * (q >> 1) + 8 * (g >> 1))) & 255u;
          const mx_bf8 x = FMT == kE2M1 ? mx_bf16x8<FMT>(v.x[t][0][q], 0, byte)
                                        : mx_bf16x8<FMT>(v.x[t][(q >> 1) % XL][2 * (q & 1)],
                                                         v.x[t][(q >> 1) % XL][2 * (q & 1) + 1], byte);
#pragma unroll
          for (int j = 0; j < JC; ++j)
            acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, v.d[j][q]), x, acc[j][t], 0, 0, 0);
        }
      v = next;
    }
#pragma unroll
    for (int j = 0; j < JC; ++j)
#pragma unroll
      for (int t = 0; t < TG; ++t) red[wave][j * TG + t][lane] = acc[j][t];
    __syncthreads();
    for (int f = wave; f < JC * TG; f += W) {
      v4f s = red[0][f][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) s += red[w][f][lane];
      const int t = f % TG * 16 + r, j = j0 + f / TG * 16 + 4 * g;
      if (__shfl(id, t) == a && j < rank)
        *reinterpret_cast<v4f*>(p + (int64_t)(t0 + t) * rank + j) = s * (alpha ? alpha[a] : 1.0f);
    }
    __syncthreads();
  }
#endif
}

// ---------------------------------------------------------------------------
// Gradients: out[a][j][c] = sum over the rows t of a of p[t][j] z[t][c].
// A workgroup takes 16 NF columns, 16 JT ranks, one adapter and one run of the
// rows.  It lists its adapter's rows among the next 512 in LDS, in order, and
// its four waves take 32 of the list in turn; rows of other adapters are not
// read.  v_mfma_f32_16x16x32_bf16 with z first: lane l = (m, g) loads NF columns
// from column NF m of the rows 8 g .. 8 g + 7 of the 32, and column i of each
// lane's makes fragment i, eight rows deep: the transposition is the choice of
// bytes at the conversion.  p, as three parts, is the other operand.
//
// The runs' sums go to `part` and are joined in order; with one run they are
// the result.
// ---------------------------------------------------------------------------
[[maybe_unused]] constexpr int kWindow = 512;
constexpr int kGradThreads = 256;
template <int FMT>
__device__ __forceinline__ mx_f2 two_codes(uint32_t w, float scale, int pair) {
#if defined(__HIP_DEVICE_COMPILE__)
  // pair: which two codes of the word (FP8: 0, 1; E2M1: 0 to 3)
  if constexpr (FMT == kE2M1) {
    return pair == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0)
           : pair == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1)
           : pair == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2)
                       : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  } else if constexpr (FMT == 0) {
    return pair == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false)
                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
  } else {
    return pair == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, false)
                     : __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, scale, true);
  }
#else
  return mx_f2{};
#endif
}

struct GradArgs {
  int M, C, rank, adapters, runs, jgroups, ctiles;
  int transposed;
  int64_t ldz;
  float* out;    // one run: the gradients; else [runs] of them
  int* counts;   // [runs][adapters] rows found, with more than one run
};

template <int FMT, int JT, int NF>
__global__ __launch_bounds__(kGradThreads, 2) void grad_kernel(GradArgs q, const uint8_t* __restrict__ Z,
                                                               const uint8_t* __restrict__ SZ,
                                                               const float* __restrict__ p,
                                                               const int32_t* __restrict__ ids) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int WORDS = FMT == kE2M1 ? NF / 8 : NF / 4, PER = FMT == kE2M1 ? 8 : 4;  // words of a lane and row, codes of a word
  __shared__ int list[kWindow];
  __shared__ int found[kWindow / 64];
  __shared__ v4f red[2][NF * JT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  int b = (int)blockIdx.x;
  const int ct = b % q.ctiles;
  b /= q.ctiles;
  const int jg = b % q.jgroups;
  b /= q.jgroups;
  const int a = b % q.adapters, run = b / q.adapters;
  const int first = (int)((int64_t)q.M * run / q.runs), end = (int)((int64_t)q.M * (run + 1) / q.runs);
  const int c0 = ct * (16 * NF), j0 = jg * (16 * JT), sk = q.C >> 5;
  const int col = c0 + NF * m;
  const bool col_in = col < q.C;
  const uint32_t zo = FMT == kE2M1 ? col >> 1 : col;
  v4f acc[NF][JT];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  struct In {
    uint32_t z[8][WORDS], s[8];
    float p[JT][8];
  };
  int total = 0;
  for (int w0 = first; w0 < end; w0 += kWindow) {
    // This adapter's rows of the window, in order.
    uint64_t mine[kWindow / kGradThreads];
#pragma unroll
    for (int k = 0; k < kWindow / kGradThreads; ++k) {
      const int t = w0 + k * kGradThreads + tid;
      mine[k] = __ballot(t < end && ids[t < end ? t : first] == a);
      if (lane == 0) found[k * 4 + wave] = __builtin_popcountll(mine[k]);
    }
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int k = 0; k < kWindow / 64; ++k) {
      if (k % 4 == wave && (mine[k / 4] >> lane & 1))
        list[n + __builtin_popcountll(mine[k / 4] & ((1ull << lane) - 1))] = k * 64 + lane;
      n += found[k];
    }
    n = __builtin_amdgcn_readfirstlane(n);
    total += n;
    __syncthreads();
    const mx_rsrc rz = mx_run(Z + (int64_t)w0 * q.ldz), rs = mx_run(SZ + (int64_t)w0 * sk);
    const mx_rsrc rp = mx_run(p + (int64_t)w0 * q.rank);
    auto load = [&](int at, In& v) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = at + 8 * g + i;
        const bool in = e < n;
        const uint32_t t = in ? (uint32_t)list[e] : 0;
        const uint32_t off = in && col_in ? t * (uint32_t)q.ldz + zo : kNowhere;
        if constexpr (WORDS == 4) {
          const nt_u32x4 w = get16(rz, off, 0);
#pragma unroll
          for (int k = 0; k < 4; ++k) v.z[i][k] = w[k];
        } else if constexpr (WORDS == 2) {
          const uint2 w = mx_get_codes(rz, off, 0);
          v.z[i][0] = w.x;
          v.z[i][1] = w.y;
        } else {
          v.z[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rz, off, 0, 0);
        }
        v.s[i] = mx_get_byte(rs, in && col_in ? t * (uint32_t)sk + (col >> 5) : kNowhere, 0);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int rk = j0 + 16 * j + m;
          v.p[j][i] = __uint_as_float(
              __builtin_amdgcn_raw_buffer_load_b32(rp, in && rk < q.rank ? (t * (uint32_t)q.rank + rk) * 4 : kNowhere, 0, 0));
        }
      }
    };
    In v;
    load(wave * 32, v);
    for (int at = wave * 32; at < n; at += 128) {
      In next;
      load(at + 128, next);
      MxParts pp[JT];
#pragma unroll
      for (int j = 0; j < JT; ++j) pp[j] = mx_parts(v.p[j]);
#pragma unroll
      for (int k = 0; k < WORDS; ++k)
#pragma unroll
        for (int h = 0; h < PER / 2; ++h) {
          nt_u32x4 even, odd;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const mx_f2 x = two_codes<FMT>(v.z[2 * i][k], __uint_as_float(v.s[2 * i] << 23), h);
            const mx_f2 y = two_codes<FMT>(v.z[2 * i + 1][k], __uint_as_float(v.s[2 * i + 1] << 23), h);
            even[i] = mx_bf16x2(x.x, y.x);
            odd[i] = mx_bf16x2(x.y, y.y);
          }
          const int f = k * PER + 2 * h;
#pragma unroll
          for (int j = 0; j < JT; ++j)
#pragma unroll
            for (int part = 2; part >= 0; --part) {
              acc[f][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, even), pp[j].part[part], acc[f][j], 0, 0, 0);
              acc[f + 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, odd), pp[j].part[part], acc[f + 1][j], 0, 0, 0);
            }
        }
      v = next;
    }
    __syncthreads();  // the list has been read
  }
  if (q.counts && ct == 0 && jg == 0 && tid == 0) q.counts[run * q.adapters + a] = total;
  if (q.counts && total == 0) return;  // nothing to add: the join leaves it out
  // Waves 2 and 3 to 0 and 1, then 1 to 0.
#pragma unroll
  for (int half = 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < JT; ++j) red[wave - half][f * JT + j][lane] = acc[f][j];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < JT; ++j) acc[f][j] += red[wave][f * JT + j][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  // A lane holds rank m and, of fragment f, the columns NF (4 g + i) + f.
  float* out = q.out + ((int64_t)run * q.adapters + a) * q.rank * q.C;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int rk = j0 + 16 * j + m;
    if (rk >= q.rank) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + NF * (4 * g + i);
      if (c >= q.C) continue;
      if (q.transposed) {
#pragma unroll
        for (int f = 0; f < NF; ++f) out[(int64_t)(c + f) * q.rank + rk] = acc[f][j][i];
      } else {
#pragma unroll
        for (int f = 0; f < NF; f += 4)
          *reinterpret_cast<v4f*>(out + (int64_t)rk * q.C + c + f) =
              v4f{acc[f][j][i], acc[f + 1][j][i], acc[f + 2][j][i], acc[f + 3][j][i]};
      }
    }
  }
#endif
}

// out = the sums of the runs that found rows, in order.  n: 16-byte units of an adapter.
__global__ __launch_bounds__(256) void grad_join_kernel(const nt_f32x4* __restrict__ part, const int* __restrict__ counts,
                                                        int runs, int adapters, int64_t n, nt_f32x4* __restrict__ out) {
  const int a = blockIdx.y;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    nt_f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 0; r < runs; ++r)
      if (counts[r * adapters + a]) s += part[((int64_t)r * adapters + a) * n + i];
    out[a * n + i] = s;
  }
}

template <int FMT>
void project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const int32_t* ids,
             int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd, int64_t stride, const float* alpha,
             float* p, hipStream_t stream) {
  if (M <= 256) {
    // One rank a workgroup until four fill the chip.
#define MXFP8_PR(JT)                                                                                            \
  hipLaunchKernelGGL((project_rows_kernel<FMT, JT>), dim3((uint32_t)(M * (rank / JT))), dim3(256), 0, stream,   \
                     (int)K, a, lda, sa, ids, (int)adapters, (int)rank, down, ldd, stride, alpha, p)
    if (M * rank < 4 * 256) MXFP8_PR(1);
    else MXFP8_PR(4);
#undef MXFP8_PR
    return;
  }
#define MXFP8_PT(JC, TG)                                                                                        \
  hipLaunchKernelGGL((project_tile_kernel<FMT, JC, TG>),                                                        \
                     dim3((uint32_t)((M + 16 * TG - 1) / (16 * TG)), (uint32_t)((rank + 16 * JC - 1) / (16 * JC))), \
                     dim3(64 * kProjectWaves), 0, stream, (int)M, (int)K, a, lda, sa, ids, (int)adapters,       \
                     (int)rank, down, ldd, stride, alpha, p)
  if (rank <= 16) MXFP8_PT(1, 2);
  else if (rank <= 32) MXFP8_PT(2, 2);
  else MXFP8_PT(4, 2);
#undef MXFP8_PT
}

// Ranks and columns of a workgroup, and the runs that the rows are split into.
struct GradShape {
  int jt, nf, jgroups, ctiles, runs;
};
GradShape grad_shape(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  GradShape s;
  s.jt = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
  s.nf = s.jt == 4 ? 8 : 16;
  s.jgroups = (int)((rank + 16 * s.jt - 1) / (16 * s.jt));
  s.ctiles = (int)((C + 16 * s.nf - 1) / (16 * s.nf));
  // Workgroups for the chip twice over, runs of 256 rows at least, and at most
  // 256 MB of partial sums.
  const int64_t wgs = (int64_t)s.ctiles * s.jgroups * adapters;
  int64_t runs = (1024 + wgs - 1) / wgs;
  const int64_t most = (M + 255) / 256, bytes = adapters * rank * C * 4;
  if (runs > most) runs = most;
  if (runs * bytes > (int64_t(256) << 20)) runs = (int64_t(256) << 20) / bytes;
  s.runs = (int)(runs < 1 ? 1 : runs);  // M == 0: one run of no rows, which gives zeros
  return s;
}

template <int FMT>
void grad(const GradShape& s, const GradArgs& q, const uint8_t* z, const uint8_t* sz, const float* p,
          const int32_t* ids, hipStream_t stream) {
  const dim3 grid((uint32_t)s.ctiles * (uint32_t)s.jgroups * (uint32_t)q.adapters * (uint32_t)s.runs);
  if (s.jt == 1) hipLaunchKernelGGL((grad_kernel<FMT, 1, 16>), grid, dim3(kGradThreads), 0, stream, q, z, sz, p, ids);
  else if (s.jt == 2) hipLaunchKernelGGL((grad_kernel<FMT, 2, 16>), grid, dim3(kGradThreads), 0, stream, q, z, sz, p, ids);
  else hipLaunchKernelGGL((grad_kernel<FMT, 4, 8>), grid, dim3(kGradThreads), 0, stream, q, z, sz, p, ids);
}

}  // namespace mx_adapters_detail

using namespace mx_adapters_detail;

void launch_mx_adapter_project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                               const int32_t* ids, int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd,
                               int64_t stride, const float* alpha, float* p, hipStream_t stream) {
  if (a_fmt == 0) project<0>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, stream);
  else if (a_fmt == 1) project<1>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, stream);
  else project<kE2M1>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, stream);
}

int64_t adapter_grad_workspace(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  const GradShape s = grad_shape(M, C, rank, adapters);
  if (s.runs == 1) return 0;
  return (int64_t)s.runs * adapters * (rank * C * 4 + 4);
}

int64_t adapter_grad_groups(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  const GradShape s = grad_shape(M, C, rank, adapters);
  return (int64_t)s.ctiles * s.jgroups * adapters * s.runs;
}

void launch_mx_adapter_grad(int64_t M, int64_t C, const uint8_t* z, int64_t ldz, int z_fmt, const uint8_t* sz,
                            const float* p, int64_t rank, const int32_t* ids, int64_t adapters, int transposed,
                            float* out, void* workspace, hipStream_t stream) {
  const GradShape s = grad_shape(M, C, rank, adapters);
  GradArgs q;
  q.M = (int)M, q.C = (int)C, q.rank = (int)rank, q.adapters = (int)adapters;
  q.runs = s.runs, q.jgroups = s.jgroups, q.ctiles = s.ctiles, q.transposed = transposed, q.ldz = ldz;
  q.out = s.runs == 1 ? out : static_cast<float*>(workspace);
  q.counts = s.runs == 1 ? nullptr : reinterpret_cast<int*>(q.out + s.runs * adapters * rank * C);
  if (z_fmt == 0) grad<0>(s, q, z, sz, p, ids, stream);
  else if (z_fmt == 1) grad<1>(s, q, z, sz, p, ids, stream);
  else grad<kE2M1>(s, q, z, sz, p, ids, stream);
  if (s.runs > 1) {
    const int64_t n = rank * C / 4, need = (n + 255) / 256;
    hipLaunchKernelGGL(grad_join_kernel, dim3((uint32_t)(need < 1024 ? need : 1024), (uint32_t)adapters), dim3(256), 0,
                       stream, reinterpret_cast<const nt_f32x4*>(workspace), q.counts, s.runs, (int)adapters, n,
                       reinterpret_cast<nt_f32x4*>(out));
  }
}

}  // namespace mxfp8
