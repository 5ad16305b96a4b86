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

#if defined(__HIP_DEVICE_COMPILE__)
// Four ranks of a row of p into its packed parts.
__device__ __forceinline__ void put_packed(const MxPacked& packed, int64_t t, int j, v4f v) {
  uint16_t* to = packed.place(t, j);
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = __float_as_uint(v[k]) & 0xFFFF0000u;
      v[k] -= __uint_as_float(w[k]);
    }
    *reinterpret_cast<nt_u32x2*>(to + part * 512) = nt_u32x2{w[0] >> 16 | w[1], w[2] >> 16 | w[3]};
  }
}
#endif

// ---------------------------------------------------------------------------
// Projection, a row at a time: a workgroup takes JT ranks of one row, its 256
// threads 8 elements of K each, step after step, the next two steps on their way.
// Each row reads its adapter for itself, which costs nothing where the rows are
// few or their adapters differ.  One row of 3584, rank 16: 3.5 us, a launch and
// the reads' latency; 61 rows of 18944, rank 64, 32 adapters: 17 us (78 MB of
// adapters, 148 MB of reads: 8.7 TB/s, mostly from the caches).
// ---------------------------------------------------------------------------
template <int FMT, int JT>
__global__ __launch_bounds__(256) void project_rows_kernel(int K, const uint8_t* __restrict__ A, int64_t lda,
                                                           const uint8_t* __restrict__ SA,
                                                           const int32_t* __restrict__ ids, int adapters, int rank,
                                                           const uint16_t* __restrict__ down, int64_t ldd,
                                                           int64_t stride, const float* __restrict__ alpha,
                                                           float* __restrict__ p, MxPacked packed) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float red[4][JT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int groups = rank / JT, t = __builtin_amdgcn_readfirstlane((int)blockIdx.x / groups);
  const int j0 = ((int)blockIdx.x - t * groups) * JT;
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
  if (tid < JT) {
    float v = (alpha ? alpha[a] : 1.0f) * ((red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]));
    to[tid] = v;
    if (packed.at) {
      uint16_t* one = packed.place(t, (j0 + tid) & ~3) + ((j0 + tid) & 3);
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint32_t w = __float_as_uint(v) & 0xFFFF0000u;
        one[part * 512] = (uint16_t)(w >> 16);
        v -= __uint_as_float(w);
      }
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// Projection of many rows.  A workgroup takes 128 rows, 16 JC ranks and a run of
// K's 128-wide chunks.  Chunks go straight to LDS, three buffers deep: the rows'
// codes and scales and the adapter's ranks, 1 KB of whole row segments an
// instruction (gathering 16 rows x 64 bytes a time costs the load path more than
// twice as much for the same bytes), and the adapter's once for all four waves,
// which take 32 rows each.  The runs' sums go to `part` and are joined in order.
//
// v_mfma_f32_16x16x32_bf16 with the adapter first: lane l holds rank, or row,
// l & 15 and, with g = l >> 4, eight of 32 k.  Which k these are is free as long
// as both sides agree, so a lane reads 16 bytes of a row at once: FP8
// k = 64 s + 16 g + 8 h + i of the chunk, E2M1 32 g + 8 h + i.
//
// The rows of a tile may name several adapters: one pass over the run for each,
// of which only its own rows are stored.  Other rows' values, infinities and NaN
// among them, stay in columns that are dropped.
//
// HBM bounds it with many rows: 8192x18944 rank 16 35 us (166 MB in all, 4.7 TB/s;
// out of the last-level cache 27), 4096x8960 rank 64 13 without the join.
// 8192x3584 rank 16 (10 us) and less are a few rounds of a chunk's latency.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128;
template <int FMT, int JC>
struct ProjectTile {
  static constexpr int XB = FMT == kE2M1 ? 64 : 128;            // bytes of a row per chunk
  static constexpr int X = kTileRows * XB, D = 16 * JC * 256, S = 1024;  // scales: 512 bytes, and as many that nobody reads
  static constexpr int STAGE = X + D + S;
};

#if defined(__HIP_DEVICE_COMPILE__)
typedef __attribute__((address_space(3))) void lds_void;
template <int BYTES>
__device__ __forceinline__ void load_lds(mx_rsrc r, uint8_t* to, uint32_t lane_off, uint32_t off) {
  if constexpr (BYTES == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, lane_off, off, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, lane_off, off, 0, 0);
}
// All but the last N of this wave's loads have landed, and its LDS reads; then
// all waves meet.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N >= 0 && N <= 63, "vmcnt");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// The next adapter that a lane's two ids name, or -1.
__device__ __forceinline__ int next_of(int id0, int id1) {
  const uint64_t a = __ballot(id0 >= 0), b = __ballot(id1 >= 0);
  return a ? __builtin_amdgcn_readlane(id0, __builtin_ctzll(a)) : b ? __builtin_amdgcn_readlane(id1, __builtin_ctzll(b)) : -1;
}
#endif

// part: [runs][M][rank]; runs == 1: p itself, and its packed parts.
template <int FMT, int JC>
__global__ __launch_bounds__(256) void project_tile_kernel(int M, int K, int runs, const uint8_t* __restrict__ A,
                                                           int64_t lda, const uint8_t* __restrict__ SA,
                                                           const int32_t* __restrict__ ids, int adapters, int rank,
                                                           const uint16_t* __restrict__ down, int64_t ldd,
                                                           int64_t stride, const float* __restrict__ alpha,
                                                           float* __restrict__ part, MxPacked packed) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef ProjectTile<FMT, JC> T;
  // Three arrays, so that the compiler's waits for what is on its way to one do
  // not hold up reads of another.
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[T::STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t ring1[T::STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t ring2[T::STAGE];
  constexpr int XI = T::X / 4096, DI = T::D / 4096;  // loads of a wave and chunk; scales: one more
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  // Quotients come from the vector unit: back to scalar registers, for the descriptors.
  const int tile = __builtin_amdgcn_readfirstlane((int)blockIdx.x / runs), run = (int)blockIdx.x - tile * runs;
  const int t0 = tile * kTileRows, j0 = (int)blockIdx.y * (16 * JC), rows = min(kTileRows, M - t0);
  const int chunks = K >> 7, sk = K >> 5;
  const int per = (chunks + runs - 1) / runs, c0 = min(run * per, chunks), c1 = min(c0 + per, chunks);
  auto id_of = [&](int t) __attribute__((always_inline)) {
    const int id = t < rows ? ids[t0 + t] : -1;
    return (uint32_t)id < (uint32_t)adapters ? id : -1;
  };
  int id0 = id_of(lane), id1 = id_of(64 + lane);
  // The rows whose results this lane holds.
  const int own[2] = {id_of(wave * 32 + r), id_of(wave * 32 + 16 + r)};
  float* to = part + ((int64_t)run * M + t0) * rank;
  if (runs == 1 && blockIdx.z == 0) {
    for (int i = threadIdx.x; i < rows * 16 * JC; i += 256) {
      const int t = i / (16 * JC), j = j0 + i % (16 * JC);
      if (j < rank && (uint32_t)ids[t0 + t] >= (uint32_t)adapters) to[(int64_t)t * rank + j] = 0.0f;
    }
  }
  int first = t0;
  asm volatile("" : "+s"(first));  // in a scalar register: what the loop above made of t0 is not
  const mx_rsrc rx = mx_run(A + (int64_t)first * lda), rs = mx_run(SA + (int64_t)first * sk);
  // 16-byte units of a row sit at unit ^ swizzle(row), so that 16 rows read at
  // one unit spread over the banks.
  auto swz_x = [](int row) { return FMT == kE2M1 ? row >> 2 & 3 : row >> 1 & 7; };
  auto swz_d = [](int row) { return row & 15; };
  uint32_t xo[XI], dof[DI];
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    constexpr int UPR = T::XB / 16;
    const int row = (i * 4 + wave) * (64 / UPR) + lane / UPR;
    xo[i] = row < rows ? (uint32_t)(row * lda) + ((lane % UPR) ^ swz_x(row)) * 16 : kNowhere;
  }
#pragma unroll
  for (int i = 0; i < DI; ++i) {
    const int row = (i * 4 + wave) * 4 + (lane >> 4);
    dof[i] = j0 + row < rank ? (uint32_t)(row * ldd * 2) + ((lane & 15) ^ swz_d(row)) * 16 : kNowhere;
  }
  // Scales: waves 0 and 1 take 64 rows each, the others zeros (their loads count all the same).
  const uint32_t so = wave < 2 && wave * 64 + lane < rows ? (uint32_t)((wave * 64 + lane) * sk) : kNowhere;
  constexpr int LOADS = XI + DI + 1;
  int turn = 0;
  for (int a = next_of(id0, id1); a >= 0; a = next_of(id0, id1)) {
    if (id0 == a) id0 = -1;
    if (id1 == a) id1 = -1;
    const bool other = turn != (int)blockIdx.z;
    turn = turn + 1 == (int)gridDim.z ? 0 : turn + 1;
    if (other) continue;
    const mx_rsrc rd = mx_run(down + a * stride + j0 * ldd);
    auto load = [&](uint8_t* to, int c) __attribute__((always_inline)) {
      const bool in = c < c1;
#pragma unroll
      for (int i = 0; i < XI; ++i) load_lds<16>(rx, to + (i * 4 + wave) * 1024, in ? xo[i] : kNowhere, c * T::XB);
#pragma unroll
      for (int i = 0; i < DI; ++i) load_lds<16>(rd, to + T::X + (i * 4 + wave) * 1024, in ? dof[i] : kNowhere, c * 256);
      load_lds<4>(rs, to + T::X + T::D + wave * 256, in ? so : kNowhere, c * 4);
    };
    v4f acc[JC][2];
#pragma unroll
    for (int j = 0; j < JC; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[j][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto chunk = [&](const uint8_t* at) __attribute__((always_inline)) {
      nt_u32x4 d[JC][4];
#pragma unroll
      for (int j = 0; j < JC; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int unit = FMT == kE2M1 ? 4 * g + q : 8 * (q >> 1) + 2 * g + (q & 1);
          d[j][q] = *reinterpret_cast<const nt_u32x4*>(at + T::X + (16 * j + r) * 256 + (unit ^ swz_d(r)) * 16);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = wave * 32 + 16 * t + r;
        const uint32_t s = *reinterpret_cast<const uint32_t*>(at + T::X + T::D + row * 4);
        nt_u32x4 x[2];
        x[0] = *reinterpret_cast<const nt_u32x4*>(at + row * T::XB + (g ^ swz_x(row)) * 16);
        if constexpr (FMT != kE2M1) x[1] = *reinterpret_cast<const nt_u32x4*>(at + row * T::XB + ((4 + g) ^ swz_x(row)) * 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t byte = (s >> (FMT == kE2M1 ? 8 * g : 16 * (q >> 1) + 8 * (g >> 1))) & 255u;
          const mx_bf8 v = FMT == kE2M1 ? mx_bf16x8<FMT>(x[0][q], 0, byte)
                                        : mx_bf16x8<FMT>(x[q >> 1][2 * (q & 1)], x[q >> 1][2 * (q & 1) + 1], byte);
#pragma unroll
          for (int j = 0; j < JC; ++j)
            acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, d[j][q]), v, acc[j][t], 0, 0, 0);
        }
      }
    };
    // Chunk c is there when all but the chunk after it has landed; the buffer
    // that c + 2 goes to, that of c - 1, has then been read by everybody.
    load(ring0, c0);
    load(ring1, c0 + 1);
    for (int c = c0; c < c1; c += 3) {
      wait_and_meet<LOADS>();
      load(ring2, c + 2);
      chunk(ring0);
      if (c + 1 >= c1) break;
      wait_and_meet<LOADS>();
      load(ring0, c + 3);
      chunk(ring1);
      if (c + 2 >= c1) break;
      wait_and_meet<LOADS>();
      load(ring1, c + 4);
      chunk(ring2);
    }
    wait_and_meet<0>();  // nothing is on its way, nobody reads: the ring may start again
    const float f = runs == 1 && alpha ? alpha[a] : 1.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < JC; ++j)
        if (own[t] == a && j0 + 16 * j + 4 * g < rank) {
          const int row = wave * 32 + 16 * t + r, rk = j0 + 16 * j + 4 * g;
          const v4f v = acc[j][t] * f;
          *reinterpret_cast<v4f*>(to + (int64_t)row * rank + rk) = v;
          if (runs == 1 && packed.at) put_packed(packed, t0 + row, rk, v);
        }
  }
#endif
}

// p = alpha times the runs' sums, in order; four ranks a thread.
__global__ __launch_bounds__(256) void project_join_kernel(const nt_f32x4* __restrict__ part, int runs, int64_t units,
                                                           int upr, const int32_t* __restrict__ ids, int adapters,
                                                           const float* __restrict__ alpha, nt_f32x4* __restrict__ p,
                                                           MxPacked packed) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < units; i += step) {
    const int a = ids[i / upr];
    const bool some = (uint32_t)a < (uint32_t)adapters;
    nt_f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int r = 0; r < runs; ++r) s += part[r * units + i];
    const float f = some && alpha ? alpha[a] : 1.0f;
    p[i] = some ? s * f : nt_f32x4{0.0f, 0.0f, 0.0f, 0.0f};  // rows without an adapter: nothing was written
#if defined(__HIP_DEVICE_COMPILE__)
    if (some && packed.at) put_packed(packed, i / upr, (int)(i % upr) * 4, s * f);
#endif
  }
}

// ---------------------------------------------------------------------------
// Gradients: out[a][j][c] = sum over the rows t of a of p[t][j] z[t][c].
// A workgroup takes 16 NF columns, 16 JT ranks, one adapter and one run of the
// rows.  It lists its adapter's rows among the next 2048 in LDS, in order, and
// its four waves take 32 of the list in turn; rows of other adapters are not
// read.  v_mfma_f32_16x16x32_bf16 with z first: lane l = (m, g) loads NF columns
// from column NF m of the rows 8 g .. 8 g + 7 of the 32, and column i of each
// lane's makes fragment i, eight rows deep: the transposition is the choice of
// bytes at the conversion.  p, as three parts, is the other operand: a lane loads
// the JT ranks from JT m of its rows, rank i of each lane's for fragment i.  The
// scales of the 32 rows come with one load and go to their lanes from there.
// What bounds it: up to 16 ranks the reads, 17 load instructions for 32 rows
// (8192x18944 rank 16 40 us, 3.9 TB/s; 8192x3584 16); past that instructions, a
// third of them p's split into its parts (4096x8960 rank 64 27 us; matrix
// instructions 25 % of the time; each 32 ranks read z again, but side by side on
// one XCD, from its cache, they took as long).
//
// The runs' sums go to `part` and are joined in order; with one run they are
// the result.
// ---------------------------------------------------------------------------
// Rows listed at once: 2048, or 512 where as many rows would pass 32-bit offsets.
[[maybe_unused]] constexpr int kWindow = 2048, kSmallWindow = 512;
constexpr int kGradThreads = 256;
// Two codes of a word (FP8: pair 0, 1; E2M1: 0 to 3) -> two bf16 values, exactly.
template <int FMT>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, float scale, int pair) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (FMT == kE2M1) {
    return __builtin_bit_cast(uint32_t, pair == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)
                                        : pair == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)
                                        : pair == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)
                                                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  } else if constexpr (FMT == 0) {
    return __builtin_bit_cast(uint32_t, pair == 0 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)
                                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true));
  } else {
    return __builtin_bit_cast(uint32_t, pair == 0 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false)
                                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true));
  }
#else
  return 0;
#endif
}

#if defined(__HIP_DEVICE_COMPILE__)
// Four scale bytes, `left` of them in the row: DWORD where rows start on one,
// else one by one.  (A choice made here would leave the count of loads on their
// way open, and every wait would be for all of them.)
template <bool DWORD>
__device__ __forceinline__ uint32_t load_scales(mx_rsrc r, uint32_t off, int left) {
  if constexpr (DWORD) return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) w |= mx_get_byte(r, k < left ? off : kNowhere, k) << (8 * k);
  return w;
}
#endif

struct GradArgs {
  int M, C, rank, adapters, runs, jgroups, ctiles;
  int per;     // rows of a run
  int window;  // kWindow or kSmallWindow
  int transposed;
  int64_t ldz;
  float* out;    // one run: the gradients; else [runs] of them
  int* counts;   // [runs][adapters] rows found, with more than one run
};

template <int FMT, int JT, int NF, bool DWORD>
__global__ __launch_bounds__(kGradThreads, 2) void grad_kernel(GradArgs q, const uint8_t* __restrict__ Z,
                                                               const uint8_t* __restrict__ SZ,
                                                               const float* __restrict__ p,
                                                               const int32_t* __restrict__ ids) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int WORDS = FMT == kE2M1 ? NF / 8 : NF / 4, CPW = FMT == kE2M1 ? 8 : 4;  // words of a lane and row, codes of a word
  // The list is filled up to whole steps of all waves, and two steps more, which are loaded ahead.
  __shared__ __attribute__((aligned(16))) uint32_t list[kWindow + 384];
  __shared__ int found[4];
  __shared__ v4f red[2][NF * JT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  // Quotients come from the vector unit: back to scalar registers, for the descriptors.
  const int b1 = __builtin_amdgcn_readfirstlane((int)blockIdx.x / q.ctiles), ct = (int)blockIdx.x - b1 * q.ctiles;
  const int b2 = __builtin_amdgcn_readfirstlane(b1 / q.jgroups), jg = b1 - b2 * q.jgroups;
  const int run = __builtin_amdgcn_readfirstlane(b2 / q.adapters), a = b2 - run * q.adapters;
  const int first = min(run * q.per, q.M), end = min(first + q.per, q.M);
  const int c0 = ct * (16 * NF), j0 = jg * (16 * JT), sk = q.C >> 5;
  // Columns and ranks past the last ones: the last ones again, for results that nobody stores.
  const int col = min(c0 + NF * m, q.C - NF), rk_in = min(j0 + JT * m, q.rank - JT);
  const uint32_t zo = FMT == kE2M1 ? col >> 1 : col;
  v4f acc[NF][JT];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int SB = NF / 2;                      // scale bytes of a row: its 16 NF columns
  constexpr int LPR = SB / 4;                     // lanes that load them, four each
  struct In {
    uint32_t z[8][WORDS], s;
    float p[8][JT];
  };
  // Which lane has the scale of row 8 g + i, and which byte it is there.
  const int block = (col >> 5) - (c0 >> 5);
  const int s_from = (8 * g * LPR + block / 4) * 4, s_shift = 8 * (block % 4);
  const uint32_t s_col = (uint32_t)(c0 >> 5) + 4 * (lane % LPR);
  int total = 0;
  for (int w0 = first; w0 < end; w0 += q.window) {
    // This adapter's rows of the window, in order: each wave counts those in a
    // quarter of it, then places them behind those of the waves before.
    const int span = min(q.window, end - w0), share = (span + 255) / 256;  // of 64 rows
    int own = lane;
    asm volatile("" : "+v"(own));  // what follows from it is not kept in registers from window to window
    constexpr int MOST = kWindow / 256;
    uint64_t mine[MOST];
    int n = 0, id[MOST];
    const mx_rsrc ri = mx_run(ids + w0);
#pragma unroll
    for (int k = 0; k < MOST; ++k) {  // all on their way at once
      const int t = (wave * share + k) * 64 + own;
      id[k] = __builtin_amdgcn_raw_buffer_load_b32(ri, k < share && t < span ? t * 4 : kNowhere, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < MOST; ++k)
      mine[k] = __ballot(k < share && (wave * share + k) * 64 + own < span && id[k] == a);
#pragma unroll
    for (int k = 0; k < MOST; ++k) n += __builtin_popcountll(mine[k]);
    if (lane == 0) found[wave] = n;
    __syncthreads();
    int at_row = 0;
    n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k < wave) at_row += found[k];
      n += found[k];
    }
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      if (k < share) {
        if (mine[k] >> own & 1)
          list[at_row + __builtin_popcountll(mine[k] & ((1ull << own) - 1))] = (wave * share + k) * 64 + own;
        at_row += __builtin_popcountll(mine[k]);
      }
    }
    n = __builtin_amdgcn_readfirstlane(n);
    total += n;
    if (n == 0) {
      __syncthreads();  // `found` has been read
      continue;
    }
    __syncthreads();
    // Places past the list's end name its first row, whose p is then not read but zero.
    for (int i = n + tid; i < ((n + 127) & ~127) + 256; i += kGradThreads) list[i] = list[0];
    __syncthreads();
    const mx_rsrc rz = mx_run(Z + (int64_t)w0 * q.ldz), rs = mx_run(SZ + (int64_t)w0 * sk);
    const mx_rsrc rp = mx_run(p + (int64_t)w0 * q.rank);
    auto load = [&](int at, In& v) __attribute__((always_inline)) {
      const nt_u32x4 lo = *reinterpret_cast<const nt_u32x4*>(list + at + 8 * g);
      const nt_u32x4 hi = *reinterpret_cast<const nt_u32x4*>(list + at + 8 * g + 4);
      const bool whole = at + 32 <= n;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t t = i < 4 ? lo[i % 4] : hi[i % 4];
        const uint32_t off = __umul24(t, (uint32_t)q.ldz) + zo;
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
        uint32_t po = __umul24(t, (uint32_t)q.rank * 4) + (uint32_t)rk_in * 4;
        if (!whole && at + 8 * g + i >= n) po = kNowhere;
        if constexpr (JT == 2) {
          const uint2 w = mx_get_codes(rp, po, 0);
          v.p[i][0] = __uint_as_float(w.x);
          v.p[i][1] = __uint_as_float(w.y);
        } else {
          v.p[i][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rp, po, 0, 0));
        }
      }
      // Row lane / LPR of the 32; bytes past the row's end are of columns that nobody stores.
      const uint32_t t = list[at + (lane / LPR) % 32];
      const bool in = lane < 32 * LPR && s_col < (uint32_t)sk;
      v.s = load_scales<DWORD>(rs, in ? __umul24(t, (uint32_t)sk) + s_col : kNowhere, sk - (int)s_col);
    };
    auto multiply = [&](const In& v) __attribute__((always_inline)) {
      float scale[8];
      int from = s_from;
      asm volatile("" : "+v"(from));  // one register, not one to each of the eight
      uint32_t sw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sw[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from + 4 * LPR * i, (int)v.s);
#pragma unroll
      for (int i = 0; i < 8; ++i) scale[i] = __uint_as_float((sw[i] >> s_shift & 255u) << 23);
      MxParts pp[JT];
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v.p[i][j];
        pp[j] = mx_parts(f);
      }
      // A word's columns at a time: as many fragments.
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        nt_u32x4 zf[CPW];
#pragma unroll
        for (int h = 0; h < CPW / 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = two_codes<FMT>(v.z[2 * i][k], scale[2 * i], h);
            const uint32_t y = two_codes<FMT>(v.z[2 * i + 1][k], scale[2 * i + 1], h);
            zf[2 * h][i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            zf[2 * h + 1][i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
          }
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int f = 0; f < CPW; ++f)
              acc[k * CPW + f][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, zf[f]), pp[j].part[part],
                                                                            acc[k * CPW + f][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Two steps' rows in registers, in turn (a copy from one to the other would
    // cost a fifth of a step's instructions).  Loads stay where they are written:
    // the compiler would move them behind the branch, down to their use.
    auto ask = [&](int at, In& x) __attribute__((always_inline)) {
      load(at, x);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    In v, w;
    ask(wave * 32, v);
    ask(wave * 32 + 128, w);
    for (int at = wave * 32; at < n; at += 256) {
      multiply(v);
      ask(at + 256, v);
      if (at + 128 >= n) break;
      multiply(w);
      ask(at + 384, w);
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
  // A lane holds ranks JT m + j and, of fragment f, the columns NF (4 g + i) + f.
  float* out = q.out + ((int64_t)run * q.adapters + a) * q.rank * q.C;
  const int rk = j0 + JT * m;
  if (rk >= q.rank) return;  // rk_in of another lane
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + NF * (4 * g + i);
    if (c >= q.C) continue;
    if (q.transposed) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < JT; ++j) out[(int64_t)(c + f) * q.rank + rk + j] = acc[f][j][i];
    } else {
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int f = 0; f < NF; f += 4)
          *reinterpret_cast<v4f*>(out + (int64_t)(rk + j) * q.C + c + f) =
              v4f{acc[f][j][i], acc[f + 1][j][i], acc[f + 2][j][i], acc[f + 3][j][i]};
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
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
      const nt_f32x4 v = part[((int64_t)r * adapters + a) * n + i];  // read in any case, used if it was written
      const bool some = counts[r * adapters + a] != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += some ? v[k] : 0.0f;
    }
    out[a * n + i] = s;
  }
}

// Whether rows are taken one by one.  That costs 0.14 us a million of M rank K, whichever adapters they name; a tile
// with its runs and their join 9 to 10 us if the rows name one adapter, and 17 to 50 if they name 32 or more, mixed.
// 512x3584 rank 16: 7.3 row by row against 7.5 in tiles (17 mixed); 192x3584 rank 64: 9.9 against 9.5; 256x3584 rank
// 64: 12.5 against 9.4 (23 mixed); 512x3584 rank 64: 22.8 against 9.7.  Past 512 rows of a short K the tiles' shared
// loads count.
bool row_by_row(int64_t M, int64_t K, int64_t rank) { return M <= 512 && M * rank * K <= 100 * 1000 * 1000; }
int64_t project_tiles(int64_t M, int64_t rank) { return (M + kTileRows - 1) / kTileRows * ((rank + 63) / 64); }
// Runs of K: a workgroup to each of 256 compute units (two to a unit where their buffers would fit: 8192x3584 rank 16
// 11.8 us in place of 9.7; one to two units: 4096x8960 rank 64 20.5 in place of 16.8), of four chunks at least
// (515x8960 rank 8: 8.2 us, with eight 8.6, with two 9.5).
int project_runs(int64_t M, int64_t K, int64_t rank) {
  if (row_by_row(M, K, rank)) return 1;
  const int64_t chunks = K / 128;
  int64_t runs = 256 / project_tiles(M, rank);
  if (runs > chunks / 4) runs = chunks / 4;
  return (int)(runs < 1 ? 1 : runs);
}
// Workgroups that share the adapters of a tile's rows, each a pass over the tile: twice those that there is room
// for (two to a compute unit up to 32 ranks, else one), since a tile may name few, and those without one end at once.  512 rows x 3584 of 32 adapters, mixed, rank 16
// and 64: 17 and 27 us (one workgroup a tile and run: 66 and 120); of one adapter 9 and 11 either way.
int project_split(int64_t M, int64_t rank, int64_t adapters, int runs) {
  int64_t split = 2 * (rank <= 32 ? 512 : 256) / (project_tiles(M, rank) * runs);
  if (split > kTileRows) split = kTileRows;
  if (split > adapters) split = adapters;
  return (int)(split < 1 ? 1 : split);
}

template <int FMT>
void project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const int32_t* ids,
             int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd, int64_t stride, const float* alpha,
             float* p, MxPacked packed, float* workspace, hipStream_t stream) {
  if (row_by_row(M, K, rank)) {
    // One rank a workgroup until four fill the chip (13x8960 rank 8: 3.1 us, with four 4.2; 64x18944 rank 64: 11.5 us
    // with four, 17.0 with one).
#define MXFP8_PR(JT)                                                                                            \
  hipLaunchKernelGGL((project_rows_kernel<FMT, JT>), dim3((uint32_t)(M * (rank / JT))), dim3(256), 0, stream,   \
                     (int)K, a, lda, sa, ids, (int)adapters, (int)rank, down, ldd, stride, alpha, p, packed)
    if (M * rank < 4 * 256) MXFP8_PR(1);
    else MXFP8_PR(4);
#undef MXFP8_PR
    return;
  }
  const int runs = project_runs(M, K, rank);
  float* to = runs == 1 ? p : workspace;
  const int split = project_split(M, rank, adapters, runs);
#define MXFP8_PT(JC)                                                                                              \
  hipLaunchKernelGGL((project_tile_kernel<FMT, JC>),                                                              \
                     dim3((uint32_t)((M + kTileRows - 1) / kTileRows * runs), (uint32_t)((rank + 16 * JC - 1) / (16 * JC)), \
                          (uint32_t)split), dim3(256), 0, stream, (int)M, (int)K, runs, a, lda, sa, ids, (int)adapters, (int)rank, down, ldd, \
                     stride, alpha, to, packed)
  // As many ranks as there are, up to 64: past them rows are read again (8192x18944 rank 16: 30 us for 16 at a time, 37
  // for 64; 4096x8960 rank 64: 27 and 17).
  if (rank <= 16) MXFP8_PT(1);
  else if (rank <= 32) MXFP8_PT(2);
  else MXFP8_PT(4);
#undef MXFP8_PT
  if (runs > 1) {
    const int64_t units = M * rank / 4, need = (units + 255) / 256;
    hipLaunchKernelGGL(project_join_kernel, dim3((uint32_t)(need < 4096 ? need : 4096)), dim3(256), 0, stream,
                       reinterpret_cast<const nt_f32x4*>(workspace), runs, units, (int)(rank / 4), ids, (int)adapters,
                       alpha, reinterpret_cast<nt_f32x4*>(p), packed);
  }
}

// Rows of an adapter that a run has at least: with 512, 4096x1536 rank 64 takes 15 us, 3000x1536 rank 128 17 and
// 1024x1536 rank 16 13 with the join; with 128, 19, 20 and 10; with 1024, 15 (16384x1536 rank 64 64 in place of 49),
// 22 and 14.
constexpr int64_t kGradRows = 512;
// Ranks and columns of a workgroup, and the runs that the rows are split into.  16 ranks by 256 columns, or past 16
// ranks 32 by 128, which read z less often: 8192x18944 rank 16 42 us against 51, 4096x8960 rank 64 39 against 32.
struct GradShape {
  int jt, nf, jgroups, ctiles, runs;
};
GradShape grad_shape(int64_t M, int64_t C, int64_t rank, int64_t adapters) {
  GradShape s;
  s.jt = rank <= 16 ? 1 : 2;
  s.nf = s.jt == 1 ? 16 : 8;
  s.jgroups = (int)((rank + 16 * s.jt - 1) / (16 * s.jt));
  s.ctiles = (int)((C + 16 * s.nf - 1) / (16 * s.nf));
  // Two workgroups to each of 256 compute units (4096x8960 rank 64: 31 us, with one 45, with four 40), kGradRows to
  // an adapter and run at least, and at most 256 MB of partial sums.
  const int64_t wgs = (int64_t)s.ctiles * s.jgroups * adapters;
  int64_t runs = 512 / wgs;
  const int64_t most = M / (kGradRows * adapters);
  if (runs > most) runs = most;
  if (runs > 1) {  // then there are at most 256 workgroups to a run, whose sums' bytes fit in 64 bits
    const int64_t bytes = adapters * rank * C * 4;
    if (runs * bytes > (int64_t(256) << 20)) runs = (int64_t(256) << 20) / bytes;
  }
  s.runs = (int)(runs < 1 ? 1 : runs);  // M == 0: one run of no rows, which gives zeros
  return s;
}

template <int FMT>
void grad(const GradShape& s, const GradArgs& q, const uint8_t* z, const uint8_t* sz, const float* p,
          const int32_t* ids, hipStream_t stream) {
  const dim3 grid((uint32_t)s.ctiles * (uint32_t)s.jgroups * (uint32_t)q.adapters * (uint32_t)s.runs);
  const bool dword = ((uintptr_t)sz & 3) == 0 && q.C % 128 == 0;
#define MXFP8_G(JT, NF, DWORD) \
  hipLaunchKernelGGL((grad_kernel<FMT, JT, NF, DWORD>), grid, dim3(kGradThreads), 0, stream, q, z, sz, p, ids)
  if (s.jt == 1) {
    if (dword) MXFP8_G(1, 16, true);
    else MXFP8_G(1, 16, false);
  } else {
    if (dword) MXFP8_G(2, 8, true);
    else MXFP8_G(2, 8, false);
  }
#undef MXFP8_G
}

}  // namespace mx_adapters_detail

using namespace mx_adapters_detail;

void launch_mx_adapter_project(int64_t M, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                               const int32_t* ids, int64_t adapters, int64_t rank, const uint16_t* down, int64_t ldd,
                               int64_t stride, const float* alpha, float* p, uint16_t* packed, float* workspace,
                               hipStream_t stream) {
  const MxPacked to{packed, (int)((rank + 15) / 16)};
  if (a_fmt == 0) project<0>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, to, workspace, stream);
  else if (a_fmt == 1) project<1>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, to, workspace, stream);
  else project<kE2M1>(M, K, a, lda, sa, ids, adapters, rank, down, ldd, stride, alpha, p, to, workspace, stream);
}

int64_t adapter_project_workspace(int64_t M, int64_t K, int64_t rank) {
  const int64_t runs = project_runs(M, K, rank);
  return runs == 1 ? 0 : runs * M * rank * (int64_t)sizeof(float);
}

int64_t adapter_packed_bytes(int64_t M, int64_t rank) { return MxPacked::elements(M, rank) * 2; }

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
  q.per = (int)((M + s.runs - 1) / s.runs + 31) / 32 * 32;
  q.runs = s.runs, q.jgroups = s.jgroups, q.ctiles = s.ctiles, q.transposed = transposed, q.ldz = ldz;
  q.window = ldz < (int64_t(1) << 31) / kWindow ? kWindow : kSmallWindow;
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
