// mxfp4_gemm.hip -- products with an MXFP4 (E2M1, one E8M0 scale per 32 of K)
// right operand on CDNA4 matrix cores (gfx950):
//
//   C[m][n] = sum over 32-wide K blocks j of
//             2^(sa[m][j] - 127) * 2^(sb[n][j] - 127) * sum_{k in j} A[m][k] * B[n][k]
//
// A in E2M1, E4M3 or E5M2, fp32 accumulation, fp32 or bf16 out.  The scaled
// matrix instructions take the element formats and the blocks' scales as they
// are, so nothing is decoded.  With an FP8 operand they align the products of 8
// consecutive k to the largest of them and cut what lies below 2^-13 of it:
// quantized normal data, K = 3584 and 18944, comes out within 3 to 5e-6 of the
// result's rms in fp32 (an fp32 product of the same values 3 to 6e-8), a
// three-hundredth of what bf16 rounds off; products in 16 bits would avoid it at
// half the rate at most.  E2M1 pairs lose nothing.
//
// With adapters, row m of C starts from up[a] p[m], a = ids[m], in place of zero:
// a few bf16 matrix instructions per tile (p in three parts, all its bits) while
// the first operands are on their way.
#include "mx_common.hpp"
#include "mx_launch.hpp"

// One translation unit can hold everything (MXFP4_GEMM_FMT undefined), or the
// build compiles this file once per format of A in parallel (0, 1, 2), without
// and with adapters (MXFP4_GEMM_ADAPT 0, 1), and once with -1 for the host
// dispatch alone.
#ifndef MXFP4_GEMM_FMT
#define MXFP4_GEMM_FMT 3
#endif

#include <type_traits>

namespace mxfp8 {

namespace mxfp4_detail {

struct NoAdapters {};
// Row m gets up[ids[m]] p[m]; ids outside 0 .. adapters - 1 nothing.
struct Adapters {
  const int32_t* ids;
  const float* p;       // [M][rank]
  const uint16_t* packed;  // p as MxPacked
  const uint16_t* up;   // [adapters] at `stride`, each [N][ldu] bf16
  int64_t ldu, stride;
  int adapters, rank;
};

template <int AFMT, typename AD>
void gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
          int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, AD ad, hipStream_t stream);

// LDS of the few-row kernel, in bytes: A's scales, B's scales, A, each in
// whole kilobytes (a copy fills whole ones); the partial sums of the waves
// take their place at the end.
template <typename I>
__host__ __device__ constexpr I kilo(I n) {
  return (n + 1023) & ~I(1023);
}
template <int AFMT, int MT, int NT, int WAVES, bool ALDS>
constexpr int64_t few_rows_lds(int64_t rows, int64_t K) {
  const int64_t a = AFMT == kE2M1 ? K / 2 : K;
  const int64_t in = kilo(16 * MT * (K / 32)) + kilo(16 * NT * (K / 32)) + (ALDS ? kilo(rows * a) : 0);
  const int64_t out = WAVES > 1 ? WAVES * MT * NT * 1024 : 0;
  return in > out ? in : out;
}
constexpr int64_t kFewRowsLds = 150 * 1024;

#if MXFP4_GEMM_FMT >= 0

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Element format as the matrix instructions number them.
template <int FMT> constexpr int kMfmaFmt = FMT == kE2M1 ? 4 : FMT;

// Lets the last matrix instruction retire before its accumulators are read:
// the compiler's own wait is too short for the last result registers of the
// scaled forms (seen with the 32x32x64 form in gemm.hip).
__device__ __forceinline__ void mfma_retire_pad() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
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

// Operands are read through buffer descriptors whose range check returns
// zeros for lanes whose offset is set to kOutside: rows past M or N, K past
// its end, scales past a row's end.  Zero codes under a zero scale byte
// (2^-127) add nothing, so no edge needs a branch.
[[maybe_unused]] constexpr uint32_t kRange = 0xF0000000u;    // bytes behind a descriptor; valid offsets stay below 2^31
[[maybe_unused]] constexpr uint32_t kOutside = 0xF8000000u;

#if defined(__HIP_DEVICE_COMPILE__)
typedef __attribute__((address_space(3))) void lds_void;
template <int BYTES>
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, uint8_t* to, uint32_t lane_off, uint32_t off) {
  if constexpr (BYTES == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)to, 16, lane_off, off, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)to, 4, lane_off, off, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)kRange, 0x00020000);
}
#endif

// Wait for this wave's loads and LDS reads, then meet the others: a bare
// s_barrier, since __syncthreads() would add a release fence.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet() {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(N >= 0 && N <= 63, "vmcnt");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// ---------------------------------------------------------------------------
// Few rows of A.  A workgroup owns 16 MT rows of A x 16 NT rows of B; its
// waves split K in contiguous runs of 128-wide chunks and add up their
// accumulators through LDS at the end, in a fixed order.  B goes from memory
// to registers without LDS (each of its bytes is used by one wave only), U
// chunks at a time, the next U on their way while these multiply; the scales
// of the workgroup's rows, and A itself where it fits (ALDS), are copied to
// LDS first.  v_mfma_scale_f32_16x16x128: lane l holds row l & 15 of both
// operands and, with g = l >> 4, the 32 E2M1 elements 32 g .. +31 of the
// chunk (16 bytes), or of FP8 the bytes 16 g .. +15 and 64 + 16 g .. +15; the
// scale of the chunk's 32-wide block g is taken from the lanes of group g.
// Operands are swapped (B first), so a lane's four results are four
// consecutive columns of C.
//
// What bounds it: the load path of a CU takes about 40 cycles for an
// instruction that gathers 16 rows x 64 bytes, whatever it brings, so the
// count of those is what matters: one per 16 rows and chunk of B, and of A
// unless it is in LDS; then latency, and about 1 us per 1000 waves started.
// 1x18944x3584 (E4M3) 8.0 us, 4.5 TB/s of B; 37x1536x8960 (E2M1 pairs) 7.6 us.
// ---------------------------------------------------------------------------
#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane_off, off, 0));
}
// n bytes (a multiple of 4) from p to LDS, by the waves of a workgroup in turn.
template <int WAVES>
__device__ __forceinline__ void copy_to_lds(const uint8_t* p, int n, uint8_t* to, int wave, int lane) {
  const __amdgpu_buffer_rsrc_t rsrc = descriptor(p);
  if (((uintptr_t)p & 15) == 0 && (n & 15) == 0) {
    for (int at = wave * 1024; at < n; at += WAVES * 1024)
      load_lds<16>(rsrc, to + at, at + lane * 16 < n ? lane * 16 : kOutside, at);
  } else {
    for (int at = wave * 256; at < n; at += WAVES * 256)
      load_lds<4>(rsrc, to + at, at + lane * 4 < n ? lane * 4 : kOutside, at);
  }
}
#endif

#if defined(__HIP_DEVICE_COMPILE__)
// The next adapter that any lane's rows name, or -1; its rows are crossed off
// with `id[i] = -1` where id[i] is it.
template <int MT>
__device__ __forceinline__ int next_adapter(const int (&id)[MT]) {
  int a = -1;
#pragma unroll
  for (int i = MT - 1; i >= 0; --i) {
    const uint64_t some = __ballot(id[i] >= 0);
    if (some) a = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(some));
  }
  return a;
}
// up p of the few-row kernel's rows: pieces of 32 ranks of each adapter that
// they name, dealt to the waves in turn.  A wave adds DEPTH of them between
// batches of the product, with the next ones on their way, so that their loads
// cost no waiting of their own while the product lasts.  (All of them in front of
// it, or a row at a time with its loads in a longer run of code, took 2 to 7 us
// more than the product alone; so does code that every workgroup fetches anew.)
// A lane's four results belong to one row, so rows of other adapters keep what
// they had, whatever this one's values are.  61x3584x18944: the product alone 30
// us, with one adapter of rank 64 33, with 32 of them 36; 1x18944x3584 7.2 and,
// rank 16, 9.4 (ids, up and p follow each other before a short product).
template <int MT, int NT, int WAVES>
struct RowAdapters {
  static constexpr int DEPTH = 2, LOADS = DEPTH * (NT + 2 * MT);
  struct Piece {
    int a;
    v4i u[NT];
    MxRaw<float> p[MT];
  };
  int id[MT], names, per, pieces, n;
  Piece v[DEPTH];
  v4f sum[MT][NT];

  __device__ __forceinline__ void load(const Adapters& ad, int m0, int n0, int rows_b, int lane, int at, Piece& v) const {
    const int r = lane & 15, g = lane >> 4;
    const bool in = at < pieces;
    const int which = in ? at / per : 0, k = (at - which * per) * 32 + 8 * g;
    v.a = in ? __builtin_amdgcn_readlane(names, which) : -2;
    const __amdgpu_buffer_rsrc_t rp = descriptor(reinterpret_cast<const uint8_t*>(ad.p + (int64_t)m0 * ad.rank));
    const __amdgpu_buffer_rsrc_t ru = descriptor(
        reinterpret_cast<const uint8_t*>(ad.up + (in ? v.a * ad.stride + (int64_t)n0 * ad.ldu : 0)));
#pragma unroll
    for (int j = 0; j < NT; ++j)
      v.u[j] = load16(ru, in && 16 * j + r < rows_b && k < ad.rank ? (uint32_t)((16 * j + r) * ad.ldu + k) * 2 : kOutside, 0);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      mx_get(rp, id[i] == v.a && k < ad.rank ? (uint32_t)((16 * i + r) * ad.rank + k) * 4 : kOutside, 0, v.p[i]);
  }
  // The ids, before anything else is asked for.
  __device__ __forceinline__ void ask(const Adapters& ad, int m0, int rows_a, int lane) {
#pragma unroll
    for (int i = 0; i < MT; ++i) id[i] = 16 * i + (lane & 15) < rows_a ? ad.ids[m0 + 16 * i + (lane & 15)] : -1;
  }
  // Lane n of `names` holds the n-th adapter; the first pieces' loads.
  __device__ __forceinline__ void start(const Adapters& ad, int m0, int n0, int rows_b, int wave, int lane) {
    int left[MT], count = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (id[i] >= ad.adapters) id[i] = -1;
      left[i] = id[i];
#pragma unroll
      for (int j = 0; j < NT; ++j) sum[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    names = -1;
    for (int a = next_adapter(left); a >= 0; a = next_adapter(left)) {
      if (lane == count) names = a;
      ++count;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (left[i] == a) left[i] = -1;
    }
    per = (ad.rank + 31) >> 5;
    pieces = count * per;
    n = wave;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(ad, m0, n0, rows_b, lane, n + d * WAVES, v[d]);
  }
  __device__ __forceinline__ void step(const Adapters& ad, int m0, int n0, int rows_b, int lane) {
    if (n >= pieces) return;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float f[8];
        mx_unpack(v[d].p[i], f);
        const MxParts p = mx_parts(f);
        const bool mine = id[i] == v[d].a;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          v4f s = sum[i][j];
#pragma unroll
          for (int part = 2; part >= 0; --part)
            s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, v[d].u[j]), p.part[part], s, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[i][j][e] = mine ? s[e] : sum[i][j][e];
        }
      }
      load(ad, m0, n0, rows_b, lane, n + (d + DEPTH) * WAVES, v[d]);
    }
    n += DEPTH * WAVES;
  }
};
#endif

template <int AFMT, int MT, int NT, int WAVES, int U, bool ALDS, typename OutT, typename AD>
__global__ __launch_bounds__(WAVES * 64) void few_rows_kernel(int M, int N, int K, const uint8_t* __restrict__ A,
                                                              int64_t lda, const uint8_t* __restrict__ SA,
                                                              const uint8_t* __restrict__ B, int64_t ldb,
                                                              const uint8_t* __restrict__ SB, OutT* __restrict__ C,
                                                              int64_t ldc, AD ad) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int PARTS = AFMT == kE2M1 ? 1 : 2;  // 16-byte parts of A per lane and chunk
  constexpr int AB = 64 * PARTS;                // bytes of a chunk of a row of A
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int tiles_n = (N + 16 * NT - 1) / (16 * NT);
  const int n0 = (int)(blockIdx.x % tiles_n) * (16 * NT), m0 = (int)(blockIdx.x / tiles_n) * (16 * MT);
  const int rows_a = min(16 * MT, M - m0), rows_b = min(16 * NT, N - n0);
  const int chunks = K >> 7, sk = K >> 5;
  const int c0 = (int)((int64_t)chunks * wave / WAVES), c1 = (int)((int64_t)chunks * (wave + 1) / WAVES);
  constexpr bool ADAPT = std::is_same_v<AD, Adapters>;
  uint8_t *lsa = lds, *lsb = lsa + kilo(16 * MT * sk), *la = lsb + kilo(16 * NT * sk);

  [[maybe_unused]] std::conditional_t<ADAPT, RowAdapters<MT, NT, WAVES>, NoAdapters> rows;
  if constexpr (ADAPT) {
    rows.ask(ad, m0, rows_a, lane);
    __builtin_amdgcn_sched_barrier(0);
  }
  copy_to_lds<WAVES>(SA + (int64_t)m0 * sk, rows_a * sk, lsa, wave, lane);
  copy_to_lds<WAVES>(SB + (int64_t)n0 * sk, rows_b * sk, lsb, wave, lane);
  const __amdgpu_buffer_rsrc_t ra = descriptor(A + (int64_t)m0 * lda), rb = descriptor(B + (int64_t)n0 * ldb);
  const int apr = chunks * AB;  // bytes of a row of A
  if constexpr (ALDS) {
    const int n = rows_a * apr;
    for (int at = wave * 1024; at < n; at += WAVES * 1024) {
      const int i = at + lane * 16, row = i / apr;
      load_lds<16>(ra, la + at, i < n ? (uint32_t)(row * lda + (i - row * apr)) : kOutside, 0);
    }
  }
  // Rows past M or N repeat the last one's: what they give is dropped.
  uint32_t ao[MT], bo[NT];
  int sao[MT], sbo[NT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int row = min(16 * t + r, rows_a - 1);
    ao[t] = (uint32_t)(ALDS ? row * apr : row * lda) + 16 * g;
    sao[t] = row * sk + g;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = min(16 * t + r, rows_b - 1);
    bo[t] = (uint32_t)(row * ldb) + 16 * g;
    sbo[t] = row * sk + g;
  }
  constexpr int AREGS = ALDS ? 1 : U;  // chunks of A held in registers
  struct Batch {
    v4i b[U][NT], a[AREGS][MT][PARTS];
  };
  auto load = [&](int c, Batch& x) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = c + u < c1;  // past the wave's run: no traffic
#pragma unroll
      for (int t = 0; t < NT; ++t) x.b[u][t] = load16(rb, in ? bo[t] : kOutside, (c + u) * 64);
      if constexpr (!ALDS) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
            x.a[u][t][part] = load16(ra, in ? ao[t] : kOutside, (c + u) * AB + part * 64);
      }
    }
  };
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int c, Batch& x) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= c1) break;
      int as[MT], bs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) bs[t] = lsb[sbo[t] + (c + u) * 4];
#pragma unroll
      for (int t = 0; t < MT; ++t) as[t] = lsa[sao[t] + (c + u) * 4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        v4i lo, hi = v4i{0, 0, 0, 0};
        if constexpr (ALDS) {
          lo = *reinterpret_cast<const v4i*>(la + ao[i] + (c + u) * AB);
          if constexpr (PARTS == 2) hi = *reinterpret_cast<const v4i*>(la + ao[i] + (c + u) * AB + 64);
        } else {
          lo = x.a[u][i][0];
          if constexpr (PARTS == 2) hi = x.a[u][i][PARTS - 1];
        }
        const v8i af = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const v8i bf = v8i{x.b[u][j][0], x.b[u][j][1], x.b[u][j][2], x.b[u][j][3], 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf, af, acc[i][j], kMfmaFmt<kE2M1>,
                                                                      kMfmaFmt<AFMT>, 0, bs[j], 0, as[i]);
        }
      }
    }
  };
  // The first two batches travel with the copies; everything has landed, in
  // every wave, before the first product.  (The empty asm uses their
  // registers: the loads cannot be moved past the wait.)
  Batch x, y;
  load(c0, x);
  load(c0 + U, y);
  if constexpr (ADAPT) rows.start(ad, m0, n0, rows_b, wave, lane);
  auto pin = [](Batch& v) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(v.b[u][t]));
    if constexpr (!ALDS) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) asm volatile("" : "+v"(v.a[u][t][part]));
    }
  };
  pin(x);
  pin(y);
  if constexpr (ADAPT) wait_loads_and_meet<RowAdapters<MT, NT, WAVES>::LOADS>();  // all but the pieces', the last
  else wait_loads_and_meet<0>();
  for (int c = c0; c < c1; c += 2 * U) {
    multiply(c, x);
    __builtin_amdgcn_sched_barrier(0);  // each load is issued a batch ahead of its use
    load(c + 2 * U, x);
    __builtin_amdgcn_sched_barrier(0);
    multiply(c + U, y);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ADAPT) rows.step(ad, m0, n0, rows_b, lane);
    load(c + 3 * U, y);
    __builtin_amdgcn_sched_barrier(0);
  }
  mfma_retire_pad();
  if constexpr (ADAPT) {
#pragma nounroll
    while (rows.n < rows.pieces) rows.step(ad, m0, n0, rows_b, lane);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] += rows.sum[i][j];
  }
  auto store = [&](int i, int j, v4f v) __attribute__((always_inline)) {
    const int m = m0 + 16 * i + r, n = n0 + 16 * j + 4 * g;
    if (m < M) store4(C + (int64_t)m * ldc + n, v, N - n);
  };
  if constexpr (WAVES == 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) store(i, j, acc[i][j]);
  } else {
    __syncthreads();  // the scales and A have been read
    v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) red[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int f = wave; f < MT * NT; f += WAVES) {  // a fragment per wave
      v4f sum = red[f * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += red[(w * MT * NT + f) * 64 + lane];
      store(f / NT, f % NT, sum);
    }
  }
#endif
}

template <int AFMT, int MT, int NT, int WAVES, int U, bool ALDS, typename AD>
void few_rows(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
              int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, AD ad, hipStream_t stream) {
  const dim3 grid((uint32_t)(((N + 16 * NT - 1) / (16 * NT)) * ((M + 16 * MT - 1) / (16 * MT))));
  const uint32_t lds = (uint32_t)few_rows_lds<AFMT, MT, NT, WAVES, ALDS>(M < 16 * MT ? M : 16 * MT, K);
  if (c_dtype == 0)
    hipLaunchKernelGGL((few_rows_kernel<AFMT, MT, NT, WAVES, U, ALDS, float, AD>), grid, dim3(WAVES * 64), lds, stream,
                       (int)M, (int)N, (int)K, a, lda, sa, b, ldb, sb, static_cast<float*>(c), ldc, ad);
  else
    hipLaunchKernelGGL((few_rows_kernel<AFMT, MT, NT, WAVES, U, ALDS, uint16_t, AD>), grid, dim3(WAVES * 64), lds, stream,
                       (int)M, (int)N, (int)K, a, lda, sa, b, ldb, sb, static_cast<uint16_t*>(c), ldc, ad);
}

// ---------------------------------------------------------------------------
// Tiles.  A workgroup of 4 waves (2 x 2) computes BM x BN of C with
// v_mfma_scale_f32_32x32x64.  One K block is what 128 bytes of a row of A
// hold: 256 elements in E2M1, 128 in FP8 (B then takes 64 bytes).  Two K
// blocks sit in LDS; each is multiplied in two stages, and while a stage
// multiplies, the fragments of the next one are read into a second register
// set.  At a K block's second stage all waves meet once; its buffer is then
// refilled with the K block after next while the stage still multiplies.
//
// Memory goes straight to LDS (buffer_load ... lds, 16 bytes a lane).  The
// buffer descriptor's range check returns zeros for lanes whose offset is set
// to kOutside: rows past M or N, the half of the last 256-wide K block that
// K = 128 mod 256 lacks, and scales past a row's end.
//
// What bounds it: the matrix cores, at the clock the board's power leaves them
// (8192x18944x3584 in E2M1 pairs 272-300 us, 3.7-4.1 PFLOP/s, the cores busy
// 52 % at 1.9 GHz; 8192x3584x18944 in E5M2 x E2M1 375-425 us, 72-76 %).  A
// 256 x 256 tile reads 64 bytes of LDS a cycle and CU (of 128) and 32 from L2,
// the same for E2M1 pairs, whose instructions take half as long for half the
// bytes, and less for FP8 x E2M1.
// ---------------------------------------------------------------------------
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileThreads = 256;
template <int BM, int BN, int AFMT>
struct Tile {
  static constexpr bool A4 = AFMT == kE2M1;
  static constexpr int KB = A4 ? 256 : 128;       // elements per K block
  static constexpr int AB = 128, BB = A4 ? 128 : 64;  // bytes of a row per K block
  static constexpr int A_ST = BM * AB, B_ST = BN * BB;
  static constexpr int STG = 4 * 32 * (BN / 2 * 4);  // epilogue staging: one fp32 strip of 32 rows per wave
  static constexpr int PB = A_ST + B_ST > STG ? A_ST + B_ST : STG;
  static constexpr int SB = KB / 32;               // scale bytes of a row per K block
  static constexpr int SROW = 4 * SB;              // and per group of four K blocks
  static constexpr int SG = (BM + BN) * SROW;      // one group of scales, A's rows then B's
  static constexpr int SGRP = 2 * SG;
};

// Keeps an address offset out of the optimiser's sight, so that LDS accesses
// stay "named array + offset" and their waits are per array.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(x));
#endif
  return x;
}

#if defined(__HIP_DEVICE_COMPILE__)
// up p as a tile's first accumulators (v_mfma_f32_32x32x16_bf16, whose results
// lie as the scaled instruction's do): 16 ranks at a time of each adapter that
// the wave's rows name, zeros for p in the rows of others.  m0, n0: the wave's
// first row and column.  What does not depend on the rows' ids is asked for
// before the tile's own first loads (`ask`).
//
// Zeros times an infinity or a NaN would not be zero.  So such values of up are
// taken out, and `spoilt` keeps, for each of a lane's rows, the columns that
// they leave without a result; add() says whether there are any.  (Choosing row
// by row what to add would take the accumulators through the vector registers.)
//
// All three parts of p, also where C is bf16: ranks that cancel can leave less of
// each than C's rounding, and a row's bits of p must not go by its batch.  (With
// the leading two, 16 bits: 8192x18944x3584 rank 64 469 us in place of 483, 4096
// rows x 3584 x 3584 of 32 adapters, mixed, rank 64 154 in place of 176.)
//
// It costs the ids' and up's latency and the instructions of a tile, 2 us for
// each, of which 1 without any adapter: 8192x18944x3584 408 us alone, 432 with
// rank 16 and 483 with rank 64; 4096x8960x1536 50, 57 and 70; 4096x1536x8960 55,
// 60 and 60; 512x3584x3584 rank 16 13.6 in place of 12.5.  Each further adapter of
// a wave's rows takes 0.4 us (512 rows, 32 adapters mixed: 29 us; rank 64: 73),
// bound by its matrix instructions and the rows of up, of which 16 ranks are 32
// bytes.
template <int MT, int NT>
struct FirstAdapters {
  static constexpr int PARTS = 3, LISTS = (MT + 1) / 2;
  struct P {
    v4i p[MT][PARTS];
  };
  int id[MT];
  P first;
  __amdgpu_buffer_rsrc_t rp;
  uint32_t po;  // a lane's place in 1 KB
  int steps;

  // Past the last row's strip: nothing is read, no row is anybody's.
  __device__ __forceinline__ void get_p(int m0, int M, int step, P& v) const {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
        v.p[i][part] = load16(rp, m0 + 32 * i < M && step < steps ? po : kOutside, ((i * steps + step) * 3 + part) * 1024);
  }
  __device__ __forceinline__ void ask(const Adapters& ad, int M, int m0, int lane) {
    steps = (ad.rank + 15) >> 4;
    po = lane * 16;
    // m0 is a multiple of 32
    rp = descriptor(reinterpret_cast<const uint8_t*>(ad.packed) + (int64_t)(m0 >> 5) * steps * (3 * 1024));
#pragma unroll
    for (int i = 0; i < MT; ++i) id[i] = m0 + 32 * i + (lane & 31) < M ? ad.ids[m0 + 32 * i + (lane & 31)] : -1;
    get_p(m0, M, 0, first);
  }
  __device__ __forceinline__ bool add(const Adapters& ad, int M, int N, int m0, int n0, int lane, v16f (&acc)[MT][NT],
                                      uint32_t (&spoilt)[MT][NT]) {
    const int r = lane & 31, g = lane >> 5;
    bool any = false;
    // Lane n & 63 of names[n >> 6] holds the n-th adapter.
    int left[MT], names[LISTS], count = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (id[i] >= ad.adapters) id[i] = -1;
      left[i] = id[i];
#pragma unroll
      for (int j = 0; j < NT; ++j) spoilt[i][j] = 0;
    }
#pragma unroll
    for (int k = 0; k < LISTS; ++k) names[k] = -1;
    for (int a = next_adapter(left); a >= 0; a = next_adapter(left)) {
#pragma unroll
      for (int k = 0; k < LISTS; ++k)
        if (lane + 64 * k == count) names[k] = a;
      ++count;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (left[i] == a) left[i] = -1;
    }
    auto name = [&](int n) __attribute__((always_inline)) {
      int a = __builtin_amdgcn_readlane(names[0], n & 63);
      if constexpr (LISTS == 2) a = n < 64 ? a : __builtin_amdgcn_readlane(names[1], n & 63);
      return a;
    };
    // Adapter by adapter 16 ranks at a time, `DEPTH` of them on their way.
    int n = 0, step = 0, next_n = 0, next_step = 0;
    auto ask_u = [&](v4i (&u)[NT]) __attribute__((always_inline)) {
      const bool some = next_n < count;
      const int k = next_step * 16 + 8 * g;
      const __amdgpu_buffer_rsrc_t ru =
          descriptor(reinterpret_cast<const uint8_t*>(ad.up + (some ? name(next_n) * ad.stride : 0) + (int64_t)n0 * ad.ldu));
#pragma unroll
      for (int j = 0; j < NT; ++j)
        u[j] = load16(ru, n0 + 32 * j + r < N && k < ad.rank && some ? (uint32_t)((32 * j + r) * ad.ldu + k) * 2 : kOutside, 0);
    };
    auto one = [&](v4i (&u)[NT], const P& now) __attribute__((always_inline)) {
      const int a = name(n);
      const bool in = step * 16 + 8 * g < ad.rank;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        // an exponent of all ones carries into the bit above it
        uint32_t over = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) over |= ((uint32_t)u[j][w] & 0x7F807F80u) + 0x00800080u;
        const uint64_t where = __ballot((over & 0x80008000u) != 0);
        if (where) {
          any = true;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = (uint32_t)u[j][w];
            u[j][w] = (int)(((x & 0x7F80u) == 0x7F80u ? 0 : x & 0xFFFFu) |
                              ((x & 0x7F800000u) == 0x7F800000u ? 0 : x & 0xFFFF0000u));
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if (id[i] == a) spoilt[i][j] |= (uint32_t)where | (uint32_t)(where >> 32);
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const bool mine = id[i] == a;
        if (!__ballot(mine)) continue;
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) {
          v4i p;
#pragma unroll
          for (int w = 0; w < 4; ++w) p[w] = mine && in ? now.p[i][part][w] : 0;
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(mx_bf8, u[j]),
                                                                __builtin_bit_cast(mx_bf8, p), acc[i][j], 0, 0, 0);
        }
      }
    };
    auto run = [&](auto depth, auto single) __attribute__((always_inline)) {
      constexpr int DEPTH = depth.value;
      constexpr bool ONE = single.value;  // up to 16 ranks: p is there already
      v4i u[DEPTH][NT];
      P p[ONE ? 1 : DEPTH];
      auto ask_next = [&](int d) __attribute__((always_inline)) {
        ask_u(u[d]);
        if constexpr (!ONE) get_p(m0, M, next_step, p[d]);
        asm volatile("" ::: "memory");  // the loads stay here
        if (ONE || ++next_step == steps) {
          next_step = 0;
          ++next_n;
        }
      };
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) ask_next(d);
#pragma nounroll
      while (n < count) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          if (n >= count) break;
          one(u[d], ONE ? first : p[d]);
          ask_next(d);
          if (ONE || ++step == steps) {
            step = 0;
            ++n;
          }
        }
      }
    };
    if (steps == 1) run(std::integral_constant<int, NT >= 4 ? 3 : 6>{}, std::true_type{});
    else run(std::integral_constant<int, 2>{}, std::false_type{});
    return any;
  }
};
#endif

// SW: scale rows that start on 16-byte boundaries are loaded 16 bytes a lane,
// others 4.
template <int BM, int BN, int AFMT, bool SW, int RING, typename OutT, typename AD>
__device__ __forceinline__ void gemm_tile(int M, int N, int K, const uint8_t* __restrict__ A, int64_t lda,
                                          const uint8_t* __restrict__ SA, const uint8_t* __restrict__ B, int64_t ldb,
                                          const uint8_t* __restrict__ SB, OutT* __restrict__ C, int64_t ldc,
                                          int tiles_m, int tiles_n, int tile_first, int sm, int sn, int wg, int nwg,
                                          uint8_t* kbuf0, uint8_t* kbuf1, uint8_t* kbuf2, uint8_t* kbuf3,
                                          uint8_t* sgrp, const AD& ad) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef Tile<BM, BN, AFMT> T;
  constexpr bool A4 = T::A4;
  constexpr int WM = BM / 2, WN = BN / 2, MT = WM / 32, NT = WN / 32;
  constexpr int A_LOADS = T::A_ST / (kTileThreads * 16), B_LOADS = T::B_ST / (kTileThreads * 16);
  constexpr int STEPS = A4 ? 2 : 1;  // 64-wide matrix steps per stage
  constexpr bool ADAPT = std::is_same_v<AD, Adapters>;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // The tile: cells of (BM << sm) x (BN << sn), in groups of 4 cell rows
  // walked column by column, 2^(sm + sn) workgroups to a cell; each XCD
  // (workgroups go round them) takes a contiguous band.
  if ((nwg & 7) == 0) wg = (wg & 7) * (nwg >> 3) + (wg >> 3);
  const int cell = tile_first + (wg >> (sm + sn)), sub = wg & ((1 << (sm + sn)) - 1);
  constexpr int GROUP = 4;
  const int group = cell / (GROUP * tiles_n), first = group * GROUP;
  const int gsz = min(tiles_m - first, GROUP), within = cell - group * GROUP * tiles_n;
  const int m0 = (((first + within % gsz) << sm) + (sub >> sn)) * BM;
  const int n0 = (((within / gsz) << sn) + (sub & ((1 << sn) - 1))) * BN;
  if (m0 >= M || n0 >= N) return;

  // K blocks that hold something, up to `last`; at least two are multiplied,
  // those past it as zeros.
  const int last = (K + T::KB - 1) / T::KB - 1, nkb = max(last + 1, 2), sk = K >> 5;
  const __amdgpu_buffer_rsrc_t ra = descriptor(A + (int64_t)m0 * lda), rb = descriptor(B + (int64_t)n0 * ldb);
  const uint8_t *pa = SA + (int64_t)m0 * sk, *pb = SB + (int64_t)n0 * sk;
  const __amdgpu_buffer_rsrc_t rsa = descriptor(pa), rsb = descriptor(pb), rsw = descriptor(wave < 2 ? pa : pb);

  // Lane offsets of the data loads: each instruction fills 1 KB of LDS in lane
  // order, 8 rows of 128 bytes (or 16 of 64).  The 16-byte unit c of row r
  // sits at unit c ^ swizzle(r), so that 16 consecutive rows read at one unit
  // hit 16 different 16-byte bank groups.
  auto swz = [](int r, int bytes) { return bytes == 128 ? (r >> 1) & 7 : (r >> 2) & 3; };
  uint32_t a_off[A_LOADS], b_off[B_LOADS];
  uint32_t a_unit, b_unit;  // first byte of the lane's unit (the swizzle repeats every load)
#pragma unroll
  for (int j = 0; j < A_LOADS; ++j) {
    const int row = (j * 4 + wave) * 8 + (lane >> 3);
    a_unit = ((lane & 7) ^ swz(row, 128)) * 16;
    a_off[j] = m0 + row < M ? (uint32_t)(row * lda) + a_unit : kOutside;
  }
#pragma unroll
  for (int j = 0; j < B_LOADS; ++j) {
    constexpr int UPR = T::BB / 16;
    const int row = (j * 4 + wave) * (64 / UPR) + lane / UPR;
    b_unit = ((lane % UPR) ^ swz(row, T::BB)) * 16;
    b_off[j] = n0 + row < N ? (uint32_t)(row * ldb) + b_unit : kOutside;
  }
  // The last K block of E2M1 pairs may be half full: its upper half reads as zeros.
  const bool half_last = A4 && (K & 255) != 0;

  auto buf_ptr = [&](int p) __attribute__((always_inline)) -> uint8_t* {
    return p == 0 ? kbuf0 : p == 1 ? kbuf1 : p == 2 ? kbuf2 : kbuf3;
  };
  constexpr int DMA_ITEMS = A_LOADS + B_LOADS;
  auto dma_item = [&](int p, int kb, int item) __attribute__((always_inline)) {
    uint8_t* buf = buf_ptr(p);
    const bool none = kb > last, cut = half_last && kb == last;
    if (item < A_LOADS) {
      const uint32_t off = none || (cut && a_unit >= 64) ? kOutside : a_off[item];
      load_lds<16>(ra, buf + (item * 4 + wave) * 1024, off, kb * T::AB);
    } else {
      const int j = item - A_LOADS;
      const uint32_t off = none || (cut && b_unit >= 64) ? kOutside : b_off[j];
      load_lds<16>(rb, buf + T::A_ST + (j * 4 + wave) * 1024, off, kb * T::BB);
    }
  };

  // Scales of four K blocks (group grp): SROW bytes of each row of A, then of
  // B, in pieces of 16 bytes, all rows' first pieces, then their second ones:
  // the 32 rows of a fragment then read at a stride of 16 bytes (two to a
  // bank; at the 32 bytes of whole rows of E2M1 pairs it was four).  Scales
  // past a row's end read as zeros, which no result uses.
  constexpr int ROWS = BM + BN, PIECES = T::SROW / 16;
  auto scale_loads = [&](int grp) __attribute__((always_inline)) {
    uint8_t* area = sgrp + (grp & 1) * T::SG;
    constexpr int BYTES = SW ? 16 : 4;
    constexpr int RPI = 4 * BYTES;         // rows per instruction: a lane each, or four lanes each
    constexpr int AI = BM / RPI, BI = BN / RPI;
    static_assert((AI % 4 == 0 && BI % 4 == 0) || (SW && AI == 2 && BI == 2), "scale rows over four waves");
#pragma unroll
    for (int piece = 0; piece < PIECES; ++piece) {
      const int from = grp * T::SROW + piece * 16 + (SW ? 0 : (lane & 3) * 4);
      uint8_t* to = area + piece * ROWS * 16;
      if constexpr (AI % 4 == 0) {
#pragma unroll
        for (int j = 0; j < (AI + BI) / 4; ++j) {
          const bool is_a = j < AI / 4;
          const int row = ((is_a ? j : j - AI / 4) * 4 + wave) * RPI + lane * RPI / 64;
          const uint32_t off = from < sk && row < (is_a ? M - m0 : N - n0) ? row * sk + from : kOutside;
          if (is_a) load_lds<BYTES>(rsa, to + (j * 4 + wave) * RPI * 16, off, 0);
          else load_lds<BYTES>(rsb, to + (j * 4 + wave) * RPI * 16, off, 0);
        }
      } else {  // waves 0 and 1 take A's rows, 2 and 3 B's
        const int row = (wave & 1) * RPI + lane;
        load_lds<BYTES>(rsw, to + wave * RPI * 16, from < sk && row < (wave < 2 ? M - m0 : N - n0) ? row * sk + from : kOutside, 0);
      }
    }
  };

  // Scale operands of a K block.  E2M1 pairs: matrix step j (0..3) takes, in
  // lane half g, unit 4 g + j of the row, so a lane's four scales are one
  // dword and the instruction picks byte j.  FP8 x E2M1: stage h multiplies
  // the 32-wide chunks h (whose scale lane half 0 supplies) and 2 + h (half
  // 1): a lane's two scales are bytes 2 g and 2 g + 1, stage h picks byte h.
  const uint32_t sa_rd = opaque((wm * WM + (lane & 31)) * 16 + g * (A4 ? 4 : 2));
  const uint32_t sb_rd = opaque((BM + wn * WN + (lane & 31)) * 16 + g * (A4 ? 4 : 2));
  auto read_scale = [&](const uint8_t* p) __attribute__((always_inline)) -> int {
    return A4 ? *reinterpret_cast<const int*>(p) : (int)*reinterpret_cast<const uint16_t*>(p);
  };
  auto read_scales = [&](int kb, int (&sa)[MT], int (&sb)[NT]) __attribute__((always_inline)) {
    const int at = (kb & 3) * T::SB;
    const uint8_t* area = sgrp + ((kb >> 2) & 1) * T::SG + (at >> 4) * ROWS * 16 + (at & 15);
#pragma unroll
    for (int t = 0; t < MT; ++t) sa[t] = read_scale(area + sa_rd + t * 512);
#pragma unroll
    for (int t = 0; t < NT; ++t) sb[t] = read_scale(area + sb_rd + t * 512);
  };

  v16f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;

  // Fragments of stage h: two 16-byte parts of a row for FP8 (the chunks h
  // and 2 + h: lane half g has bytes 16 g .. +15 of both) and for E2M1 pairs
  // (the stage's two matrix steps); one part for E2M1 against FP8 (lane half g
  // has chunk h + 2 g whole).
  constexpr int BPARTS = A4 ? 2 : 1;
  constexpr int DS_ITEMS = 2 * MT + BPARTS * NT;
  uint32_t a_rd[2][2], b_rd[2][BPARTS];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = wm * WM + (lane & 31), c = wn * WN + (lane & 31);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int unit = A4 ? 4 * g + 2 * h + part : 4 * part + 2 * h + g;
      a_rd[h][part] = opaque(r * T::AB + ((unit ^ swz(r, 128)) << 4));
    }
#pragma unroll
    for (int part = 0; part < BPARTS; ++part) {
      const int unit = A4 ? 4 * g + 2 * h + part : h + 2 * g;
      b_rd[h][part] = opaque(T::A_ST + c * T::BB + ((unit ^ swz(c, T::BB)) << 4));
    }
  }
  struct Frags {
    v4i a[MT][2], b[NT][BPARTS];
  };
  auto ds_item = [&](int p, int h, int item, Frags& f) __attribute__((always_inline)) {
    const uint8_t* buf = buf_ptr(p);
    if (item < 2 * MT) {
      f.a[item >> 1][item & 1] =
          *reinterpret_cast<const v4i*>(buf + a_rd[h][item & 1] + (item >> 1) * 32 * T::AB);
    } else {
      const int t = (item - 2 * MT) / BPARTS, part = (item - 2 * MT) % BPARTS;
      f.b[t][part] = *reinterpret_cast<const v4i*>(buf + b_rd[h][part] + t * 32 * T::BB);
    }
  };
  auto wide = [](v4i lo, v4i hi) __attribute__((always_inline)) -> v8i {
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };

  // One stage: matrix instruction i, then the LDS reads of the next stage and
  // the loads whose turn comes after it.  rd: read stage next_h of
  // buffer next_p into nf; sc: K block kb + 1's scales too.  dma: load K block
  // kb + RING into buffer p.  sg: load the next scale group.
  constexpr int MFMAS = MT * NT * STEPS;
  // Fragment reads over the first half of the stage, loads over all of it
  // (8192x3584x18944, E2M1 pairs / E5M2 x E2M1: half 243 / 373 us, three
  // quarters 246 / 376, all 241 / 375, a quarter 260 / 445; loads over the
  // first or last half only: 251 / 379 and 253 / 393).
  constexpr int DS_SPAN = MFMAS / 2;
  auto stage = [&](int p, int h, int kb, bool rd, int next_p, int next_h, bool sc, bool dma, bool sg, const Frags& f,
                   Frags& nf, const int (&sa)[MT], const int (&sb)[NT], int (&nsa)[MT], int (&nsb)[NT])
                   __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
      const int step = i / (MT * NT), mt = i % (MT * NT) / NT, nt = i % NT;
      if constexpr (A4) {
        const v8i a = wide(f.a[mt][step], v4i{0, 0, 0, 0}), b = wide(f.b[nt][step], v4i{0, 0, 0, 0});
#define MXFP8_STEP(SEL)                                                                                         \
  acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[mt][nt], kMfmaFmt<kE2M1>,             \
                                                               kMfmaFmt<kE2M1>, SEL, sb[nt], SEL, sa[mt])
        if (h == 0 && step == 0) MXFP8_STEP(0);
        else if (h == 0) MXFP8_STEP(1);
        else if (step == 0) MXFP8_STEP(2);
        else MXFP8_STEP(3);
#undef MXFP8_STEP
      } else {
        const v8i a = wide(f.a[mt][0], f.a[mt][1]), b = wide(f.b[nt][0], v4i{0, 0, 0, 0});
        if (h == 0)
          acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[mt][nt], kMfmaFmt<kE2M1>,
                                                                       kMfmaFmt<AFMT>, 0, sb[nt], 0, sa[mt]);
        else
          acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[mt][nt], kMfmaFmt<kE2M1>,
                                                                       kMfmaFmt<AFMT>, 1, sb[nt], 1, sa[mt]);
      }
      if (sc && i == 0) read_scales(kb + 1, nsa, nsb);
      if (sg && i == 0) scale_loads((kb >> 2) + 1);  // after the scale reads: same array
#pragma unroll
      for (int item = 0; item < DS_ITEMS; ++item)
        if (rd && item * DS_SPAN / DS_ITEMS == i) ds_item(next_p, next_h, item, nf);
#pragma unroll
      for (int item = 0; item < DMA_ITEMS; ++item)
        if (dma && item * MFMAS / DMA_ITEMS == i) dma_item(p, kb + RING, item);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  Frags f0, f1;
  int sa0[MT], sb0[NT], sa1[MT], sb1[NT];
  // K block kb in buffer p.  dma: K block kb + RING exists; next: kb + 1 does.
  // With four buffers two K blocks stay in flight across the wait.
  auto kblock = [&](int p, int kb, bool dma, bool next, bool sg, const int (&sa)[MT], const int (&sb)[NT],
                    int (&nsa)[MT], int (&nsb)[NT]) __attribute__((always_inline)) {
    stage(p, 0, kb, true, p, 1, false, false, false, f0, f1, sa, sb, nsa, nsb);
    if (next) wait_loads_and_meet<(RING - 2) * DMA_ITEMS>();
    stage(p, 1, kb, next, (p + 1) % RING, 0, next, dma, sg, f1, f0, sa, sb, nsa, nsb);
  };

  [[maybe_unused]] uint32_t spoilt[MT][NT];
  [[maybe_unused]] bool spoils = false;

  // Epilogue: each wave stages a 32-row strip at a time in its own part of a
  // buffer nobody reads any more and writes whole row segments, past the
  // caches (C is written once).  A lane holds, of each 32 x 32 block, row
  // lane & 31 and the columns 8 q + 4 g .. +3.
  auto epilogue = [&](uint8_t* stage_buf) __attribute__((always_inline)) {
    constexpr bool F32 = sizeof(OutT) == 4;
    constexpr int P = F32 ? WN * 4 : WN * 2 + 16;  // bytes per staged row
    constexpr int CH = F32 ? WN / 4 : WN / 8;      // 16-byte pieces per row
    constexpr int PER = F32 ? 4 : 8, ROWS_PER = 64 / CH;
    uint8_t* stg = stage_buf + wave * (32 * P);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v4f v = v4f{acc[mt][nt][4 * q], acc[mt][nt][4 * q + 1], acc[mt][nt][4 * q + 2], acc[mt][nt][4 * q + 3]};
          if constexpr (F32)
            *reinterpret_cast<v4f*>(stg + (lane & 31) * P + (((nt * 8 + 2 * q + g) ^ (lane & 15)) * 16)) = v;
          else
            *reinterpret_cast<uint2*>(stg + (lane & 31) * P + (nt * 32 + 8 * q + 4 * g) * 2) =
                make_uint2(mx_bf16x2(v[0], v[1]), mx_bf16x2(v[2], v[3]));
        }
#pragma unroll
      for (int it = 0; it < 32 / ROWS_PER; ++it) {
        const int rr = it * ROWS_PER + lane / CH, ch = lane % CH;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rr * P + ((F32 ? ch ^ (rr & 15) : ch) * 16));
        const int m = m0 + wm * WM + mt * 32 + rr, n = n0 + wn * WN + ch * PER;
        if (m < M) {
          OutT* dst = C + (int64_t)m * ldc + n;
          if (n + PER <= N) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dst));
          } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (n + i < N) {
                if constexpr (F32) dst[i] = __uint_as_float(v[i]);
                else dst[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
              }
          }
        }
      }
    }
    // Columns that a value of up leaves without a result, over what was written (a
    // choice among the values above costs 2 us a tile, spoilt or not).
    if constexpr (ADAPT) {
      if (spoils) {
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int m = m0 + wm * WM + mt * 32 + (lane & 31), n = n0 + wn * WN + nt * 32;
            if (m < M) {
#pragma nounroll
              for (uint32_t left = spoilt[mt][nt]; left; left &= left - 1) {
                const int at = n + __builtin_ctz(left);
                if (at < N) {
                  if constexpr (F32) C[(int64_t)m * ldc + at] = __builtin_nanf("");
                  else C[(int64_t)m * ldc + at] = 0x7FC0;
                }
              }
            }
          }
      }
    }
  };

  [[maybe_unused]] std::conditional_t<ADAPT, FirstAdapters<MT, NT>, NoAdapters> lead;
  if constexpr (ADAPT) {
    lead.ask(ad, M, m0 + wm * WM, lane);
    __builtin_amdgcn_sched_barrier(0);
  }
  // The first RING K blocks in flight.
  scale_loads(0);
#pragma unroll
  for (int q = 0; q < RING; ++q)
#pragma unroll
    for (int item = 0; item < DMA_ITEMS; ++item) dma_item(q, q, item);
  if constexpr (ADAPT) {
    spoils = lead.add(ad, M, N, m0 + wm * WM, n0 + wn * WN, lane, acc, spoilt);
    mfma_retire_pad();
  }
  wait_loads_and_meet<(RING - 1) * DMA_ITEMS>();
#pragma unroll
  for (int item = 0; item < DS_ITEMS; ++item) ds_item(0, 0, item, f0);
  read_scales(0, sa0, sb0);

  if constexpr (RING == 4) {
    // K blocks in fours, then up to three more.  Every one loads the block four
    // later and reads the next one's fragments, whether or not they exist (then
    // zeros), so that the waits count the same loads everywhere.
    int kb = 0;
#pragma nounroll
    for (; kb + 4 <= nkb; kb += 4) {
      kblock(0, kb, true, true, true, sa0, sb0, sa1, sb1);
      kblock(1, kb + 1, true, true, false, sa1, sb1, sa0, sb0);
      kblock(2, kb + 2, true, true, false, sa0, sb0, sa1, sb1);
      kblock(3, kb + 3, true, true, false, sa1, sb1, sa0, sb0);
    }
    if (kb < nkb) {
      kblock(0, kb, true, true, true, sa0, sb0, sa1, sb1);
      if (kb + 1 < nkb) {
        kblock(1, kb + 1, true, true, false, sa1, sb1, sa0, sb0);
        if (kb + 2 < nkb) kblock(2, kb + 2, true, true, false, sa0, sb0, sa1, sb1);
      }
    }
    mfma_retire_pad();
    wait_loads_and_meet<0>();  // nothing is on its way to the buffers any more
    epilogue(kbuf0);
  } else {
  // K blocks whose second stage loads a later one, in fours (one scale group
  // each), then a pair and a lone one.
  const int main_kb = nkb - 2;
  int kb = 0;
#pragma nounroll
  for (; kb + 3 < main_kb; kb += 4) {
    kblock(0, kb, true, true, true, sa0, sb0, sa1, sb1);
    kblock(1, kb + 1, true, true, false, sa1, sb1, sa0, sb0);
    kblock(0, kb + 2, true, true, false, sa0, sb0, sa1, sb1);
    kblock(1, kb + 3, true, true, false, sa1, sb1, sa0, sb0);
    asm volatile("; four K blocks");  // differs from the pair's: shared code would move the accumulators about
  }
  if (kb + 1 < main_kb) {
    kblock(0, kb, true, true, true, sa0, sb0, sa1, sb1);
    kblock(1, kb + 1, true, true, false, sa1, sb1, sa0, sb0);
    asm volatile("; two K blocks");
    kb += 2;
  }
  if (kb < main_kb) {
    kblock(0, kb, true, true, false, sa0, sb0, sa1, sb1);
#pragma unroll
    for (int t = 0; t < MT; ++t) sa0[t] = sa1[t];
#pragma unroll
    for (int t = 0; t < NT; ++t) sb0[t] = sb1[t];
  }
  const int p = nkb & 1;  // buffer of K block nkb - 2
  kblock(p, nkb - 2, false, true, false, sa0, sb0, sa1, sb1);
  kblock(p ^ 1, nkb - 1, false, false, false, sa1, sb1, sa0, sb0);
  mfma_retire_pad();
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));  // the accumulators stay where they are
  epilogue(buf_ptr(p));
  }
#endif
}

template <int BM, int BN, int AFMT, bool SW, int RING, typename OutT, typename AD>
__global__ __launch_bounds__(kTileThreads, BM == 128 && RING == 2 ? 2 : 1) void tile_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ SA,
    const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ SB, OutT* __restrict__ C, int64_t ldc,
    int tiles_m, int tiles_n, AD ad) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef Tile<BM, BN, AFMT> T;
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf0[T::PB];
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf1[T::PB];
  __shared__ __attribute__((aligned(1024))) uint8_t sgrp[T::SGRP];
  if constexpr (RING == 4) {
    __shared__ __attribute__((aligned(1024))) uint8_t kbuf2[T::PB];
    __shared__ __attribute__((aligned(1024))) uint8_t kbuf3[T::PB];
    gemm_tile<BM, BN, AFMT, SW, RING, OutT, AD>(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, tiles_m, tiles_n, 0, 0, 0,
                                            blockIdx.x, gridDim.x, kbuf0, kbuf1, kbuf2, kbuf3, sgrp, ad);
  } else {
    gemm_tile<BM, BN, AFMT, SW, RING, OutT, AD>(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, tiles_m, tiles_n, 0, 0, 0,
                                            blockIdx.x, gridDim.x, kbuf0, kbuf1, nullptr, nullptr, sgrp, ad);
  }
#endif
}

// The 256 x 256 cells past the last full round of the chip as 128 x 128
// quadrants (first in launch order), the full rounds after them.
template <int AFMT, bool SW, typename OutT, typename AD>
__global__ __launch_bounds__(kTileThreads, 1) void tail_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ SA,
    const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ SB, OutT* __restrict__ C, int64_t ldc,
    int tiles_m, int tiles_n, int big, AD ad) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef Tile<256, 256, AFMT> T;
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf0[T::PB];
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf1[T::PB];
  __shared__ __attribute__((aligned(1024))) uint8_t sgrp[T::SGRP];
  const int nq = (int)gridDim.x - big, b = blockIdx.x;
  if (b >= nq)
    gemm_tile<256, 256, AFMT, SW, 2, OutT, AD>(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, tiles_m, tiles_n, 0, 0, 0, b - nq,
                                        big, kbuf0, kbuf1, nullptr, nullptr, sgrp, ad);
  else
    gemm_tile<128, 128, AFMT, SW, 2, OutT, AD>(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, tiles_m, tiles_n, big, 1, 1, b, nq,
                                        kbuf0, kbuf1, nullptr, nullptr, sgrp, ad);
#endif
}

template <int AFMT, bool SW, typename OutT, typename AD>
void tiles(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
           int64_t ldb, const uint8_t* sb, OutT* c, int64_t ldc, AD ad, hipStream_t stream) {
  const int bm = (int)((M + 255) / 256), bn = (int)((N + 255) / 256), big = bm * bn;
  const int sm = (int)((M + 127) / 128), sn = (int)((N + 127) / 128), cus = device_cus();
  // 128 x 128 tiles while they fit on the CUs at two per CU.  At one per CU
  // nothing else hides a K block's load, so four buffers hold it (us, four /
  // two: E4M3 x E2M1 256x3584x18944 59 / 88, 1024x3584x3584 15.9 / 20.4; E2M1
  // pairs 38 / 57, 11.6 / 13.4); a short K is over before that pays
  // (1000x1024x1024 6.4 / 6.1, 5.8 / 5.2; 512x8960x1536 12.8 / 12.7, 9.6 / 9.8).
  if (sm * sn <= cus && K >= 1536) {
    hipLaunchKernelGGL((tile_kernel<128, 128, AFMT, SW, 4, OutT, AD>), dim3(sm * sn), dim3(kTileThreads), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, c, ldc, sm, sn, ad);
    return;
  }
  if (sm * sn <= 2 * cus) {
    hipLaunchKernelGGL((tile_kernel<128, 128, AFMT, SW, 2, OutT, AD>), dim3(sm * sn), dim3(kTileThreads), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, c, ldc, sm, sn, ad);
    return;
  }
  const int tail = big % cus;
  if (big > cus && tail > 0 && 4 * tail <= cus)
    hipLaunchKernelGGL((tail_kernel<AFMT, SW, OutT, AD>), dim3(big + 3 * tail), dim3(kTileThreads), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, c, ldc, bm, bn, big - tail, ad);
  else
    hipLaunchKernelGGL((tile_kernel<256, 256, AFMT, SW, 2, OutT, AD>), dim3(big), dim3(kTileThreads), 0, stream, (int)M,
                       (int)N, (int)K, a, lda, sa, b, ldb, sb, c, ldc, bm, bn, ad);
}

template <int AFMT, typename AD>
void gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, const uint8_t* sa, const uint8_t* b,
          int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, AD ad, hipStream_t stream) {
  const int chunks = (int)(K / 128);
  const int64_t n16 = (N + 15) / 16, pairs = ((N + 31) / 32) * ((M + 31) / 32), cus = device_cus();
#define MXFP4_FEW(MT, NT, WAVES, U)                                                                           \
  (few_rows_lds<AFMT, MT, NT, WAVES, true>(M < 16 * MT ? M : 16 * MT, K) <= kFewRowsLds                       \
       ? few_rows<AFMT, MT, NT, WAVES, U, true>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream) \
       : few_rows<AFMT, MT, NT, WAVES, U, false>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream))
  if (mxfp4_few_rows(M, N, K, cus)) {
    if (M <= 16) {
      // Two waves a workgroup where a run of K is short or the workgroups are
      // many (E4M3, two / four waves: 1x8960x1536 3.8 / 4.2 us, 1x18944x3584
      // 8.2 / 8.7; 1x3584x18944 9.1 / 8.8, 8x4096x4096 5.4 / 5.2), unless each
      // then copies many rows of A (E2M1 pairs, 16x18944x3584: 11.9 / 10.3).
      // Where many workgroups would hold much of A each, wider ones (E4M3,
      // 16x18944x3584: 12.8 against 15.6).
      const bool wide_a = M * (AFMT == kE2M1 ? K / 2 : K) > 32 * 1024 && n16 >= 512;
      if (wide_a) MXFP4_FEW(1, 2, 8, 2);
      else if (chunks <= 16 || (n16 >= 512 && M <= 8))  // A, 32 KB at most, always fits
        few_rows<AFMT, 1, 1, 2, 4, true>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream);
      else MXFP4_FEW(1, 1, 4, 4);
    } else if (pairs < 128 && M <= 48) {
      // Few workgroups of 32 x 32 (us, 16x16, 16x32 and 32x32 ones, E4M3 x
      // E2M1 and E2M1 pairs: 37x1536x8960 10.8 / 7.7, 11.9 / 8.1, 16.7 / 12.0;
      // 64x1536x8960 15.7 / 8.6, 12.3 / 8.5, 17.0 / 12.3).
      MXFP4_FEW(1, 1, 4, 4);
    } else if (pairs < 128) {
      MXFP4_FEW(1, 2, 8, 2);
    } else if (pairs <= cus) {
      MXFP4_FEW(2, 2, 4, 4);
    } else {
      // 32 x 64 ones where those of 32 x 32 would take a second round (us,
      // 32x64 / 32x32: 128x3584x3584 8.8 / 15.5, 7.8 / 8.9; 256x1536x18944 37 /
      // 55, 29 / 37).
      MXFP4_FEW(2, 4, 4, 1);
    }
  } else {
    const bool sw = K % 512 == 0 && (((uintptr_t)sa | (uintptr_t)sb) & 15) == 0;
    float* cf = static_cast<float*>(c);
    uint16_t* cb = static_cast<uint16_t*>(c);
    if (c_dtype == 0)
      sw ? tiles<AFMT, true>(M, N, K, a, lda, sa, b, ldb, sb, cf, ldc, ad, stream)
         : tiles<AFMT, false>(M, N, K, a, lda, sa, b, ldb, sb, cf, ldc, ad, stream);
    else
      sw ? tiles<AFMT, true>(M, N, K, a, lda, sa, b, ldb, sb, cb, ldc, ad, stream)
         : tiles<AFMT, false>(M, N, K, a, lda, sa, b, ldb, sb, cb, ldc, ad, stream);
  }
#undef MXFP4_FEW
}

#define MXFP4_GEMM(FMT, AD)                                                                                     \
  template void gemm<FMT, AD>(int64_t, int64_t, int64_t, const uint8_t*, int64_t, const uint8_t*, const uint8_t*, \
                              int64_t, const uint8_t*, void*, int64_t, int, AD, hipStream_t);
#if MXFP4_GEMM_FMT == 3
MXFP4_GEMM(0, NoAdapters)
MXFP4_GEMM(1, NoAdapters)
MXFP4_GEMM(2, NoAdapters)
MXFP4_GEMM(0, Adapters)
MXFP4_GEMM(1, Adapters)
MXFP4_GEMM(2, Adapters)
#elif MXFP4_GEMM_ADAPT
MXFP4_GEMM(MXFP4_GEMM_FMT, Adapters)
#else
MXFP4_GEMM(MXFP4_GEMM_FMT, NoAdapters)
#endif
#undef MXFP4_GEMM

#endif  // MXFP4_GEMM_FMT >= 0

}  // namespace mxfp4_detail

#if MXFP4_GEMM_FMT == 3 || MXFP4_GEMM_FMT < 0
// Few rows or tiles.  Up to 16 rows B crosses a CU's load path once however
// wide it is.  Beyond, the few-row kernel is the faster one while its
// workgroups all fit on the chip, one to a CU, since it has four times or
// more as many of them as there are tiles; with a second round of them the
// tiles win (us, few rows / tiles, E4M3 x E2M1 and E2M1 pairs, one round:
// 64x3584x8960 17.2 / 26.7, 12.6 / 18.8; 128x3584x3584 8.8 / 13.4, 7.8 / 9.5;
// 512x1024x1024 5.5 / 6.1, 4.9 / 5.2; 32x14336x4096 12.2 / 14.1, 10.0 / 10.4;
// more: 40x16384x3584 17 / 13, 12.1 / 10.0; 256x3584x3584 19.2 / 14.2,
// 15.7 / 10.3; 1024x1024x1024 9.1 / 6.2, 8.4 / 5.3).  The few-row kernel
// takes as many scales as fit in LDS and 2^26 rows of B (its grid).
bool mxfp4_few_rows(int64_t M, int64_t N, int64_t K, int64_t cus) {
  using namespace mxfp4_detail;
  const int64_t pairs = ((N + 31) / 32) * ((M + 31) / 32), wide = ((N + 63) / 64) * ((M + 31) / 32);
  // A's own place in LDS is not counted: rows that do not fit stay in memory.
  return (M <= 16 ? N <= kFewRowsN : wide <= cus) &&
         (M <= 16 || pairs <= cus ? few_rows_lds<0, 2, 2, 4, false>(0, K)
                                  : few_rows_lds<0, 2, 4, 4, false>(0, K)) <= kFewRowsLds;
}

namespace {
template <typename AD>
void any_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
              const uint8_t* b, int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype, AD ad,
              hipStream_t stream) {
  using mxfp4_detail::gemm;
  if (a_fmt == 0) gemm<0, AD>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream);
  else if (a_fmt == 1) gemm<1, AD>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream);
  else gemm<kE2M1, AD>(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream);
}
}  // namespace

void launch_mxfp4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt, const uint8_t* sa,
                       const uint8_t* b, int64_t ldb, const uint8_t* sb, void* c, int64_t ldc, int c_dtype,
                       hipStream_t stream) {
  any_gemm(M, N, K, a, lda, a_fmt, sa, b, ldb, sb, c, ldc, c_dtype, mxfp4_detail::NoAdapters{}, stream);
}

void launch_mxfp4_gemm_adapted(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda, int a_fmt,
                               const uint8_t* sa, const uint8_t* b, int64_t ldb, const uint8_t* sb, const int32_t* ids,
                               int64_t adapters, int64_t rank, const float* p, const uint16_t* packed, const uint16_t* up,
                               int64_t ldu, int64_t stride, void* c, int64_t ldc, int c_dtype, hipStream_t stream) {
  const mxfp4_detail::Adapters ad{ids, p, packed, up, ldu, stride, (int)adapters, (int)rank};
  any_gemm(M, N, K, a, lda, a_fmt, sa, b, ldb, sb, c, ldc, c_dtype, ad, stream);
}

#endif

}  // namespace mxfp8
