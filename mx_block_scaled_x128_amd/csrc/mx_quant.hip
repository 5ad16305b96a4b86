// mx_quant.hip -- MX quantizers and their inverse for gfx950:
//   mxfp4_quantize   rows into E2M1 codes, one E8M0 scale per 32 columns;
//   mx_quantize_t    32-token blocks down the columns, codes transposed, into
//                    E4M3 / E5M2 / E2M1: the operands whose K axis is the
//                    token axis (dW) or the output features (dX from W);
//   mx_requantize_t  the same from FP8 codes (an activation kept in 8 bits):
//                    the weight gradient's operand without the tensor itself;
//   mx_dequantize    codes and scales back to values.
// For a block with largest magnitude amax, e its exponent (mx_scale):
//   scale byte = e + 127,  code = cast(x * 2^-e), to nearest even, saturating.
// All four move each byte once.  HBM bounds the row-wise ones; the transposers
// come near it, held back by vector instructions and scattered scale lines
// (from codes most) and by a launch's start and end.
#include <type_traits>

#include "mx_common.hpp"
#include "mx_launch.hpp"

namespace mxfp8 {

namespace mx_quant_detail {

constexpr int kThreads = 256;
// Workgroups at most, grid-stride beyond.  The quantizer keeps 8 per compute
// unit (18944x3584 bf16: 30.2 us, 64 per unit 32.3); dequantizing to 16 bits
// writes twice what it reads and is faster with 64 and two units a lane
// (8192x18944: 74.5 us; 8 per unit and four units 81.9; 86.4 with ordinary
// stores).
constexpr uint32_t kQuantBlocks = 256 * 8, kDequantBlocks = 256 * 64;
constexpr int kQuantUnits = 4, kDequantUnits = 2;

// The row-wise kernels walk units of 8 elements in row-major order; a wave
// takes U * 64 consecutive units at a time, so only one division per wave and
// round (on the scalar unit) finds the row, and lanes step over row ends
// themselves.
struct Place {
  int64_t row;
  uint32_t unit;  // within the row
};
struct RowWalk {
  int64_t row0;
  uint32_t unit0, upr;
  __device__ __forceinline__ RowWalk(int64_t base, uint32_t units_per_row) : upr(units_per_row) {
    row0 = base <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)base / upr) : base / upr;
    unit0 = (uint32_t)(base - row0 * upr);
  }
  __device__ __forceinline__ Place at(uint32_t step) const {
    uint32_t c = unit0 + step;
    int64_t r = row0;
    if (c >= upr) {
      const uint32_t d = c / upr;
      r += d;
      c -= d * upr;
    }
    return Place{r, c};
  }
};

template <typename InT, bool CEIL, int U, bool NT>
__global__ __launch_bounds__(kThreads) void mxfp4_rows_kernel(const InT* __restrict__ x, int64_t ldx, uint32_t upr,
                                                              int64_t total, uint8_t* __restrict__ q,
                                                              int64_t ldq, uint8_t* __restrict__ s) {
  const uint32_t lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 64) * (64 * U);
  for (int64_t base = wave * (64 * U); base < total; base += step) {
    const RowWalk walk(base, upr);
    MxRaw<InT> raw[U];
    Place p[U];
    bool act[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = walk.at(u * 64 + lane);
      act[u] = base + u * 64 + lane < total;
      if (act[u]) mx_load_raw<NT>(x + p[u].row * ldx + p[u].unit * 8, raw[u]);
      else mx_zero_raw(raw[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      mx_unpack(raw[u], f);
      // a row holds whole blocks, so a quad never straddles rows or the end
      const uint32_t sc = mx_scale<kE2M1, CEIL>(max_quad(absmax8(f)));
      const uint2 w = mx_codes8<kE2M1, CEIL>(f, sc);
      if (act[u]) {
        mx_store_codes8<kE2M1>(q + p[u].row * ldq + p[u].unit * 4, w);
        if ((lane & 3) == 0) s[p[u].row * (upr >> 2) + (p[u].unit >> 2)] = (uint8_t)sc;
      }
    }
  }
}

template <int FMT, typename OutT, int U, bool NT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                                 const uint8_t* __restrict__ s, uint32_t upr,
                                                                 int64_t total, OutT* __restrict__ y, int64_t ldy) {
  const uint32_t lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 64) * (64 * U);
  for (int64_t base = wave * (64 * U); base < total; base += step) {
    const RowWalk walk(base, upr);
    uint2 w[U];
    uint32_t b[U];
    Place p[U];
    bool act[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = walk.at(u * 64 + lane);
      act[u] = base + u * 64 + lane < total;
      w[u] = make_uint2(0u, 0u);
      b[u] = 0;
      if (act[u]) {
        w[u] = mx_load_codes8<FMT>(q + p[u].row * ldq + p[u].unit * MxFmt<FMT>::code_bits);
        b[u] = s[p[u].row * (upr >> 2) + (p[u].unit >> 2)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      mx_decode8<FMT>(w[u], mx_factor(b[u]), f);
      if (act[u]) mx_store8<NT>(y + p[u].row * ldy + p[u].unit * 8, f);
    }
  }
}

// ---------------------------------------------------------------------------
// 32-token blocks down the columns, transposed.  One workgroup per 128 tokens
// x 128 channels.  A thread holds 4 tokens x CH channels (16 bytes of a row,
// or 32 of fp32), so that each load instruction takes 8 whole 128-byte (or
// 256-byte) row segments; the 8 lanes of a wave that share a channel chunk
// hold 32 tokens of it, which are one MX block: its maximum is three DPP steps
// and no barrier.  Codes go through an LDS tile (rows of 128 codes, padded)
// and leave as whole rows of the output; the tile's 128 x 4 scale bytes leave
// as one dword per channel.
// Tiles are taken token by token, each XCD (workgroups go round them) a
// contiguous run: the 4-byte pieces that neighbouring tiles write of one line
// of scales, and read of one line of a source's, then meet in one L2
// (channel by channel across the XCDs, 8 codes to a load: 4099x8960 codes 21.8
// us, 8192x8960 bf16 44.8; this way 17.5 and 41.0, and 16.0 and 40.6 with the
// conversions that take the scale; 8960x1536 fp32 into E2M1 stays at 13.1).
// SRC: MXFP8_F32 / MXFP8_BF16 elements, or 2 + FP8 format for codes with
// scales per 32 columns.
// ---------------------------------------------------------------------------
template <int SRC> struct Source {  // codes
  typedef uint8_t T;
  static constexpr int CH = 16;
};
template <> struct Source<0> {
  typedef float T;
  static constexpr int CH = 8;
};
template <> struct Source<1> {
  typedef uint16_t T;
  static constexpr int CH = 8;
};
constexpr int kTile = 128;
template <int SRC> constexpr int kTThreads = kTile / 4 * (kTile / Source<SRC>::CH);

template <int SRC, int FMT, bool CEIL, bool NT>
__global__ __launch_bounds__(kTThreads<SRC>) void mx_transpose_kernel(
    const void* __restrict__ x, int64_t ldx, const uint8_t* __restrict__ s, uint32_t rows, uint32_t cols,
    uint8_t* __restrict__ qt, int64_t ldqt, uint32_t rows_out, uint8_t* __restrict__ st) {
  constexpr int THREADS = kTThreads<SRC>, CH = Source<SRC>::CH;
  constexpr int RB = kTile * MxFmt<FMT>::code_bits / 8;  // bytes of 128 codes
  constexpr int PITCH = RB + 8;
  __shared__ __attribute__((aligned(16))) uint8_t tile[kTile * PITCH];
  __shared__ __attribute__((aligned(4))) uint8_t stile[kTile * 4];
  const uint32_t tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const uint32_t tr = (lane & 7) + 8 * (w & 3);    // token chunk: tokens tr*4 .. tr*4+3
  const uint32_t tc = (lane >> 3) + 8 * (w >> 2);  // channel chunk: channels tc*CH .. tc*CH+CH-1
  const uint32_t gx = (cols + 127) >> 7, gy = (rows_out + 127) >> 7;
  const uint32_t t = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (t >= gx * gy) return;  // the grid is a multiple of 8
  const uint32_t bx = t / gy, by = t - bx * gy;
  const uint32_t c0 = bx * kTile, t0 = by * kTile;
  const bool cact = c0 + tc * CH < cols;
  // The four tokens as read; eight channels at a time are converted.
  typedef typename Source<SRC>::T T;
  typename std::conditional<SRC < 2, MxRaw<T>, nt_u32x4>::type raw[4];
  float factor[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = t0 + tr * 4 + i;
    const bool in = cact && r < rows;
    if constexpr (SRC < 2) {
      if (in) mx_load_raw<NT>(static_cast<const T*>(x) + (int64_t)r * ldx + c0 + tc * CH, raw[i]);
      else mx_zero_raw(raw[i]);
    } else {
      raw[i] = nt_u32x4{0, 0, 0, 0};
      uint32_t b = 0;
      if (in) {
        raw[i] = *reinterpret_cast<const nt_u32x4*>(static_cast<const uint8_t*>(x) + (int64_t)r * ldx + c0 + tc * CH);
        b = s[(int64_t)r * (cols >> 5) + ((c0 + tc * CH) >> 5)];
      }
      factor[i] = mx_factor(b);
    }
  }
#pragma unroll
  for (int part = 0; part < CH / 8; ++part) {
    float f[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (SRC < 2) {
        mx_unpack(raw[i], f[i]);
      } else {
        const uint2 w8 = part == 0 ? make_uint2(raw[i].x, raw[i].y) : make_uint2(raw[i].z, raw[i].w);
        mx_decode8<(SRC < 2 ? 0 : SRC - 2)>(w8, factor[i], f[i]);
      }
    }
    uint32_t sc[8], top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = max_oct(max(max(abs_bits(f[0][j]), abs_bits(f[1][j])), max(abs_bits(f[2][j]), abs_bits(f[3][j]))));
      sc[j] = mx_scale_finite<FMT, CEIL>(m);
      top = max(top, m);
    }
    const uint32_t ch = tc * CH + part * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t o = mx_codes4<FMT, CEIL>(f[0][j], f[1][j], f[2][j], f[3][j], sc[j]);
      if constexpr (FMT == kE2M1) *reinterpret_cast<uint16_t*>(tile + (ch + j) * PITCH + tr * 2) = (uint16_t)o;
      else *reinterpret_cast<uint32_t*>(tile + (ch + j) * PITCH + tr * 4) = o;
    }
    // Channels with an infinity or a NaN, once more (rare: one test for eight).
    if (top >= kInfBits) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, abs_bits(f[i][j]));
        m = max_oct(m);  // the same in the eight lanes of the block, which all are here
        if (m < kInfBits) continue;
        sc[j] = 255u;
        if constexpr (FMT == kE2M1) *reinterpret_cast<uint16_t*>(tile + (ch + j) * PITCH + tr * 2) = 0;
        else *reinterpret_cast<uint32_t*>(tile + (ch + j) * PITCH + tr * 4) = 0;
      }
    }
    if ((lane & 7) == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) stile[(ch + j) * 4 + (w & 3)] = (uint8_t)sc[j];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
  constexpr int CPR = RB / 16;  // 16-byte chunks per tile row
#pragma unroll
  for (int rep = 0; rep < kTile * CPR / THREADS; ++rep) {
    const uint32_t idx = rep * THREADS + tid;
    const uint32_t ch = idx / CPR, ck = idx % CPR;
    if (c0 + ch < cols && t0 + ck * (kTile / CPR) < rows_out) {
      const uint2 a = *reinterpret_cast<const uint2*>(tile + ch * PITCH + ck * 16);
      const uint2 b = *reinterpret_cast<const uint2*>(tile + ch * PITCH + ck * 16 + 8);
      store_codes(qt + (int64_t)(c0 + ch) * ldqt + ((int64_t)by * RB + ck * 16), make_uint4(a.x, a.y, b.x, b.y));
    }
  }
  const uint32_t ngt = rows_out >> 5;
  if (tid < kTile && c0 + tid < cols) {
    uint8_t* dst = st + (int64_t)(c0 + tid) * ngt + (t0 >> 5);
    if ((ngt & 3) == 0 && ((uintptr_t)st & 3) == 0) {
      *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(stile + tid * 4);
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        if ((t0 >> 5) + i < ngt) dst[i] = stile[tid * 4 + i];
    }
  }
}

uint32_t row_blocks(int64_t total, int u, uint32_t most) {
  const int64_t per = (int64_t)kThreads * u;
  const int64_t n = (total + per - 1) / per;
  return (uint32_t)(n < most ? n : most);
}

// Several units in flight per lane where that still fills the chip with
// workgroups, else one.
bool deep(int64_t total) { return total >= (int64_t)kThreads * 4 * device_cus(); }

template <typename InT, bool CEIL>
void rows4(const InT* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* s,
           hipStream_t stream) {
  const uint32_t upr = (uint32_t)(cols / kLaneElems);
  const int64_t total = rows * upr;
#define MXFP8_ROWS4(U, NT)                                                                                         \
  hipLaunchKernelGGL((mxfp4_rows_kernel<InT, CEIL, U, NT>), dim3(row_blocks(total, U, kQuantBlocks)), dim3(kThreads), 0, stream, \
                     x, ldx, upr, total, q, ldq, s)
  if (!deep(total)) MXFP8_ROWS4(1, false);
  else if (stream_loads(rows, cols, sizeof(InT))) MXFP8_ROWS4(kQuantUnits, true);
  else MXFP8_ROWS4(kQuantUnits, false);
#undef MXFP8_ROWS4
}
template <typename InT>
void rows4(const InT* x, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t* q, int64_t ldq, uint8_t* s,
           hipStream_t stream) {
  if (rule == 0) rows4<InT, true>(x, rows, cols, ldx, q, ldq, s, stream);
  else rows4<InT, false>(x, rows, cols, ldx, q, ldq, s, stream);
}

template <int FMT, typename OutT>
void dequantize(const uint8_t* q, int64_t ldq, const uint8_t* s, int64_t rows, int64_t cols, OutT* y, int64_t ldy,
                hipStream_t stream) {
  const uint32_t upr = (uint32_t)(cols / kLaneElems);
  const int64_t total = rows * upr;
#define MXFP8_DEQ(U, NT)                                                                                            \
  hipLaunchKernelGGL((mx_dequantize_kernel<FMT, OutT, U, NT>), dim3(row_blocks(total, U, kDequantBlocks)),          \
                     dim3(kThreads), 0, stream, q, ldq, s, upr, total, y, ldy)
  if (!deep(total)) MXFP8_DEQ(1, false);
  else if (stream_loads(rows, cols, sizeof(OutT))) MXFP8_DEQ(kDequantUnits, true);
  else MXFP8_DEQ(kDequantUnits, false);
#undef MXFP8_DEQ
}

template <int SRC, int FMT, bool CEIL>
void transpose(const void* x, int64_t ldx, const uint8_t* s, int64_t rows, int64_t cols, uint8_t* qt, int64_t ldqt,
               int64_t rows_out, uint8_t* st, hipStream_t stream) {
  const dim3 grid((uint32_t)((((cols + 127) / 128) * ((rows_out + 127) / 128) + 7) / 8 * 8));
  if (SRC < 2 && stream_loads(rows, cols, SRC == 0 ? 4 : 2))
    hipLaunchKernelGGL((mx_transpose_kernel<SRC, FMT, CEIL, (SRC < 2)>), grid, dim3(kTThreads<SRC>), 0,
                       stream, x, ldx, s, (uint32_t)rows, (uint32_t)cols, qt, ldqt, (uint32_t)rows_out, st);
  else
    hipLaunchKernelGGL((mx_transpose_kernel<SRC, FMT, CEIL, false>), grid, dim3(kTThreads<SRC>), 0,
                       stream, x, ldx, s, (uint32_t)rows, (uint32_t)cols, qt, ldqt, (uint32_t)rows_out, st);
}

template <int SRC>
void transpose_to(const void* x, int64_t ldx, const uint8_t* s, int64_t rows, int64_t cols, int fmt, int rule,
                  uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* st, hipStream_t stream) {
#define MXFP8_T(FMT)                                                                       \
  (rule == 0 ? transpose<SRC, FMT, true>(x, ldx, s, rows, cols, qt, ldqt, rows_out, st, stream) \
             : transpose<SRC, FMT, false>(x, ldx, s, rows, cols, qt, ldqt, rows_out, st, stream))
  if (fmt == 0) MXFP8_T(0);
  else if (fmt == 1) MXFP8_T(1);
  else MXFP8_T(kE2M1);
#undef MXFP8_T
}

}  // namespace mx_quant_detail

using namespace mx_quant_detail;

void launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t* q,
                           int64_t ldq, uint8_t* s, hipStream_t stream) {
  if (dtype == 0) rows4(static_cast<const float*>(x), rows, cols, ldx, rule, q, ldq, s, stream);
  else rows4(static_cast<const uint16_t*>(x), rows, cols, ldx, rule, q, ldq, s, stream);
}

void launch_mx_dequantize(const uint8_t* q, int64_t ldq, int fmt, const uint8_t* s, int64_t rows, int64_t cols,
                          void* y, int y_dtype, int64_t ldy, hipStream_t stream) {
  float* yf = static_cast<float*>(y);
  uint16_t* yb = static_cast<uint16_t*>(y);
#define MXFP8_DEQ(FMT)                                                                     \
  (y_dtype == 0 ? dequantize<FMT, float>(q, ldq, s, rows, cols, yf, ldy, stream)           \
                : dequantize<FMT, uint16_t>(q, ldq, s, rows, cols, yb, ldy, stream))
  if (fmt == 0) MXFP8_DEQ(0);
  else if (fmt == 1) MXFP8_DEQ(1);
  else MXFP8_DEQ(kE2M1);
#undef MXFP8_DEQ
}

void launch_mx_quantize_t(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule,
                          uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* st, hipStream_t stream) {
  if (dtype == 0) transpose_to<0>(x, ldx, nullptr, rows, cols, fmt, rule, qt, ldqt, rows_out, st, stream);
  else transpose_to<1>(x, ldx, nullptr, rows, cols, fmt, rule, qt, ldqt, rows_out, st, stream);
}

void launch_mx_requantize_t(const uint8_t* q, int64_t ldq, int q_fmt, const uint8_t* s, int64_t rows, int64_t cols,
                            int fmt, int rule, uint8_t* qt, int64_t ldqt, int64_t rows_out, uint8_t* st,
                            hipStream_t stream) {
  if (q_fmt == 0) transpose_to<2>(q, ldq, s, rows, cols, fmt, rule, qt, ldqt, rows_out, st, stream);
  else transpose_to<3>(q, ldq, s, rows, cols, fmt, rule, qt, ldqt, rows_out, st, stream);
}

}  // namespace mxfp8
