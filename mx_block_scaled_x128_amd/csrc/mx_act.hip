// mx_act.hip -- SwiGLU and RMSNorm that keep their input in 8 bits for the
// backward pass (gfx950).
//
// Forward, per row of x:
//   SwiGLU   x = (g, u),  h = g * sigma(g) * u,  sigma(g) = 1 / (1 + 2^(-g log2 e))
//   RMSNorm  r = 1 / sqrt(mean(x^2) + eps),  y = x * r * w
// h and y leave as MX codes (32-element blocks, one E8M0 scale), the operand
// of the product that follows; x itself is kept as MX codes (RMSNorm: and r)
// in place of the 16- or 32-bit tensor.
//
// Backward, on the kept values x~ (codes times scales):
//   SwiGLU   dg = dh * u~ * sigma * (1 + g~ * (1 - sigma)),  du = dh * g~ * sigma
//   RMSNorm  c = dy * w,  xh = x~ * r,  dx = r * (c - xh * mean(c * xh)),
//            dw = sum over rows of dy * xh
// Arithmetic is in fp32, RMSNorm's mean and root in 64 bits (and the squares of
// rows that leave fp32's range); the codes and the gradients' own type are the
// only roundings to fewer bits.  Each tensor is read and written once: HBM
// bounds all four.
#include "mx_common.hpp"
#include "mx_launch.hpp"

namespace mxfp8 {

namespace mx_act_detail {

constexpr int kThreads = 256;
// SwiGLU's workgroups at most, grid-stride beyond, and units per lane.  With
// 8192x18944 bf16 (us, 8 / 64 / 256 / 1024 workgroups per compute unit,
// stores past the caches): forward two units a lane 178 / 163 / 166 / 174,
// one unit 169 at 256; backward two units 232 / 209 / 199 / 199, one unit 194
// at 256.  With ordinary stores of what is kept and of dx: 214 and 221 at 64.
constexpr uint32_t kForwardBlocks = 256 * 64, kBackwardBlocks = 256 * 256;
constexpr int kForwardUnits = 2;

// sigma(g).  exp2 and rcp are the hardware's (1 ulp each); the argument's own
// rounding puts a relative error of |g| * 2^-24 on top.  2^(-g log2 e) = inf
// for very negative g gives 0.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

template <typename InT, int FMT, bool CEIL, bool KEEP, int U, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_forward_kernel(
    const InT* __restrict__ x, int64_t ldx, int64_t rows, uint32_t upr, uint8_t* __restrict__ h, int64_t ldh,
    uint8_t* __restrict__ hs, uint8_t* __restrict__ kept, int64_t ldk, uint8_t* __restrict__ ks) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t nwaves = gridDim.x * (kThreads / 64);
  const uint32_t cols = upr * 8, nb = upr >> 2;
  // items of 64 U units of one row; a wave's item is uniform
  const uint32_t ipr = (upr + 64 * U - 1) / (64 * U);
  const int64_t items = rows * ipr;
  for (int64_t it = wave; it < items; it += nwaves) {
    const int64_t row = it <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)it / ipr) : it / ipr;
    const uint32_t unit0 = (uint32_t)(it - row * ipr) * (64 * U) + lane;
    const InT* xr = x + row * ldx;
    MxRaw<InT> rg[U], ru[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t unit = unit0 + i * 64;
      if (unit < upr) {
        mx_load_raw<NT>(xr + unit * 8, rg[i]);
        mx_load_raw<NT>(xr + cols + unit * 8, ru[i]);
      } else {
        mx_zero_raw(rg[i]);
        mx_zero_raw(ru[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t unit = unit0 + i * 64;
      float g[8], u[8], v[8];
      mx_unpack(rg[i], g);
      mx_unpack(ru[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = g[j] * sigmoid(g[j]) * u[j];
      const uint32_t sv = mx_scale<FMT, CEIL>(max_quad(absmax8(v)));
      if constexpr (KEEP) {
        const uint32_t sg = mx_scale<FMT, CEIL>(max_quad(absmax8(g)));
        const uint32_t su = mx_scale<FMT, CEIL>(max_quad(absmax8(u)));
        if (unit < upr) {
          uint8_t* kr = kept + row * ldk;
          mx_keep_codes8<NT>(kr + unit * 8, mx_codes8<FMT, CEIL>(g, sg));
          mx_keep_codes8<NT>(kr + cols + unit * 8, mx_codes8<FMT, CEIL>(u, su));
          if ((lane & 3) == 0) {
            ks[row * (2 * nb) + (unit >> 2)] = (uint8_t)sg;
            ks[row * (2 * nb) + nb + (unit >> 2)] = (uint8_t)su;
          }
        }
      }
      if (unit < upr) {
        mx_store_codes8<FMT>(h + row * ldh + unit * 8, mx_codes8<FMT, CEIL>(v, sv));
        if ((lane & 3) == 0) hs[row * nb + (unit >> 2)] = (uint8_t)sv;
      }
    }
  }
}

template <typename T, int FMT, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    const uint8_t* __restrict__ kept, int64_t ldk, const uint8_t* __restrict__ ks, const T* __restrict__ dh,
    int64_t lddh, int64_t rows, uint32_t upr, T* __restrict__ dx, int64_t lddx) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t nwaves = gridDim.x * (kThreads / 64);
  const uint32_t cols = upr * 8, nb = upr >> 2;
  const uint32_t ipr = (upr + 63) / 64;
  const int64_t items = rows * ipr;
  for (int64_t it = wave; it < items; it += nwaves) {
    const int64_t row = it <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)it / ipr) : it / ipr;
    const uint32_t unit = (uint32_t)(it - row * ipr) * 64 + lane;
    if (unit >= upr) continue;
    const uint2 wg = mx_load_codes8<FMT>(kept + row * ldk + unit * 8);
    const uint2 wu = mx_load_codes8<FMT>(kept + row * ldk + cols + unit * 8);
    const uint32_t bg = ks[row * (2 * nb) + (unit >> 2)], bu = ks[row * (2 * nb) + nb + (unit >> 2)];
    MxRaw<T> rd;
    mx_load_raw<NT>(dh + row * lddh + unit * 8, rd);
    float g[8], u[8], d[8], dg[8], du[8];
    mx_decode8<FMT>(wg, mx_factor(bg), g);
    mx_decode8<FMT>(wu, mx_factor(bu), u);
    mx_unpack(rd, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid(g[j]);
      const float a = d[j] * s;
      du[j] = a * g[j];
      dg[j] = a * u[j] * __builtin_fmaf(g[j], 1.0f - s, 1.0f);
    }
    mx_store8<NT>(dx + row * lddx + unit * 8, dg);
    mx_store8<NT>(dx + row * lddx + cols + unit * 8, du);
  }
}

// ---------------------------------------------------------------------------
// RMSNorm.  WPR waves share a row (1 up to 4096 columns, 4 up to 16384, then
// 16), each lane holding NU units of 8 elements, 64 WPR units apart (only the
// last may lie past the row's end): the row stays in registers between its sum
// and its output, and the next row is on its way meanwhile.  With WPR = 1 each
// wave walks rows of its own, else the whole workgroup one row at a time.  w
// is copied to LDS once per workgroup, dw stays in registers until the end.
// 16384x3584 bf16: forward 42-50 us (4.9-5.8 TB/s), backward 56 us (5.3 TB/s)
// and 5 us for the last sum of dw; with w in registers and no row ahead the
// backward pass took 87 us.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// Sum over the waves of one row, the same order in each of them.
template <int WPR, typename T>
__device__ __forceinline__ T row_sum(T v, uint32_t wave) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    __shared__ T red[WPR];
    __syncthreads();  // red of the row before has been read
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += red[i];
  }
  return v;
}

// w in LDS as two planes, the first and the last four elements of each unit:
// a wave's reads of a plane are 1 KB without a gap.
struct WeightLds {
  nt_f32x4 *lo, *hi;
  __device__ __forceinline__ WeightLds(nt_f32x4* lds, uint32_t upr) : lo(lds), hi(lds + upr) {}
  __device__ __forceinline__ void fill(const float* __restrict__ w, uint32_t upr, uint32_t threads) const {
    for (uint32_t u = threadIdx.x; u < upr; u += threads) {
      lo[u] = reinterpret_cast<const nt_f32x4*>(w)[2 * u];
      hi[u] = reinterpret_cast<const nt_f32x4*>(w)[2 * u + 1];
    }
    __syncthreads();
  }
  __device__ __forceinline__ void get(uint32_t unit, uint32_t upr, float (&f)[8]) const {
    uint32_t u = unit < upr ? unit : 0;
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(u));  // read again each time: kept across rows, w would cost 8 registers a unit
#endif
    const nt_f32x4 a = lo[u], b = hi[u];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename InT, int FMT, bool CEIL, int NU, int WPR, int THREADS>
__global__ __launch_bounds__(THREADS) void rmsnorm_forward_kernel(
    const InT* __restrict__ x, int64_t ldx, int64_t rows, uint32_t upr, const float* __restrict__ w,
    float eps, uint8_t* __restrict__ y, int64_t ldy, uint8_t* __restrict__ ys, uint8_t* __restrict__ kept, int64_t ldk,
    uint8_t* __restrict__ ks, float* __restrict__ rstd) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ nt_f32x4 lds[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr uint32_t RPW = WPR == 1 ? THREADS / 64 : 1;  // rows per workgroup and round
  static_assert(WPR == 1 || THREADS == 64 * WPR, "one row per workgroup");
  const uint32_t unit0 = (WPR == 1 ? 0 : wave * 64) + lane;
  constexpr uint32_t USTEP = WPR * 64;
  const uint32_t nb = upr >> 2;
  // Lane offsets: one per tensor; the last unit's own, outside past the row's end.
  const bool last_in = unit0 + (NU - 1) * USTEP < upr;
  const uint32_t cx = unit0 * 8 * sizeof(InT), cq = unit0 * 8, cs = (lane & 3) == 0 ? unit0 >> 2 : kNowhere;
  auto at = [&](int i, uint32_t off) __attribute__((always_inline)) {
    return i < NU - 1 || last_in ? off : kNowhere;
  };
  auto load = [&](int64_t row, MxRaw<InT> (&raw)[NU]) __attribute__((always_inline)) {
    const mx_rsrc rx = mx_run(x + row * ldx);
#pragma unroll
    for (int i = 0; i < NU; ++i) mx_get(rx, at(i, cx), i * USTEP * 8 * sizeof(InT), raw[i]);
  };
  const WeightLds wl(lds, upr);
  MxRaw<InT> next[NU];
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + (WPR == 1 ? wave : 0);
  load(row < rows ? row : rows - 1, next);
  wl.fill(w, upr, THREADS);
  for (; row < rows; row += step) {
    const int64_t ahead = row + step < rows ? row + step : row;  // the last row's own again
    MxRaw<InT> raw[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) raw[i] = next[i];
    load(ahead, next);
    // Eight chains over the units, joined pair by pair, and the row's few last
    // steps in 64 bits: what r is off by moves a whole row across the casts' ties.
    float sq[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float f[8];
      mx_unpack(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[j] = __builtin_fmaf(f[j], f[j], sq[j]);
    }
    float ss = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
    ss = row_sum<WPR>(ss, wave);
#pragma unroll
    for (int i = 0; i < NU; ++i) again(raw[i]);
    double sum = ss;
    // Squares that overflow in fp32, or so few bits left that eps does not cover
    // the loss: once more in 64 bits (the same branch in all waves of the row).
    if (!(ss < __builtin_inff()) || ss + eps * (float)(upr * 8) < 0x1p-100f) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float f[8];
        mx_unpack(raw[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)f[j], (double)f[j], sum);
        again(raw[i]);
      }
      sum = row_sum<WPR>(sum, wave);
    }
    const float r = (float)(1.0 / __builtin_sqrt(sum / (double)(upr * 8) + (double)eps));
    const mx_rsrc ry = mx_run(y + row * ldy), rys = mx_run(ys + row * nb);
    const mx_rsrc rk = mx_run(kept + row * ldk), rks = mx_run(ks + row * nb);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float f[8], v[8], wf[8];
      wl.get(unit0 + i * USTEP, upr, wf);
      mx_unpack(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = f[j] * r * wf[j];
      const uint32_t sv = mx_scale<FMT, CEIL>(max_quad(absmax8(v)));
      mx_put_codes(ry, at(i, cq), i * USTEP * 8, mx_codes8<FMT, CEIL>(v, sv));
      mx_put_byte(rys, at(i, cs), i * USTEP / 4, sv);
      if (kept) {
        const uint32_t sk = mx_scale<FMT, CEIL>(max_quad(absmax8(f)));
        mx_put_codes(rk, at(i, cq), i * USTEP * 8, mx_codes8<FMT, CEIL>(f, sk));
        mx_put_byte(rks, at(i, cs), i * USTEP / 4, sk);
      }
    }
    if (kept && unit0 == 0) rstd[row] = r;
  }
#endif
}

// One row's share of a lane, as read.
template <typename T, int NU>
struct BackwardIn {
  uint2 code[NU];
  uint32_t b[NU];
  MxRaw<T> dy[NU];
  float r;
};

// part: [gridDim.x][8 upr] partial sums of dw, one row per workgroup.
template <typename T, int FMT, int NU, int WPR, int THREADS>
__global__ __launch_bounds__(THREADS) void rmsnorm_backward_kernel(
    const uint8_t* __restrict__ kept, int64_t ldk, const uint8_t* __restrict__ ks, const float* __restrict__ rstd,
    const float* __restrict__ w, const T* __restrict__ dy, int64_t lddy, int64_t rows, uint32_t upr,
    T* __restrict__ dx, int64_t lddx, float* __restrict__ part) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ nt_f32x4 lds[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr uint32_t RPW = WPR == 1 ? THREADS / 64 : 1;
  static_assert(WPR == 1 || THREADS == 64 * WPR, "one row per workgroup");
  const uint32_t unit0 = (WPR == 1 ? 0 : wave * 64) + lane;
  constexpr uint32_t USTEP = WPR * 64;
  const uint32_t nb = upr >> 2;
  const float inv_cols = 1.0f / (float)(upr * 8);
  typedef BackwardIn<T, NU> In;
  // Lane offsets: one per tensor; the last unit's own, outside past the row's end.
  const bool last_in = unit0 + (NU - 1) * USTEP < upr;
  const uint32_t ck = unit0 * 8, cd = unit0 * 8 * sizeof(T), cs = unit0 >> 2;
  auto at = [&](int i, uint32_t off) __attribute__((always_inline)) {
    return i < NU - 1 || last_in ? off : kNowhere;
  };
  auto load = [&](int64_t row, In& in) __attribute__((always_inline)) {
    const mx_rsrc rk = mx_run(kept + row * ldk), rs = mx_run(ks + row * nb), rd = mx_run(dy + row * lddy);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      in.code[i] = mx_get_codes(rk, at(i, ck), i * USTEP * 8);
      in.b[i] = mx_get_byte(rs, at(i, cs), i * USTEP / 4);
      mx_get(rd, at(i, cd), i * USTEP * 8 * sizeof(T), in.dy[i]);
    }
    in.r = rstd[row];
  };
  // A row ahead where two rows fit in the registers (16-bit dy).
  constexpr bool AHEAD = sizeof(T) == 2;
  const WeightLds wl(lds, upr);
  float dw[NU][8];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  In next;
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + (WPR == 1 ? wave : 0);
  load(row < rows ? row : rows - 1, next);
  wl.fill(w, upr, THREADS);
  for (; row < rows; row += step) {
    const int64_t ahead = row + step < rows ? row + step : row;  // the last row's own again
    In in = next;
    if constexpr (AHEAD) load(ahead, next);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float xh[8], d[8], wf[8];
      wl.get(unit0 + i * USTEP, upr, wf);
      mx_decode8<FMT>(in.code[i], mx_factor(in.b[i]) * in.r, xh);
      mx_unpack(in.dy[i], d);
      float p = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = d[j] * xh[j];
        dw[i][j] += t;
        p = __builtin_fmaf(t, wf[j], p);
      }
      dot += p;
      __builtin_amdgcn_sched_barrier(0);  // unit after unit: side by side they need every register
    }
    const float k = row_sum<WPR>(dot, wave) * inv_cols;
    const mx_rsrc rx = mx_run(dx + row * lddx);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      again(in.code[i]);
      again(in.dy[i]);
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float xh[8], d[8], wf[8];
      wl.get(unit0 + i * USTEP, upr, wf);
      mx_decode8<FMT>(in.code[i], mx_factor(in.b[i]) * in.r, xh);
      mx_unpack(in.dy[i], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = in.r * __builtin_fmaf(xh[j], -k, d[j] * wf[j]);
      mx_put8(rx, at(i, cd), i * USTEP * 8 * sizeof(T), d, T());
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!AHEAD) load(ahead, next);
  }
  // The workgroup's rows, one group of waves after the other, into LDS (w is
  // not needed any more) and out: the same sum on every run.
  __syncthreads();
  for (uint32_t turn = 0; turn < RPW; ++turn) {
    if (WPR > 1 || wave == turn) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const uint32_t unit = unit0 + i * USTEP;
        if (unit < upr) {
          const nt_f32x4 a = {dw[i][0], dw[i][1], dw[i][2], dw[i][3]}, b = {dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
          wl.lo[unit] = turn ? wl.lo[unit] + a : a;
          wl.hi[unit] = turn ? wl.hi[unit] + b : b;
        }
      }
    }
    __syncthreads();
  }
  nt_f32x4* out = reinterpret_cast<nt_f32x4*>(part + (int64_t)blockIdx.x * (upr * 8));
  for (uint32_t u = threadIdx.x; u < upr; u += THREADS) {
    out[2 * u] = wl.lo[u];
    out[2 * u + 1] = wl.hi[u];
  }
#endif
}

// dw[c] = sum of part[p][c]: 16 waves take every 16th row, in order, then add
// up in order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ part, uint32_t parts, uint32_t cols,
                                                          float* __restrict__ dw) {
  __shared__ float sum[16][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (uint32_t p = wave; p < parts; p += 16) s += part[(int64_t)p * cols + c];
  }
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][lane];
    dw[c] = t;
  }
}

// Waves per row and units per lane.
struct NormShape {
  int wpr, nu;
};
NormShape norm_shape(int64_t cols) {
  const int upr = (int)(cols / kLaneElems);
  NormShape n;
  n.wpr = upr <= 512 ? 1 : upr <= 2048 ? 4 : 16;
  n.nu = (upr + 64 * n.wpr - 1) / (64 * n.wpr);
  return n;
}
// Workgroups for the rows, at rpw rows a round, at most cap.
uint32_t norm_blocks(int64_t rows, int64_t rpw, int64_t cap) {
  const int64_t b = (rows + rpw - 1) / rpw;
  return (uint32_t)(b < cap ? b : cap);
}
// Waves of a workgroup with WPR = 1.  Backward: 8, all that a compute unit
// takes at two per SIMD, so that there is one row of partial sums per compute
// unit.
constexpr int kForwardWaves = 4, kBackwardWaves = 8;

template <typename InT, int FMT, bool CEIL, bool KEEP>
void swiglu_forward(const void* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* h, int64_t ldh, uint8_t* hs,
                    uint8_t* kept, int64_t ldk, uint8_t* ks, hipStream_t stream) {
  const uint32_t upr = (uint32_t)(cols / kLaneElems);
  const bool deep = rows * upr >= (int64_t)kThreads * kForwardUnits * 4 * device_cus();
  const int u = deep ? kForwardUnits : 1;
  const int64_t items = rows * ((upr + 64 * u - 1) / (64 * u)), need = (items + 3) / 4;
  const uint32_t blocks = (uint32_t)(need < kForwardBlocks ? need : kForwardBlocks);
#define MXFP8_SF(U, NT)                                                                                          \
  hipLaunchKernelGGL((swiglu_forward_kernel<InT, FMT, CEIL, KEEP, U, NT>), dim3(blocks), dim3(kThreads), 0, stream, \
                     static_cast<const InT*>(x), ldx, rows, upr, h, ldh, hs, kept, ldk, ks)
  if (!deep) MXFP8_SF(1, false);
  else if (stream_loads(rows, 2 * cols, sizeof(InT))) MXFP8_SF(kForwardUnits, true);
  else MXFP8_SF(kForwardUnits, false);
#undef MXFP8_SF
}

template <typename T, int FMT>
void swiglu_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const void* dh, int64_t lddh, int64_t rows,
                     int64_t cols, void* dx, int64_t lddx, hipStream_t stream) {
  const uint32_t upr = (uint32_t)(cols / kLaneElems);
  const int64_t items = rows * ((upr + 63) / 64), need = (items + 3) / 4;
  const uint32_t blocks = (uint32_t)(need < kBackwardBlocks ? need : kBackwardBlocks);
#define MXFP8_SB(NT)                                                                                              \
  hipLaunchKernelGGL((swiglu_backward_kernel<T, FMT, NT>), dim3(blocks), dim3(kThreads), 0, stream, kept, ldk, ks, \
                     static_cast<const T*>(dh), lddh, rows, upr, static_cast<T*>(dx), lddx)
  if (stream_loads(rows, cols, sizeof(T))) MXFP8_SB(true);
  else MXFP8_SB(false);
#undef MXFP8_SB
}

template <typename InT, int FMT, bool CEIL>
void rmsnorm_forward(const void* x, int64_t rows, int64_t cols, int64_t ldx, const float* w, float eps, uint8_t* y,
                     int64_t ldy, uint8_t* ys, uint8_t* kept, int64_t ldk, uint8_t* ks, float* rstd,
                     hipStream_t stream) {
  const NormShape n = norm_shape(cols);
#define MXFP8_NF(WPR, NU, WAVES)                                                                                    \
  case NU:                                                                                                          \
    hipLaunchKernelGGL((rmsnorm_forward_kernel<InT, FMT, CEIL, NU, WPR, 64 * WAVES>),                               \
                       dim3(norm_blocks(rows, WAVES / WPR, 1024)), dim3(64 * WAVES), (uint32_t)cols * 4, stream,    \
                       static_cast<const InT*>(x), ldx, rows, (uint32_t)(cols / kLaneElems), w, eps, y, ldy, ys,    \
                       kept, ldk, ks, rstd);                                                                        \
    break;
  if (n.wpr == 1) {
    switch (n.nu) {
      MXFP8_NF(1, 1, kForwardWaves) MXFP8_NF(1, 2, kForwardWaves) MXFP8_NF(1, 3, kForwardWaves)
      MXFP8_NF(1, 4, kForwardWaves) MXFP8_NF(1, 5, kForwardWaves) MXFP8_NF(1, 6, kForwardWaves)
      MXFP8_NF(1, 7, kForwardWaves) MXFP8_NF(1, 8, kForwardWaves)
    }
  } else if (n.wpr == 4) {
    switch (n.nu) {
      MXFP8_NF(4, 3, 4) MXFP8_NF(4, 4, 4) MXFP8_NF(4, 5, 4) MXFP8_NF(4, 6, 4) MXFP8_NF(4, 7, 4) MXFP8_NF(4, 8, 4)
    }
  } else {
    switch (n.nu) { MXFP8_NF(16, 3, 16) MXFP8_NF(16, 4, 16) }
  }
#undef MXFP8_NF
}

template <typename T, int FMT>
void rmsnorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, const float* w,
                      const void* dy, int64_t lddy, int64_t rows, int64_t cols, void* dx, int64_t lddx, float* part,
                      int64_t parts, hipStream_t stream) {
  const NormShape n = norm_shape(cols);
#define MXFP8_NB(WPR, NU, WAVES)                                                                                   \
  case NU:                                                                                                         \
    hipLaunchKernelGGL((rmsnorm_backward_kernel<T, FMT, NU, WPR, 64 * WAVES>), dim3((uint32_t)parts),              \
                       dim3(64 * WAVES), (uint32_t)cols * 4, stream, kept, ldk, ks, rstd, w,                       \
                       static_cast<const T*>(dy), lddy, rows, (uint32_t)(cols / kLaneElems), static_cast<T*>(dx),  \
                       lddx, part);                                                                                \
    break;
  if (n.wpr == 1) {
    switch (n.nu) {
      MXFP8_NB(1, 1, kBackwardWaves) MXFP8_NB(1, 2, kBackwardWaves) MXFP8_NB(1, 3, kBackwardWaves)
      MXFP8_NB(1, 4, kBackwardWaves) MXFP8_NB(1, 5, kBackwardWaves) MXFP8_NB(1, 6, kBackwardWaves)
      MXFP8_NB(1, 7, kBackwardWaves) MXFP8_NB(1, 8, kBackwardWaves)
    }
  } else if (n.wpr == 4) {
    switch (n.nu) {
      MXFP8_NB(4, 3, 4) MXFP8_NB(4, 4, 4) MXFP8_NB(4, 5, 4) MXFP8_NB(4, 6, 4) MXFP8_NB(4, 7, 4) MXFP8_NB(4, 8, 4)
    }
  } else {
    switch (n.nu) { MXFP8_NB(16, 3, 16) MXFP8_NB(16, 4, 16) }
  }
#undef MXFP8_NB
}

}  // namespace mx_act_detail

using namespace mx_act_detail;

void launch_mx_swiglu_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int rule,
                              uint8_t* h, int64_t ldh, uint8_t* hs, uint8_t* kept, int64_t ldk, uint8_t* ks,
                              hipStream_t stream) {
#define MXFP8_K(T, FMT, CEIL)                                                                             \
  (kept ? swiglu_forward<T, FMT, CEIL, true>(x, rows, cols, ldx, h, ldh, hs, kept, ldk, ks, stream)       \
        : swiglu_forward<T, FMT, CEIL, false>(x, rows, cols, ldx, h, ldh, hs, nullptr, 0, nullptr, stream))
#define MXFP8_R(T, FMT) (rule == 0 ? MXFP8_K(T, FMT, true) : MXFP8_K(T, FMT, false))
  if (dtype == 0) fmt == 0 ? MXFP8_R(float, 0) : MXFP8_R(float, 1);
  else fmt == 0 ? MXFP8_R(uint16_t, 0) : MXFP8_R(uint16_t, 1);
#undef MXFP8_R
#undef MXFP8_K
}

void launch_mx_swiglu_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, int fmt, const void* dh, int dtype,
                               int64_t lddh, int64_t rows, int64_t cols, void* dx, int64_t lddx, hipStream_t stream) {
#define MXFP8_B(T, FMT) swiglu_backward<T, FMT>(kept, ldk, ks, dh, lddh, rows, cols, dx, lddx, stream)
  if (dtype == 0) fmt == 0 ? MXFP8_B(float, 0) : MXFP8_B(float, 1);
  else fmt == 0 ? MXFP8_B(uint16_t, 0) : MXFP8_B(uint16_t, 1);
#undef MXFP8_B
}

void launch_mx_rmsnorm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w,
                               float eps, int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* ys, uint8_t* kept,
                               int64_t ldk, uint8_t* ks, float* rstd, hipStream_t stream) {
#define MXFP8_R(T, FMT)                                                                                          \
  (rule == 0                                                                                                     \
       ? rmsnorm_forward<T, FMT, true>(x, rows, cols, ldx, w, eps, y, ldy, ys, kept, ldk, ks, rstd, stream)      \
       : rmsnorm_forward<T, FMT, false>(x, rows, cols, ldx, w, eps, y, ldy, ys, kept, ldk, ks, rstd, stream))
  if (dtype == 0) fmt == 0 ? MXFP8_R(float, 0) : MXFP8_R(float, 1);
  else fmt == 0 ? MXFP8_R(uint16_t, 0) : MXFP8_R(uint16_t, 1);
#undef MXFP8_R
}

int64_t rmsnorm_backward_parts(int64_t rows, int64_t cols) {
  const NormShape n = norm_shape(cols);
  return norm_blocks(rows, n.wpr == 1 ? kBackwardWaves : 1, n.wpr == 4 ? 512 : 256);
}

void launch_mx_rmsnorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, int fmt,
                                const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols,
                                void* dx, int64_t lddx, float* dw, float* workspace, int64_t parts,
                                hipStream_t stream) {
  if (rows > 0) {
#define MXFP8_B(T, FMT) \
  rmsnorm_backward<T, FMT>(kept, ldk, ks, rstd, w, dy, lddy, rows, cols, dx, lddx, workspace, parts, stream)
  if (dtype == 0) fmt == 0 ? MXFP8_B(float, 0) : MXFP8_B(float, 1);
  else fmt == 0 ? MXFP8_B(uint16_t, 0) : MXFP8_B(uint16_t, 1);
#undef MXFP8_B
  }
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((uint32_t)((cols + 63) / 64)), dim3(1024), 0, stream, workspace,
                     (uint32_t)parts, (uint32_t)cols, dw);
}

}  // namespace mxfp8
