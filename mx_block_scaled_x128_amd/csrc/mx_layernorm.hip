// mx_layernorm.hip -- LayerNorm with MX codes out and its normalised input kept
// in 8 bits for the backward pass (gfx950).
//
// Forward, per row of x:  mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//   xh = (x - mu) * r,  y = xh * w + b.
// y leaves as MX codes; xh (not x: a row's offset would use up the eight bits)
// is kept as MX codes, with r.
// Backward, on the kept xh:  c = dy * w,
//   dx = r * (c - mean(c) - xh * mean(c * xh)),
//   dw = sum over rows of dy * xh,  db = sum over rows of dy.
//
// The mean is taken twice: m0 from the sum of x, and the mean of x - m0, which
// is what m0's rounding left; the squares are of x - m0, exact where x lies
// near m0.  So a row far from zero loses nothing but what its own type lost.
// Arithmetic is in fp32, the root the hardware's and one Newton step; rows whose
// squares leave fp32's range, or of whose variance m0's rounding is a sixteenth or
// more, are scaled by a power of two and taken in 64 bits.
//
// A workgroup works on RB rows at a time, as many waves as a row has units of
// 8 elements (up to 16 waves; then 2 or 4 units to a lane), with the next RB
// rows on their way.  A lane keeps its columns, so w, b, and the backward
// pass's sums dw and db stay in its registers.  Each tensor is read and written
// once: HBM bounds both passes.  16384x3584 bf16, kept: forward 57 us (238 MB, 4.2
// TB/s of the 5.1 that a copy reaches; the rest is instructions, two casts and
// three passes over the registers), backward 59 and 4.7 for the sums (293 MB, 5.0
// TB/s).  515x8960 fp32 backward 16 us (42 MB): 256 workgroups that take two or
// three rows one after the other, the latency of each row's reads and its sums.
#include "mx_common.hpp"
#include "mx_launch.hpp"

namespace mxfp8 {

namespace mx_layernorm_detail {

#if defined(__HIP_DEVICE_COMPILE__)
// The largest |f|, NaN if one is: absmax8 in 4 instructions.
__device__ __forceinline__ uint32_t largest8(const float (&f)[8]) {
  float m;
  asm("v_maximum3_f32 %0, |%1|, |%2|, |%3|" : "=v"(m) : "v"(f[0]), "v"(f[1]), "v"(f[2]));
  asm("v_maximum3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(f[3]), "v"(f[4]));
  asm("v_maximum3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(f[5]), "v"(f[6]));
  asm("v_maximum3_f32 %0, %0, |%1|, |%1|" : "+v"(m) : "v"(f[7]));
  return __float_as_uint(m);
}
// Sum of eight elements as read.
__device__ __forceinline__ float sum8(const MxRaw<float>& r) {
  return ((r.a.x + r.a.y) + (r.a.z + r.a.w)) + ((r.b.x + r.b.y) + (r.b.z + r.b.w));
}
__device__ __forceinline__ float sum8(const MxRaw<uint16_t>& r) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 one = {(__bf16)1.0f, (__bf16)1.0f};
  float s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, r.v.x), one, 0.0f, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, r.v.y), one, s, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, r.v.z), one, s, false);
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, r.v.w), one, s, false);
}

// LDS written before is read after, by all waves; loads from memory stay in flight.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// N sums over the workgroup at once, uniform in every lane.  red has two
// buffers of N sums of up to 16 waves, used in turn: a buffer is written again
// only after everybody has met once more.
constexpr int kSums = 8;
struct Reduce {
  float* red;  // [2][kSums][16]
  int waves, wave, lane, turn;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= kSums, "sums");
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = sum64(v[n]);
    if (waves > 1) {
      float* to = red + turn * kSums * 16;
      turn ^= 1;
      if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) to[n * 16 + wave] = v[n];
      }
      meet();
      // a sum to each row of 16 lanes
#pragma unroll
      for (int n = 0; n < N; n += 4) {
        const int mine = n + (lane >> 4);
        const float s = sum16(mine < N && (lane & 15) < waves ? to[mine * 16 + (lane & 15)] : 0.0f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < N) v[n + k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), 16 * k));
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v[n])));
  }
};
#endif

// One value over the workgroup, in 64 bits: the sum, or the largest.  `red`: 16 doubles.
template <bool MAX>
__device__ __forceinline__ double row64(double v, double* red, int waves, int wave, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double o = __shfl_xor(v, m);
    v = MAX ? (v > o ? v : o) : v + o;
  }
  __syncthreads();
  if (lane == 0) red[wave] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < waves; ++i) v = MAX ? (v > red[i] ? v : red[i]) : v + red[i];
  return v;
}

#if defined(__HIP_DEVICE_COMPILE__)
// Eight elements of w or b: kept in registers with one unit to a lane, else
// read (from the caches) each time they are used.
__device__ __forceinline__ void vector8(const float* p, uint32_t lane, uint32_t off, float (&f)[8]) {
  asm volatile("" : "+v"(lane));  // not moved out of the loop over rows
  MxRaw<float> v;
  mx_get(mx_run(p), lane, off, v);
  mx_unpack(v, f);
}
#endif

template <typename InT, int NU>
__device__ __forceinline__ void words_again(MxRaw<InT> (&raw)[NU]) {
#pragma unroll
  for (int i = 0; i < NU; ++i) again(raw[i]);
}

template <typename InT, int FMT, bool CEIL, int NU, int RB>
__global__ __launch_bounds__(1024) void forward_kernel(
    const InT* __restrict__ x, int64_t ldx, int64_t rows, uint32_t upr, const float* __restrict__ w,
    const float* __restrict__ b, float eps, uint8_t* __restrict__ y, int64_t ldy, uint8_t* __restrict__ ys,
    uint8_t* __restrict__ kept, int64_t ldk, uint8_t* __restrict__ ks, float* __restrict__ rstd) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float red[2 * kSums * 16];
  __shared__ double wide[16];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const uint32_t unit0 = wave * 64 + lane, ustep = waves * 64, nb = upr >> 2;
  Reduce reduce{red, (int)waves, (int)wave, (int)lane, 0};
  // Lane offsets: one per tensor; the last unit's own, outside past the row's
  // end, and outside in rows past the last.
  const bool last_in = unit0 + (NU - 1) * ustep < upr;
  const uint32_t cx = unit0 * 8 * sizeof(InT), cq = unit0 * 8, cs = (lane & 3) == 0 ? unit0 >> 2 : kNowhere;
  auto at = [&](int i, bool in, uint32_t off) __attribute__((always_inline)) {
    return in && (i < NU - 1 || last_in) ? off : kNowhere;
  };
  auto load = [&](int64_t row0, MxRaw<InT> (&raw)[RB][NU]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const bool in = row0 + k < rows;
      const mx_rsrc rx = mx_run(x + (in ? row0 + k : 0) * ldx);
#pragma unroll
      for (int i = 0; i < NU; ++i) mx_get(rx, at(i, in, cx), i * ustep * 8 * (uint32_t)sizeof(InT), raw[k][i]);
    }
  };
  // Units past the row's end: zeros in the sums of x; the differences are masked.
  constexpr bool AHEAD = NU <= 2;
  MxRaw<InT> raw[RB][NU];
  const int64_t step = (int64_t)gridDim.x * RB;
  int64_t row0 = (int64_t)blockIdx.x * RB;
  load(row0, raw);
  constexpr bool KEEP_W = NU == 1;
  auto affine = [&](int i, float (&wf)[8], float (&bf)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) wf[j] = 1.0f, bf[j] = 0.0f;
    if (w) vector8(w, at(i, true, unit0 * 32), i * ustep * 32, wf);
    if (b) vector8(b, at(i, true, unit0 * 32), i * ustep * 32, bf);
  };
  float wk[8], bk[8];
  if constexpr (KEEP_W) affine(0, wk, bk);
  const double n = (double)(upr * 8);
  const float inv_n = (float)(1.0 / n), inv_n_low = (float)(1.0 / n - (double)inv_n);
  for (; row0 < rows; row0 += step) {
    MxRaw<InT> next[RB][NU];
    if constexpr (AHEAD) load(row0 + step, next);
    float s1[RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      s1[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < NU; ++i) s1[k] += sum8(raw[k][i]);
    }
    reduce(s1);
    float m0[RB], e[2 * RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      words_again(raw[k]);
      // One rounded m0 for both uses: as a product, it would be contracted into
      // each difference, which then would round differences of its own.  Sixteen
      // bits of it where x has eight: so nearly all differences are exact.
      m0[k] = s1[k] * inv_n;
      if constexpr (sizeof(InT) == 2) m0[k] = __uint_as_float((__float_as_uint(m0[k]) + 0x80u) & 0xFFFFFF00u);
      asm volatile("" : "+v"(m0[k]));
      e[2 * k] = 0.0f, e[2 * k + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float f[8], a = 0.0f, q = 0.0f;
        mx_unpack(raw[k][i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = f[j] - m0[k];
          a += d;
          q = __builtin_fmaf(d, d, q);
        }
        const bool in = i < NU - 1 || last_in;
        e[2 * k] += in ? a : 0.0f;
        e[2 * k + 1] += in ? q : 0.0f;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    reduce(e);
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      words_again(raw[k]);
      const int64_t row = row0 + k;
      const bool in = row < rows;
      const mx_rsrc ry = mx_run(y + row * ldy), rys = mx_run(ys + row * nb);
      const mx_rsrc rk = mx_run(kept + row * ldk), rks = mx_run(ks + row * nb);
      // 1 / n in two parts and one Newton step with its own rounding error behind
      // the hardware's root (1 ulp): r is the nearest fp32 value or the next to
      // what the variance gives.  What r is off by moves a whole row across the
      // casts' ties.  (The same in 64 bits, in every wave of a row: 16384x3584
      // bf16 75 us in place of 60.)
      const float delta = __builtin_fmaf(e[2 * k], inv_n, e[2 * k] * inv_n_low);
      const float var = __builtin_fmaf(e[2 * k + 1], inv_n,
                                       __builtin_fmaf(e[2 * k + 1], inv_n_low, __builtin_fmaf(-delta, delta, eps)));
      float r = __builtin_amdgcn_rsqf(var);
      {
        const float t = var * r, low = __builtin_fmaf(var, r, -t);
        r = __builtin_fmaf(r * 0.5f, __builtin_fmaf(-t, r, 1.0f) - low * r, r);
      }
      const float shift = -delta * r;
      // Squares that overflow in fp32 or vanish there, an eps that takes the
      // variance out of its range, or a row so nearly of equal
      // values that m0's rounding is a good part of them, a sixteenth and more, and
      // eps does not cover that: what is left when delta^2 is taken out would have
      // lost the bits that cancel.  The row scaled by a power of two, once more in
      // 64 bits (the same branch in all waves).
      double mean = 0.0, rr = 0.0;
      float scale = 0.0f;
      if (in && (!(var > 0.9375f * e[2 * k + 1] * inv_n && var < 0x1p127f) || e[2 * k + 1] + eps * (float)(upr * 8) < 0x1p-100f)) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          float f[8];
          mx_unpack(raw[k][i], f);
          top = max(top, absmax8(f));
        }
        top = (uint32_t)row64<true>((double)top, wide, waves, wave, lane);
        // 2^-e for the largest |x| in [2^e, 2^(e+1)); NaN and infinities stay what they are
        const int ex = (int)(top >> 23) - 127;
        scale = ldexpf(1.0f, -(ex < -126 ? -126 : ex > 126 ? 126 : ex));
        double sum = 0.0, sq = 0.0;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          float f[8];
          mx_unpack(raw[k][i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += (double)(f[j] * scale);
        }
        mean = row64<false>(sum, wide, waves, wave, lane) / n;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          float f[8];
          mx_unpack(raw[k][i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double d = (double)(f[j] * scale) - mean;
            if (i < NU - 1 || last_in) sq = __builtin_fma(d, d, sq);
          }
        }
        sq = row64<false>(sq, wide, waves, wave, lane);
        rr = 1.0 / __builtin_sqrt(sq / n + (double)eps * (double)scale * (double)scale);
        r = (float)(rr * (double)scale);
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float f[8], v[8];
        mx_unpack(raw[k][i], f);
        if (scale == 0.0f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j] - m0[k], r, shift);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = (float)(((double)(f[j] * scale) - mean) * rr);
        }
        float wl[8], bl[8];
        if constexpr (!KEEP_W) affine(i, wl, bl);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(f[j], KEEP_W ? wk[j] : wl[j], KEEP_W ? bk[j] : bl[j]);
        const uint32_t sv = mx_scale<FMT, CEIL>(max_quad(largest8(v)));
        mx_put_codes(ry, at(i, in, cq), i * ustep * 8, mx_codes8<FMT, CEIL>(v, sv));
        mx_put_byte(rys, at(i, in, cs), i * ustep / 4, sv);
        if (kept) {
          const uint32_t sk = mx_scale<FMT, CEIL>(max_quad(largest8(f)));
          mx_put_codes(rk, at(i, in, cq), i * ustep * 8, mx_codes8<FMT, CEIL>(f, sk));
          mx_put_byte(rks, at(i, in, cs), i * ustep / 4, sk);
        }
      }
      if (kept && in && threadIdx.x == 0) rstd[row] = r;
      __builtin_amdgcn_sched_barrier(0);  // row after row: side by side they need every register
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int i = 0; i < NU; ++i) raw[k][i] = next[k][i];
    } else {
      load(row0 + step, raw);
    }
  }
#endif
}

// Rows of a batch as read by a lane.
template <typename T, int NU, int RB>
struct BackwardIn {
  uint2 code[RB][NU];
  uint32_t b[RB][NU];
  MxRaw<T> dy[RB][NU];
  float r[RB];
};

// part: [gridDim.x][2][8 upr] partial sums of dw and of db; null: none are wanted.
template <typename T, int FMT, int NU, int RB>
__global__ __launch_bounds__(1024) void backward_kernel(const uint8_t* __restrict__ kept, int64_t ldk,
                                                        const uint8_t* __restrict__ ks, const float* __restrict__ rstd,
                                                        const float* __restrict__ w, const T* __restrict__ dy,
                                                        int64_t lddy, int64_t rows, uint32_t upr, T* __restrict__ dx,
                                                        int64_t lddx, float* __restrict__ part) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float red[2 * kSums * 16];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const uint32_t unit0 = wave * 64 + lane, ustep = waves * 64, nb = upr >> 2;
  Reduce reduce{red, (int)waves, (int)wave, (int)lane, 0};
  typedef BackwardIn<T, NU, RB> In;
  const bool last_in = unit0 + (NU - 1) * ustep < upr;
  const uint32_t ck = unit0 * 8, cd = unit0 * 8 * sizeof(T), cs = unit0 >> 2;
  auto at = [&](int i, bool in, uint32_t off) __attribute__((always_inline)) {
    return in && (i < NU - 1 || last_in) ? off : kNowhere;
  };
  // Rows and units past the end read as zero codes, scales and gradients: they add nothing.
  auto load = [&](int64_t row0, In& v) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const bool in = row0 + k < rows;
      const int64_t row = in ? row0 + k : 0;
      const mx_rsrc rk = mx_run(kept + row * ldk), rs = mx_run(ks + row * nb), rd = mx_run(dy + row * lddy);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        v.code[k][i] = mx_get_codes(rk, at(i, in, ck), i * ustep * 8);
        v.b[k][i] = mx_get_byte(rs, at(i, in, cs), i * ustep / 4);
        mx_get(rd, at(i, in, cd), i * ustep * 8 * (uint32_t)sizeof(T), v.dy[k][i]);
      }
      v.r[k] = rstd[row];
    }
  };
  constexpr bool AHEAD = NU <= 2, KEEP_W = NU == 1;
  float dw[NU][8], db[NU][8], wk[8];
  auto weights = [&](int i, float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.0f;
    if (w) vector8(w, at(i, true, unit0 * 32), i * ustep * 32, f);
  };
  if constexpr (KEEP_W) weights(0, wk);
#pragma unroll
  for (int i = 0; i < NU; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f, db[i][j] = 0.0f;
  }
  const float inv_n = (float)(1.0 / (double)(upr * 8));
  const int64_t step = (int64_t)gridDim.x * RB;
  int64_t row0 = (int64_t)blockIdx.x * RB;
  In v;
  load(row0, v);
  for (; row0 < rows; row0 += step) {
    In next;
    if constexpr (AHEAD) load(row0 + step, next);
    float s[2 * RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      s[2 * k] = 0.0f, s[2 * k + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float xh[8], d[8], wl[8];
        if constexpr (!KEEP_W) weights(i, wl);
        mx_decode8<FMT>(v.code[k][i], mx_factor(v.b[k][i]), xh);
        mx_unpack(v.dy[k][i], d);
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = d[j] * xh[j], wj = KEEP_W ? wk[j] : wl[j];
          dw[i][j] += t;
          db[i][j] += d[j];
          p = __builtin_fmaf(d[j], wj, p);
          q = __builtin_fmaf(t, wj, q);
        }
        s[2 * k] += p;
        s[2 * k + 1] += q;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    reduce(s);
#pragma unroll
    for (int k = 0; k < RB; ++k) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        again(v.code[k][i]);
        again(v.dy[k][i]);
      }
      const int64_t row = row0 + k;
      const bool in = row < rows;
      const mx_rsrc rx = mx_run(dx + row * lddx);
      const float mc = s[2 * k] * inv_n, mx = s[2 * k + 1] * inv_n;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float xh[8], d[8], wl[8];
        if constexpr (!KEEP_W) weights(i, wl);
        mx_decode8<FMT>(v.code[k][i], mx_factor(v.b[k][i]), xh);
        mx_unpack(v.dy[k][i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wj = KEEP_W ? wk[j] : wl[j];
          d[j] = v.r[k] * __builtin_fmaf(xh[j], -mx, __builtin_fmaf(d[j], wj, -mc));
        }
        mx_put8(rx, at(i, in, cd), i * ustep * 8 * (uint32_t)sizeof(T), d, T());
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (AHEAD) v = next;
    else load(row0 + step, v);
  }
  if (part) {
    const mx_rsrc rw = mx_run(part + (int64_t)blockIdx.x * (upr * 16)), rb = mx_run(part + (int64_t)blockIdx.x * (upr * 16) + upr * 8);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      mx_put8(rw, at(i, true, unit0 * 32), i * ustep * 32, dw[i], 0.0f);
      mx_put8(rb, at(i, true, unit0 * 32), i * ustep * 32, db[i], 0.0f);
    }
  }
#endif
}

// dw and db: the sums of their columns of part, 16 waves taking every 16th row
// in order, then added up in order.
__global__ __launch_bounds__(1024) void weight_sum_kernel(const float* __restrict__ part, uint32_t parts, uint32_t cols,
                                                          float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sum[16][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < 2 * cols) {
#pragma unroll 8
    for (uint32_t p = wave; p < parts; p += 16) s += part[(int64_t)p * (2 * cols) + c];
  }
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < 2 * cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][lane];
    if (c < cols) dw[c] = t;
    else db[c - cols] = t;
  }
}

// Units per lane, waves per row (all of a workgroup's).
struct Shape {
  int nu, waves;
};
Shape shape(int64_t cols) {
  const int upr = (int)(cols / kLaneElems);
  Shape s;
  s.nu = upr <= 1024 ? 1 : upr <= 2048 ? 2 : 4;
  s.waves = (upr + 64 * s.nu - 1) / (64 * s.nu);
  return s;
}
// Rows of a batch, whose sums share the waits for them, as many as 128 registers
// hold: forward 16384x3584 bf16 55 us with 4, 57 with 2, 63 with 1; 8192x3584 fp32
// 32 with 2 or 1, 70 with 4 (spills).  Backward bf16 59 with 2, 62 with 1, 157
// with 4; 8192x3584 fp32 53 with 1, 56 with 2.
template <typename T>
constexpr int forward_batch() {
  return sizeof(T) == 2 ? 4 : 2;
}
template <typename T>
constexpr int backward_batch(int nu) {
  return nu == 1 && sizeof(T) == 2 ? 2 : 1;
}
// Workgroups: up to 16 waves to each of 256 compute units, whatever the device has
// (the size of the backward pass's workspace goes by it).  Half as many: forward
// 16384x3584 bf16 65 us in place of 54; twice as many 56, backward 67 in place of 59.
int64_t most_groups(int waves) { return 256 * (16 / waves > 1 ? 16 / waves : 1); }
int64_t groups(int64_t rows, int rb, int waves) {
  const int64_t need = (rows + rb - 1) / rb, most = most_groups(waves);
  return need < most ? need : most;
}

template <typename InT, int FMT, bool CEIL>
void forward(const void* x, int64_t rows, int64_t cols, int64_t ldx, const float* w, const float* b, float eps,
             uint8_t* y, int64_t ldy, uint8_t* ys, uint8_t* kept, int64_t ldk, uint8_t* ks, float* rstd,
             hipStream_t stream) {
  const Shape s = shape(cols);
#define MXFP8_F(NU, RB)                                                                                           \
  hipLaunchKernelGGL((forward_kernel<InT, FMT, CEIL, NU, RB>), dim3((uint32_t)groups(rows, RB, s.waves)),         \
                     dim3(64 * s.waves), 0, stream, static_cast<const InT*>(x), ldx, rows,                        \
                     (uint32_t)(cols / kLaneElems), w, b, eps, y, ldy, ys, kept, ldk, ks, rstd)
  // While each row can have a workgroup, a batch would only lengthen it: 1x3584 bf16 3.0 us, with 4 5.5.
  if (s.nu == 1 && rows <= most_groups(s.waves)) MXFP8_F(1, 1);
  else if (s.nu == 1) MXFP8_F(1, forward_batch<InT>());
  else if (s.nu == 2) MXFP8_F(2, 1);
  else MXFP8_F(4, 1);
#undef MXFP8_F
}

template <typename T, int FMT>
void backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, const float* w, const void* dy,
              int64_t lddy, int64_t rows, int64_t cols, void* dx, int64_t lddx, float* part, int64_t parts,
              hipStream_t stream) {
  const Shape s = shape(cols);
#define MXFP8_B(NU)                                                                                                   \
  hipLaunchKernelGGL((backward_kernel<T, FMT, NU, backward_batch<T>(NU)>), dim3((uint32_t)parts), dim3(64 * s.waves), 0,       \
                     stream, kept, ldk, ks, rstd, w, static_cast<const T*>(dy), lddy, rows,                           \
                     (uint32_t)(cols / kLaneElems), static_cast<T*>(dx), lddx, part)
  if (s.nu == 1) MXFP8_B(1);
  else if (s.nu == 2) MXFP8_B(2);
  else MXFP8_B(4);
#undef MXFP8_B
}

}  // namespace mx_layernorm_detail

using namespace mx_layernorm_detail;

void launch_mx_layernorm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const float* w,
                                 const float* b, float eps, int fmt, int rule, uint8_t* y, int64_t ldy, uint8_t* ys,
                                 uint8_t* kept, int64_t ldk, uint8_t* ks, float* rstd, hipStream_t stream) {
#define MXFP8_R(T, FMT)                                                                                         \
  (rule == 0 ? forward<T, FMT, true>(x, rows, cols, ldx, w, b, eps, y, ldy, ys, kept, ldk, ks, rstd, stream)    \
             : forward<T, FMT, false>(x, rows, cols, ldx, w, b, eps, y, ldy, ys, kept, ldk, ks, rstd, stream))
  if (dtype == 0) fmt == 0 ? MXFP8_R(float, 0) : MXFP8_R(float, 1);
  else fmt == 0 ? MXFP8_R(uint16_t, 0) : MXFP8_R(uint16_t, 1);
#undef MXFP8_R
}

int64_t layernorm_backward_parts(int64_t rows, int64_t cols) {
  const Shape s = shape(cols);
  return groups(rows, backward_batch<uint16_t>(s.nu), s.waves);
}

void launch_mx_layernorm_backward(const uint8_t* kept, int64_t ldk, const uint8_t* ks, const float* rstd, int fmt,
                                  const float* w, const void* dy, int dtype, int64_t lddy, int64_t rows, int64_t cols,
                                  void* dx, int64_t lddx, float* dw, float* db, float* workspace, hipStream_t stream) {
  const int64_t parts = layernorm_backward_parts(rows, cols);
  float* part = dw ? workspace : nullptr;
  if (rows > 0) {
#define MXFP8_B(T, FMT) \
  backward<T, FMT>(kept, ldk, ks, rstd, w, dy, lddy, rows, cols, dx, lddx, part, parts, stream)
    if (dtype == 0) fmt == 0 ? MXFP8_B(float, 0) : MXFP8_B(float, 1);
    else fmt == 0 ? MXFP8_B(uint16_t, 0) : MXFP8_B(uint16_t, 1);
#undef MXFP8_B
  }
  if (dw)
    hipLaunchKernelGGL(weight_sum_kernel, dim3((uint32_t)((2 * cols + 63) / 64)), dim3(1024), 0, stream, workspace,
                       (uint32_t)parts, (uint32_t)cols, dw, db);
}

}  // namespace mxfp8
