// mx_common.hpp -- device helpers of the MX operators (32-element blocks with
// one E8M0 scale): the E2M1 format next to E4M3 and E5M2, block exponents
// under both rules, the casts with the scale already divided out, and the way
// back from codes to values.
//
// E2M1 [OCP MX element format]: bias 1, no infinities or NaN, magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6; largest finite value 6 = 1.5 * 2^2.  Two codes
// to a byte, the even element in the low four bits.
//
// Non-finite input.  A block that holds an infinity or a NaN gets the scale
// byte 255 (E8M0's NaN) and zero codes; every reader (mx_unscale here, the
// matrix cores in the products) turns its elements into NaN.  The largest
// |x| as an integer finds both: the patterns of inf and NaN are above every
// finite one.
#pragma once

#include "device_common.hpp"

namespace mxfp8 {

constexpr int kE2M1 = 2;
constexpr uint32_t kInfBits = 0x7F800000u;

// Elements per lane of the row-wise kernels: 8 (16 bytes of bf16, 8 of FP8
// codes, 4 of E2M1 codes); 4 lanes, a DPP quad, share one MX block.
constexpr int kLaneElems = 8;

template <int FMT> struct MxFmt {
  static constexpr int q = FmtInfo<FMT>::q;
  static constexpr float fmax = FmtInfo<FMT>::fmax;
  static constexpr uint32_t frac_max = 0x600000u;  // fmax = 1.75 * 2^q
  static constexpr int code_bits = 8;
};
template <> struct MxFmt<kE2M1> {
  static constexpr int q = 2;
  static constexpr float fmax = 6.0f;
  static constexpr uint32_t frac_max = 0x400000u;  // fmax = 1.5 * 2^q
  static constexpr int code_bits = 4;
};

// Scale byte of a block from the bits of its largest |x|.  The exponent e is,
// ceil: the smallest with amax <= fmax * 2^e; otherwise floor(log2 amax) - q;
// clamped to [-127, 127], which a subnormal amax reaches at the low end; the
// byte is e + 127.  fmax = (1 + frac_max / 2^23) * 2^q, so under the ceil rule
// the exponent field grows by one exactly when the fraction passes frac_max,
// that is when adding 0x7FFFFF - frac_max carries into it.
template <int FMT, bool CEIL>
__device__ __forceinline__ uint32_t mx_scale_finite(uint32_t amax_bits) {
  const uint32_t field = (amax_bits + (CEIL ? 0x7FFFFFu - MxFmt<FMT>::frac_max : 0u)) >> 23;
  return __builtin_elementwise_sub_sat(field, (uint32_t)MxFmt<FMT>::q);
}
// The same, and 255 for a block with an infinity or a NaN.
template <int FMT, bool CEIL>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits) {
  return amax_bits < kInfBits ? mx_scale_finite<FMT, CEIL>(amax_bits) : 255u;
}

// Codes of values under scale byte `byte` (not 255): cast(x * 2^-e), to
// nearest even, saturating.  The conversions divide by the scale themselves
// (they take 2^e as a float, of which they use the exponent field); E2M1 ones
// saturate.  FP8 ones do not, so where values can pass fmax (the floor rule
// leaves them up to 2^(q+1)) the value is scaled and held to +-fmax first.
template <int FMT>
__device__ __forceinline__ float mx_fit(float x, uint32_t byte) {
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e
  return __builtin_amdgcn_fmed3f(x * inv, -MxFmt<FMT>::fmax, MxFmt<FMT>::fmax);
}
// Four values: FP8 codes in 32 bits, E2M1 codes in the low 16.
typedef short mx_s2 __attribute__((ext_vector_type(2)));
template <int FMT, bool CEIL>
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d, uint32_t byte) {
#if defined(__HIP_DEVICE_COMPILE__)
  const float scale = __uint_as_float(byte << 23);
  if constexpr (FMT == kE2M1) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, scale, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c, d, scale, 1);
  } else if constexpr (CEIL && FMT == 0) {
    mx_s2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true));
  } else if constexpr (CEIL) {
    mx_s2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, a, b, scale, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, c, d, scale, true));
  } else {
    return cvt4<FMT>(mx_fit<FMT>(a, byte), mx_fit<FMT>(b, byte), mx_fit<FMT>(c, byte), mx_fit<FMT>(d, byte));
  }
#else
  return 0;
#endif
}

// Eight codes: FP8 in both words, E2M1 in the first; zeros under scale byte 255.
template <int FMT, bool CEIL>
__device__ __forceinline__ uint2 mx_codes8(const float (&f)[8], uint32_t byte) {
  uint2 o = make_uint2(0u, 0u);
  if constexpr (FMT == kE2M1) {
    o.x = mx_codes4<FMT, CEIL>(f[0], f[1], f[2], f[3], byte) | mx_codes4<FMT, CEIL>(f[4], f[5], f[6], f[7], byte) << 16;
  } else {
    o.x = mx_codes4<FMT, CEIL>(f[0], f[1], f[2], f[3], byte);
    o.y = mx_codes4<FMT, CEIL>(f[4], f[5], f[6], f[7], byte);
  }
  if (byte == 255u) o = make_uint2(0u, 0u);
  return o;
}

__device__ __forceinline__ uint32_t absmax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
  return m;
}

// 2^(b - 127) of a scale byte: NaN for 255, the subnormal 2^-127 for 0.
__device__ __forceinline__ float mx_factor(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

typedef float mx_f2 __attribute__((ext_vector_type(2)));

// Eight codes -> the values they stand for (exact but for fp32's own range).
template <int FMT>
__device__ __forceinline__ void mx_decode8(uint2 w, float factor, float (&f)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
  mx_f2 v[4];
  if constexpr (FMT == kE2M1) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w.x, 1.0f, 3);
  } else if constexpr (FMT == 0) {
    v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
    v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
    v[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
    v[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
  } else {
    v[0] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w.x, false);
    v[1] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w.x, true);
    v[2] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w.y, false);
    v[3] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w.y, true);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = v[j].x * factor;
    f[2 * j + 1] = v[j].y * factor;
  }
#endif
}

// Eight codes of one lane from memory: 8 bytes of FP8, 4 of E2M1.
template <int FMT>
__device__ __forceinline__ uint2 mx_load_codes8(const uint8_t* p) {
  if constexpr (FMT == kE2M1) return make_uint2(*reinterpret_cast<const uint32_t*>(p), 0u);
  const nt_u32x2 v = *reinterpret_cast<const nt_u32x2*>(p);
  return make_uint2(v.x, v.y);
}
template <int FMT>
__device__ __forceinline__ void mx_store_codes8(uint8_t* p, uint2 v) {
  if constexpr (FMT == kE2M1) *reinterpret_cast<uint32_t*>(p) = v.x;
  else store_codes(p, v);
}
// NT: past the caches, for codes that nobody reads soon (what is kept for a
// backward pass).
template <bool NT>
__device__ __forceinline__ void mx_keep_codes8(uint8_t* p, uint2 v) {
  if constexpr (NT) __builtin_nontemporal_store(nt_u32x2{v.x, v.y}, reinterpret_cast<nt_u32x2*>(p));
  else store_codes(p, v);
}

// Eight fp32 values out, as fp32 or rounded (nearest even) to bf16.
typedef __bf16 mx_bf2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t mx_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((mx_f2{lo, hi}), mx_bf2));
}
// NT: past the caches, for outputs larger than they are.
template <bool NT, typename V>
__device__ __forceinline__ void mx_store16(void* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}
template <bool NT>
__device__ __forceinline__ void mx_store8(float* p, const float (&f)[8]) {
  mx_store16<NT>(p, nt_f32x4{f[0], f[1], f[2], f[3]});
  mx_store16<NT>(p + 4, nt_f32x4{f[4], f[5], f[6], f[7]});
}
template <bool NT>
__device__ __forceinline__ void mx_store8(uint16_t* p, const float (&f)[8]) {
  mx_store16<NT>(p, nt_u32x4{mx_bf16x2(f[0], f[1]), mx_bf16x2(f[2], f[3]), mx_bf16x2(f[4], f[5]),
                             mx_bf16x2(f[6], f[7])});
}

// Raw words of eight input elements, converted where they are used.
template <typename T> struct MxRaw;
template <> struct MxRaw<uint16_t> { nt_u32x4 v; };
template <> struct MxRaw<float> { nt_f32x4 a, b; };
template <bool NT>
__device__ __forceinline__ void mx_load_raw(const uint16_t* p, MxRaw<uint16_t>& r) {
  r.v = NT ? __builtin_nontemporal_load(reinterpret_cast<const nt_u32x4*>(p)) : *reinterpret_cast<const nt_u32x4*>(p);
}
template <bool NT>
__device__ __forceinline__ void mx_load_raw(const float* p, MxRaw<float>& r) {
  r.a = NT ? __builtin_nontemporal_load(reinterpret_cast<const nt_f32x4*>(p)) : *reinterpret_cast<const nt_f32x4*>(p);
  r.b = NT ? __builtin_nontemporal_load(reinterpret_cast<const nt_f32x4*>(p + 4))
           : *reinterpret_cast<const nt_f32x4*>(p + 4);
}
__device__ __forceinline__ void mx_zero_raw(MxRaw<uint16_t>& r) { r.v = nt_u32x4{0, 0, 0, 0}; }
__device__ __forceinline__ void mx_zero_raw(MxRaw<float>& r) { r.a = nt_f32x4{0, 0, 0, 0}; r.b = r.a; }
__device__ __forceinline__ void mx_unpack(const MxRaw<uint16_t>& r, float (&f)[8]) {
  f[0] = bf16_lo(r.v.x); f[1] = bf16_hi(r.v.x); f[2] = bf16_lo(r.v.y); f[3] = bf16_hi(r.v.y);
  f[4] = bf16_lo(r.v.z); f[5] = bf16_hi(r.v.z); f[6] = bf16_lo(r.v.w); f[7] = bf16_hi(r.v.w);
}
__device__ __forceinline__ void mx_unpack(const MxRaw<float>& r, float (&f)[8]) {
  f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
  f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}

// A row (or any run below 2 GiB) behind a buffer descriptor: accesses are a
// lane's 32-bit offset plus a uniform one, so the offsets of a lane's units
// cost one register per tensor and not two per unit.  A lane offset of
// kNowhere is outside the descriptor's range: it reads zeros and writes
// nothing.
#if defined(__HIP_DEVICE_COMPILE__)
typedef __amdgpu_buffer_rsrc_t mx_rsrc;
constexpr uint32_t kNowhere = 0xF8000000u;
__device__ __forceinline__ mx_rsrc mx_run(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0xF0000000u, 0x00020000);
}
__device__ __forceinline__ void mx_get(mx_rsrc r, uint32_t lane, uint32_t at, MxRaw<uint16_t>& v) {
  v.v = __builtin_bit_cast(nt_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, at, 0));
}
__device__ __forceinline__ void mx_get(mx_rsrc r, uint32_t lane, uint32_t at, MxRaw<float>& v) {
  v.a = __builtin_bit_cast(nt_f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, at, 0));
  v.b = __builtin_bit_cast(nt_f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, at + 16, 0));
}
__device__ __forceinline__ uint2 mx_get_codes(mx_rsrc r, uint32_t lane, uint32_t at) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, lane, at, 0);
  return make_uint2(v[0], v[1]);
}
__device__ __forceinline__ uint32_t mx_get_byte(mx_rsrc r, uint32_t lane, uint32_t at) {
  return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, lane, at, 0);
}
typedef unsigned int mx_u4 __attribute__((vector_size(16)));
typedef unsigned int mx_u2 __attribute__((vector_size(8)));
// 16-byte stores take the whole offset in the lane's register.  A store of
// more than 8 bytes still reads its data registers when the next instruction
// may write them; the compiler waits for that with a constant uniform offset
// but not with one in a register, and the first of the four words was then
// wrong now and then (seen on fp32 rows, 16 lanes at a time).
__device__ __forceinline__ void mx_put16(mx_rsrc r, uint32_t off, mx_u4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0);
}
__device__ __forceinline__ void mx_put8(mx_rsrc r, uint32_t lane, uint32_t at, const float (&f)[8], uint16_t) {
  mx_put16(r, lane + at, mx_u4{mx_bf16x2(f[0], f[1]), mx_bf16x2(f[2], f[3]), mx_bf16x2(f[4], f[5]),
                               mx_bf16x2(f[6], f[7])});
}
__device__ __forceinline__ void mx_put8(mx_rsrc r, uint32_t lane, uint32_t at, const float (&f)[8], float) {
  mx_put16(r, lane + at,
           mx_u4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])});
  mx_put16(r, lane + at + 16,
           mx_u4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])});
}
__device__ __forceinline__ void mx_put_codes(mx_rsrc r, uint32_t lane, uint32_t at, uint2 v) {
  __builtin_amdgcn_raw_buffer_store_b64(mx_u2{v.x, v.y}, r, lane, at, 0);
}
__device__ __forceinline__ void mx_put_byte(mx_rsrc r, uint32_t lane, uint32_t at, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b8((uint8_t)v, r, lane, at, 0);
}
#endif

}  // namespace mxfp8
