// mx_device.hpp -- gfx950 device helpers of the MXFP4 kernels.
//
// gfx950 converts between MXFP4 and wider types itself: the v_cvt_scalef32_*
// instructions take a float scale of which only the exponent field counts, so
// a scale byte s is passed as the bit pattern s << 23.  They round half to
// even, clip at 6, give subnormals, and s = 255 gives NaN (a test holds them to
// all codes, scales and halfway cases).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wqbmm {

typedef float mx_f4 __attribute__((ext_vector_type(4)));
typedef float mx_f2 __attribute__((ext_vector_type(2)));
typedef uint32_t mx_u4 __attribute__((ext_vector_type(4)));
typedef int mx_i4 __attribute__((ext_vector_type(4)));
typedef int mx_i8v __attribute__((ext_vector_type(8)));
typedef __bf16 mx_bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 mx_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_h8 __attribute__((ext_vector_type(8)));
typedef unsigned short mx_u16x2 __attribute__((ext_vector_type(2)));

constexpr int MX_F16 = 0, MX_BF16 = 1, MX_F32 = 2;     // wqbmm_dtype

__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(s << 23); }

__device__ __forceinline__ uint32_t dword_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// The float value of the low 16-bit value of v.
template <int DT>
__device__ __forceinline__ float mx_lo(uint32_t v) {
  if constexpr (DT == MX_BF16) return __uint_as_float(v << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}
template <int DT>
__device__ __forceinline__ float mx_hi(uint32_t v) {
  if constexpr (DT == MX_BF16) return __uint_as_float(v & 0xffff0000u);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(v >> 16));
}
// fp32 -> 16 bits, half to even.
template <int DT>
__device__ __forceinline__ uint16_t mx_round16(float f) {
  if constexpr (DT == MX_BF16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// Scale byte of a block from the bit pattern of its largest magnitude as
// fp32: floor(log2) is the exponent field less 127 (subnormals lie below the
// smallest scale anyway); 255 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// The largest magnitude of a block of 16-bit values, given the largest 16-bit
// pattern without sign (patterns order as values do, NaN above all).
template <int DT>
__device__ __forceinline__ uint32_t mx_top_bits(uint32_t top16) {
  if constexpr (DT == MX_BF16) return top16 << 16;
  else return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)top16));
}
__device__ __forceinline__ uint32_t mx_max16(uint4 v, uint32_t so_far) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  mx_u16x2 m = __builtin_bit_cast(mx_u16x2, so_far);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_u16x2, w[i] & 0x7fff7fffu));
  return __builtin_bit_cast(uint32_t, m);
}
__device__ __forceinline__ uint32_t mx_max16_fold(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Eight values (16 bytes of 16-bit ones) -> eight codes in a dword, lowest
// index in the lowest nibble.  scale: mx_scale(s), s < 255.
template <int DT>
__device__ __forceinline__ uint32_t mx_encode8(uint4 v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r = 0;
  if constexpr (DT == MX_BF16) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, w[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, w[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, w[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(mx_bf2, w[3]), scale, 3);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(mx_h2, w[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(mx_h2, w[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(mx_h2, w[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(mx_h2, w[3]), scale, 3);
  }
  return r;
}
__device__ __forceinline__ uint32_t mx_encode8_f32(const float (&v)[8], float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
  return r;
}

// Eight codes -> eight 16-bit values times scale, ready as an MFMA operand.
template <int DT>
__device__ __forceinline__ uint4 mx_decode8(uint32_t c, float scale) {
  if constexpr (DT == MX_BF16) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3)));
  } else {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 3)));
  }
}

// A quarter of it: the two values of byte `part` (a constant once inlined).
template <int DT>
__device__ __forceinline__ uint32_t mx_decode2(uint32_t c, int part, float scale) {
  if constexpr (DT == MX_BF16) {
    return part == 0   ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0))
           : part == 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1))
           : part == 2 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2))
                       : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  } else {
    return part == 0   ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 0))
           : part == 1 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 1))
           : part == 2 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 2))
                       : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 3));
  }
}

// D[16][16] += A[16][32] . B[32][16] in fp32.  Lane l gives row l%16 of A and
// column l%16 of B, eight values each of the same eight k; it gets column l%16
// of D, rows 4*(l/16) + i.
template <int DT>
__device__ __forceinline__ mx_f4 mx_mfma16(uint4 a, uint4 b, mx_f4 c) {
  if constexpr (DT == MX_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mx_bf8, a), __builtin_bit_cast(mx_bf8, b),
                                                   c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(mx_h8, a), __builtin_bit_cast(mx_h8, b),
                                                  c, 0, 0, 0);
}

// D[16][16] += A[16][128] . B[128][16], both MXFP4: lane l gives the block
// l/16 (32 codes, one scale byte) of row / column l%16.  SA, SB: which byte of
// the scale dwords.
template <int SA, int SB>
__device__ __forceinline__ mx_f4 mx_mfma4(uint4 a, uint32_t sa, uint4 b, uint32_t sb, mx_f4 c) {
  const mx_i8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const mx_i8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// fp16 values as the exact sum of two bf16 ones: 11 significant bits are 8 and
// the rest.  An infinity has rest 0 (inf - inf would be NaN).
__device__ __forceinline__ void mx_split8(uint4 v, uint4& hi, uint4& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f0 = mx_lo<MX_F16>(w[i]), f1 = mx_hi<MX_F16>(w[i]);
    const mx_bf2 b = {(__bf16)f0, (__bf16)f1};
    h[i] = __builtin_bit_cast(uint32_t, b);
    const float r0 = f0 - mx_lo<MX_BF16>(h[i]), r1 = f1 - mx_hi<MX_BF16>(h[i]);
    const mx_bf2 r = {(__bf16)(__builtin_isfinite(f0) ? r0 : 0.0f), (__bf16)(__builtin_isfinite(f1) ? r1 : 0.0f)};
    l[i] = __builtin_bit_cast(uint32_t, r);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Four fp32 values as the sum of three bf16 parts each, packed: 24 significant
// bits are eight, eight and eight, cut off and not rounded, so that no part is
// larger than the value (below 2^-110 the last part loses bits that bf16 does not
// have).  An infinity has rests 0 (inf - inf would be NaN).
__device__ __forceinline__ void mx_split24(mx_f4 v, uint2 (&part)[3]) {
  uint32_t o[3][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      o[n][i] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);           // the upper halves
      a = __builtin_isinf(a) ? 0.0f : a - __uint_as_float(ua & 0xffff0000u);
      b = __builtin_isinf(b) ? 0.0f : b - __uint_as_float(ub & 0xffff0000u);
    }
  }
#pragma unroll
  for (int n = 0; n < 3; ++n) part[n] = make_uint2(o[n][0], o[n][1]);
}

}  // namespace wqbmm
