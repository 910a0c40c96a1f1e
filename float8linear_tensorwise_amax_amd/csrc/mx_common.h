// Shared by the microscaled 4-bit (MXFP4) kernels: element types, and the
// arithmetic of a block.
//
// 32 consecutive values along a product's contraction form a block with one
// e8m0 scale byte e, standing for 2^(e - 127) (255: NaN), and 32 e2m1 codes
// (sign, two exponent bits, one mantissa bit: magnitudes 0, 0.5, 1, 1.5, 2,
// 3, 4, 6).  With m the block's largest magnitude:
//   floor rule: e - 127 = floor(log2 m) - 2       (values in (6, 8) * 2^(e-127) saturate)
//   ceil rule : the smallest e - 127 with m <= 6 * 2^(e - 127)
//   (e >= 0; a block of zeros has e = 0; an Inf or NaN in the block gives
//   e = 255 and zero codes, so the whole block reads back as NaN)
//   code = RNE_sat(x * 2^(127 - e)), ties to the even mantissa, sign kept.
// A code byte holds two elements, the even one in its low half; a block is 16
// bytes, which is exactly what one lane feeds the 16 x 16 x 128 f8f6f4 matrix
// instruction, next to that block's one scale byte.
#pragma once

#include "device_common.h"
#include "internal.h"

namespace f8lin {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at any 2-byte address (rows of odd length start anywhere)
typedef u32x4 u32x4_u __attribute__((aligned(2)));
typedef u32x2 u32x2_u __attribute__((aligned(2)));

constexpr int kMxBlock = 32;
constexpr int kMxNan = 255;

// e8m0 byte of a block whose largest magnitude has these binary32 bits (sign
// clear).  bits >> 23 is the exponent field; the ceil rule takes one more when
// the mantissa exceeds 1.5 (6 = 1.5 * 2^2).  Subnormal and tiny maxima clamp
// to 0: m < 2^-124 fits 8 * 2^-127, and for the ceil rule m <= 1.5 * 2^-125.
template <int RULE>
__device__ __forceinline__ int mx_scale_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return kMxNan;
  int e = (int)(bits >> 23) - 2;
  if (RULE == F8LIN_MX_CEIL) e += (bits & 0x7FFFFFu) > 0x400000u ? 1 : 0;
  return max(e, 0);
}

// The scale as the binary32 value the conversion instructions take: only its
// exponent field is read, and 0 there stands for 2^-127.
__device__ __forceinline__ float mx_scale_f32(int e) { return __uint_as_float((uint32_t)e << 23); }

// Eight values -> eight codes (value i in bits 4i .. 4i + 3), divided by the
// scale, rounded to nearest even and saturated by v_cvt_scalef32_pk_fp4_f32.
__device__ __forceinline__ uint32_t mx_cvt8(const float (&v)[8], float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
  return r;
}

template <int DT>
struct MxElem;  // storage type of an f8lin_dtype
template <>
struct MxElem<F8LIN_BF16> {
  typedef uint16_t type;
};
template <>
struct MxElem<F8LIN_FP16> {
  typedef uint16_t type;
};
template <>
struct MxElem<F8LIN_FP32> {
  typedef uint32_t type;
};

__device__ __forceinline__ float f16_bits_to_f32(uint32_t h) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));     // lanes 1 0 3 2
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Element `bits` of type DT as binary32 (exact).
template <int DT>
__device__ __forceinline__ float elem_f32(uint32_t bits) {
  if constexpr (DT == F8LIN_BF16) return __uint_as_float(bits << 16);
  if constexpr (DT == F8LIN_FP16) return f16_bits_to_f32(bits);
  return __uint_as_float(bits);
}

// binary32 -> element bits of type dt (nearest even).
__device__ __forceinline__ uint32_t f32_to_elem(float v, int dt) {
  if (dt == F8LIN_BF16) return f32_to_bf16_rne(v);
  if (dt == F8LIN_FP16) return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
  return __float_as_uint(v);
}
__host__ __device__ __forceinline__ int elem_bytes(int dt) { return dt == F8LIN_FP32 ? 4 : 2; }

// Eight consecutive elements as they lie in memory: the 16-bit types in
// pairs, as the conversion instructions take them.
template <int DT>
struct Raw8 {
  u32x4 w[DT == F8LIN_FP32 ? 2 : 1];
};

// Eight elements of type DT at p (any element address); `n` of them exist
// (the rest read as +0).  ONCE: the launch reads them once, so that they need
// no place in the L2.
template <int DT, bool ONCE = false>
__device__ __forceinline__ Raw8<DT> load_raw8(const typename MxElem<DT>::type *p, int n) {
  Raw8<DT> r;
  if (n >= 8) {
#pragma unroll
    for (int h = 0; h < (DT == F8LIN_FP32 ? 2 : 1); ++h) {
      const u32x4_u *q = reinterpret_cast<const u32x4_u *>(p + 4 * h);
      r.w[h] = ONCE ? __builtin_nontemporal_load(q) : *q;
    }
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? (uint32_t)p[i] : 0u;
    if constexpr (DT == F8LIN_FP32) {
      r.w[0] = u32x4{e[0], e[1], e[2], e[3]};
      r.w[1] = u32x4{e[4], e[5], e[6], e[7]};
    } else {
      r.w[0] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
  }
  return r;
}

// Largest magnitude of pairs of 16-bit elements, per half (integer order of
// the magnitude bits is the order of the values, NaN last).
__device__ __forceinline__ uint32_t pair_mag_max(uint32_t m, uint32_t w) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m),
                                                                __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu)));
}

// binary32 bits of the 16-bit magnitude m.
template <int DT>
__device__ __forceinline__ uint32_t mag_f32_bits(uint32_t m) {
  if constexpr (DT == F8LIN_BF16) return m << 16;
  if constexpr (DT == F8LIN_FP16) return __float_as_uint(f16_bits_to_f32(m));
  return m;
}

// Largest magnitude of the eight, as bits of type DT.
template <int DT>
__device__ __forceinline__ uint32_t raw_mag(const Raw8<DT> &r) {
  uint32_t m = 0;
  if constexpr (DT == F8LIN_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(r.w[0][i] & 0x7FFFFFFFu, r.w[1][i] & 0x7FFFFFFFu));
    return m;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = pair_mag_max(m, r.w[0][i]);
    return max(m & 0xFFFFu, m >> 16);
  }
}

// Two elements (a packed pair) -> two codes in byte `SEL` of r.
template <int DT, int SEL>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t r, uint32_t w, float scale) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  if constexpr (DT == F8LIN_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w), scale, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(f16x2_t, w), scale, SEL);
}
template <int DT>
__device__ __forceinline__ uint32_t cvt_pairs(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float scale) {
  uint32_t r = 0;
  r = cvt_pair<DT, 0>(r, a, scale);
  r = cvt_pair<DT, 1>(r, b, scale);
  r = cvt_pair<DT, 2>(r, c, scale);
  return cvt_pair<DT, 3>(r, d, scale);
}

// The eight elements' codes.
template <int DT>
__device__ __forceinline__ uint32_t raw_codes(const Raw8<DT> &r, float scale) {
  if constexpr (DT == F8LIN_FP32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i >> 2][i & 3]);
    return mx_cvt8(v, scale);
  } else {
    return cvt_pairs<DT>(r.w[0][0], r.w[0][1], r.w[0][2], r.w[0][3], scale);
  }
}

// Element i of eight, as binary32.
template <int DT>
__device__ __forceinline__ float raw_value(const Raw8<DT> &r, int i) {
  if constexpr (DT == F8LIN_FP32) return __uint_as_float(r.w[i >> 2][i & 3]);
  else return elem_f32<DT>((r.w[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

}  // namespace f8lin
