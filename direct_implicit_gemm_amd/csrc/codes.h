// codes.h -- the codes of an 8-bit cache on the device: rounding to them, and
// the values they stand for in units of the scale, which fp16 and bfloat16
// hold exactly.
#pragma once

#include "attention_common.h"
#include "libconv.h"

namespace libconv {

template <int CF> constexpr float kMostCode = CF == LIBCONV_CACHE_I8 ? 127.0f : 448.0f;

// The 4 codes of a word.
template <int CF> __device__ __forceinline__ void code_values(uint32_t w, float* f) {
  if constexpr (CF == LIBCONV_CACHE_I8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(w >> (8 * j));
  } else {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = lo[0]; f[1] = lo[1]; f[2] = hi[0]; f[3] = hi[1];
  }
}

// The 4 codes of a word in a 16-bit type.
template <int CF, int DT> __device__ __forceinline__ u32x2_t code_values16(uint32_t w) {
  if constexpr (CF == LIBCONV_CACHE_I8) {
    float f[4];
    code_values<CF>(w, f);
    return u32x2_t{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])};
  } else if constexpr (DT == DT_F16) {
    return u32x2_t{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
  } else {
    return u32x2_t{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
  }
}
// 8 codes: an operand of a matrix instruction.
template <int CF, int DT>
__device__ __forceinline__ u32x4_t code_values16(uint32_t w0, uint32_t w1) {
  const u32x2_t a = code_values16<CF, DT>(w0), b = code_values16<CF, DT>(w1);
  return u32x4_t{a[0], a[1], b[0], b[1]};
}

// 8 codes times a power of two, for products that the type holds.
template <int CF, int DT>
__device__ __forceinline__ u32x4_t code_values16(uint32_t w0, uint32_t w1, float power) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i == 0 ? w0 : w1;
    if constexpr (CF == LIBCONV_CACHE_I8) {
      float f[4];
      code_values<CF>(w, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] *= power;
      v[2 * i] = pack2<DT>(f[0], f[1]);
      v[2 * i + 1] = pack2<DT>(f[2], f[3]);
    } else if constexpr (DT == DT_F16) {   // (the conversions multiply by the power of two)
      v[2 * i] = __builtin_bit_cast(uint32_t,
                                    __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, power, false));
      v[2 * i + 1] = __builtin_bit_cast(uint32_t,
                                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, power, true));
    } else {
      v[2 * i] = __builtin_bit_cast(uint32_t,
                                    __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, false));
      v[2 * i + 1] = __builtin_bit_cast(uint32_t,
                                        __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, true));
    }
  }
  return v;
}

// The codes of 4 values, given in units of the scale: to nearest even, an
// infinity as the largest code (the conversion to 8-bit floats would make a NaN
// of it), a NaN as NaN or 0.
template <int CF> __device__ __forceinline__ uint32_t codes_of(const float* x) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = fminf(fmaxf(x[j], -kMostCode<CF>), kMostCode<CF>);
    if constexpr (CF == LIBCONV_CACHE_I8) v[j] = x[j] != x[j] ? 0.0f : __builtin_rintf(v[j]);
    else v[j] = x[j] != x[j] ? x[j] : v[j];
  }
  if constexpr (CF == LIBCONV_CACHE_I8) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= ((uint32_t)(int)v[j] & 0xffu) << (8 * j);
    return w;
  } else {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  }
}

// The same for numbers within the codes' range.
template <int CF> __device__ __forceinline__ uint32_t codes_within(const float* x) {
  if constexpr (CF == LIBCONV_CACHE_I8) {
    // 1.5 * 2^23 + x: the sum's rounding is x's, and its lowest byte the code
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = __builtin_bit_cast(uint32_t, x[j] + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    return lo | hi;
  } else {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
  }
}

}  // namespace libconv
