// attention_common.h -- what the kernels of prefix_attention and of
// cache_attention share: lane exchanges, the transposing LDS read, the packing
// of probabilities, the order of workgroups over the XCDs.
#pragma once

#include "device_common.h"

namespace libconv {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e38f;   // the maximum of no keys: finite, so that no
                                              // difference of maxima is a NaN

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// The larger of v in this lane and in the lane 32 away.
__device__ __forceinline__ float swap_halves_max(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  // (through scalars: a bit cast of a vector's element takes element 0)
  const uint32_t lower = r[0], upper = r[1];
  return fmaxf(__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper));
}

// 4 elements of one column of 16-bit elements: the 16 lanes of a quarter wave
// name 8 bytes each of 4 rows.  `p` is restrict so that the read has a scope of
// its own: without one, the compiler lets it wait for every copy to LDS that
// is on its way, those of the next tile among them.
__device__ __forceinline__ u32x2_t read_column(const unsigned char* __restrict p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4_t*)p));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  if constexpr (DT == DT_F16) {
    typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2_t));
  } else {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  }
}

// Workgroups that read the same keys (one entry and key head) follow one
// another on one XCD, whose L2 then holds those keys: dispatch deals
// workgroups out to the 8 XCDs in turn.
__device__ __forceinline__ int xcd_order(int id, int n) {
  const int per = n >> 3, more = n & 7, x = id & 7;
  return x * per + (x < more ? x : more) + (id >> 3);
}

}  // namespace libconv
