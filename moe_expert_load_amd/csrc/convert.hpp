// Rounding to bf16 by the hardware's conversion.
#pragma once

#include "common.hpp"

namespace moonep {

// Two fp32 values as packed bf16 (lo in bits 0-15), rounded to nearest even,
// subnormals and all (v_cvt_pk_bf16_f32); NaN stays NaN.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

}  // namespace moonep
