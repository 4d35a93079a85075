// 8-bit activation checkpoints: e4m3 codes under one power of two per 32
// consecutive values of a row.
//
// Scale 2^k of a block: the least k >= -127 with max |finite x| <= 448 * 2^k
// (448 is e4m3's largest value), so nothing saturates; stored as k + 127.  A
// code is x / 2^k rounded to nearest even: off by at most 2^-4 of the value,
// or by 2^-10 * 2^k below 2^-6 * 2^k.  448 = 1.75 * 2^8, so with the largest
// magnitude 1.m * 2^e the exponent k is e - 8, and one more if 1.m > 1.75: in
// the bf16 bits, adding 31 carries into the exponent exactly when the seven
// mantissa bits exceed 96.  Dividing by the power of two is exact, and so is a
// code times its scale in bf16 (a code has 4 significant bits).
#pragma once

#include "common.hpp"

namespace moonep {

typedef unsigned int q8_u32x2 __attribute__((ext_vector_type(2)));
typedef float q8_f32x2 __attribute__((ext_vector_type(2)));

constexpr int kQ8Block = 32;

// Largest finite magnitude (bf16 bits) of eight packed values.
__device__ __forceinline__ uint32_t q8_top(const u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t lo = v[q] & 0x7fffu, hi = (v[q] >> 16) & 0x7fffu;
    m = max(m, lo >= 0x7f80u ? 0u : lo);
    m = max(m, hi >= 0x7f80u ? 0u : hi);
  }
  return m;
}

// Maximum over each group of four adjacent lanes (a block of 32 values).
__device__ __forceinline__ uint32_t q8_group_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));
  return m;
}

// Scale byte of a block from its largest magnitude.
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t top) {
  const uint32_t e = (top + 31u) >> 7;
  return e > 8u ? e - 8u : 0u;
}

__device__ __forceinline__ float q8_code_in(float f, float inv) {
  // e4m3 has no infinity: a value that is not finite becomes NaN
  return fabsf(f) < INFINITY ? f * inv : __uint_as_float(0x7fc00000u);
}

// Codes of eight values under scale byte b.
__device__ __forceinline__ q8_u32x2 q8_encode(const u32x4 v, uint32_t b) {
  const float inv = __uint_as_float((254u - b) << 23);       // 2^-k
  int w[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    w[q] = __builtin_amdgcn_cvt_pk_fp8_f32(q8_code_in(bf16_lo(v[2 * q]), inv),
                                           q8_code_in(bf16_hi(v[2 * q]), inv), w[q], false);
    w[q] = __builtin_amdgcn_cvt_pk_fp8_f32(q8_code_in(bf16_lo(v[2 * q + 1]), inv),
                                           q8_code_in(bf16_hi(v[2 * q + 1]), inv), w[q], true);
  }
  return q8_u32x2{(uint32_t)w[0], (uint32_t)w[1]};
}

__device__ __forceinline__ float q8_scale(uint32_t b) {       // 2^k; k = -127 is subnormal
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// The eight values that codes w under scale byte b stand for.
__device__ __forceinline__ void q8_decode(const q8_u32x2 w, uint32_t b, float (&f)[8]) {
  const float s = q8_scale(b);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const q8_f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
    const q8_f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
    f[4 * q] = lo[0] * s;
    f[4 * q + 1] = lo[1] * s;
    f[4 * q + 2] = hi[0] * s;
    f[4 * q + 3] = hi[1] * s;
  }
}

// The same as packed bf16 (exact: the low halves are zero).
__device__ __forceinline__ u32x4 q8_decode_bf16(const q8_u32x2 w, uint32_t b) {
  float f[8];
  q8_decode(w, b, f);
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = (__float_as_uint(f[2 * q]) >> 16) | (__float_as_uint(f[2 * q + 1]) & 0xffff0000u);
  return o;
}

}  // namespace moonep
