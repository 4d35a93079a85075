// What follows a matrix product on its way out: bias, activation, dropout and
// residual, eight consecutive columns of a row at a time; and dropout's numbers.
//
//   z = product + bias,   v = act(z),   y = residual + (kept ? v * scale : 0)
//
// Dropout draws 16 bits per value from Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), a keyed bijection
// of a 128-bit counter: block n of step s under a seed covers the values 8n ..
// 8n + 7 of the tensor, so the backward draws the same numbers from the same
// three and no mask is stored.  A block costs 20 32-bit multiplications that
// give both halves, about 15 instruction slots a value: more than half of what
// a pass at the memory's rate leaves, which is why a block serves eight values
// and not four.
#pragma once

#include "common.hpp"
#include "convert.hpp"

namespace moonep {

struct DropKey {
  uint32_t seed_lo, seed_hi, step_lo, step_hi;
};

__device__ __forceinline__ DropKey drop_key(const int64_t* rng) {
  const uint64_t seed = (uint64_t)rng[0], step = (uint64_t)rng[1];
  return DropKey{uint32_t(seed), uint32_t(seed >> 32), uint32_t(step), uint32_t(step >> 32)};
}

// The eight 16-bit numbers of block n: value i has bits 16 (i % 2) .. of word i / 2.
__device__ __forceinline__ u32x4 drop_bits(const DropKey& k, uint64_t n) {
  uint32_t a = uint32_t(n), b = uint32_t(n >> 32), c = k.step_lo, d = k.step_hi;
  uint32_t k0 = k.seed_lo, k1 = k.seed_hi;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t x = uint64_t(a) * 0xD2511F53u, z = uint64_t(c) * 0xCD9E8D57u;
    a = uint32_t(z >> 32) ^ b ^ k0;
    b = uint32_t(z);
    c = uint32_t(x >> 32) ^ d ^ k1;
    d = uint32_t(x);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{a, b, c, d};
}

// v with the values whose number is below `cut` zero and the others scaled.
__device__ __forceinline__ void drop8(float (&v)[8], const DropKey& k, uint64_t n, uint32_t cut,
                                      float scale) {
  const u32x4 w = drop_bits(k, n);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
    v[i] = bits >= cut ? v[i] * scale : 0.f;
  }
}

// 1 / x by the hardware reciprocal (1 ulp).
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution below -a, a >= 0, and e = exp(-a^2 / 2): Phi(-a) =
// e * erfcx(a / sqrt 2) / 2, the second factor a polynomial in t = 1 / (1 +
// 0.375 a) fitted to it for the least relative error over all a (2.3e-7; 4.7e-7
// with fp32 arithmetic), so the far tail keeps its leading digits.
__device__ __forceinline__ float normal_tail(float a, float& e) {
  e = __expf(-0.5f * a * a);
  const float t = rcp_fast(fmaf(0.375f, a, 1.f));
  float g = -0.032910704612731934f;
  g = fmaf(g, t, 0.1368783563375473f);
  g = fmaf(g, t, -0.18651820719242096f);
  g = fmaf(g, t, 0.05062931030988693f);
  g = fmaf(g, t, 0.01562977209687233f);
  g = fmaf(g, t, 0.088637575507164f);
  g = fmaf(g, t, 0.1284458190202713f);
  g = fmaf(g, t, 0.14960457384586334f);
  g = fmaf(g, t, 0.14960338175296783f);
  return e * (g * t);
}

constexpr float kTanh2 = 1.5957691216057308f;              // 2 sqrt(2 / pi)

// 1 / (1 + exp(-2u)), 2u = kTanh2 (z + 0.044715 z^3): (1 + tanh u) / 2.
__device__ __forceinline__ float tanh_share(float z) {
  return rcp_fast(1.f + __expf(-kTanh2 * fmaf(0.044715f * z * z, z, z)));
}

// act(z) of eight values; `act` is the same for the whole launch.
__device__ __forceinline__ void act8(float (&z)[8], int act) {
  if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      const float below = normal_tail(fabsf(z[i]), e);
      z[i] *= z[i] < 0.f ? below : 1.f - below;
    }
  } else if (act == MOE_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= tanh_share(z[i]);
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= rcp_fast(1.f + __expf(-z[i]));
  } else if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];   // NaN passes
  } else if (act == MOE_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = z[i] < 0.f ? 0.f : z[i] * z[i];
  }
}

// d[i] *= act'(z[i]).
__device__ __forceinline__ void act_grad8(float (&d)[8], const float (&z)[8], int act) {
  if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      const float below = normal_tail(fabsf(z[i]), e);
      d[i] *= fmaf(0.3989422804014327f * z[i], e, z[i] < 0.f ? below : 1.f - below);
    }
  } else if (act == MOE_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = tanh_share(z[i]), q = s * (1.f - s);
      // where s has reached 0 or 1 the second term is below every digit, and z^2 may overflow
      const float bend = z[i] * q * (kTanh2 * fmaf(0.134145f * z[i], z[i], 1.f));
      d[i] *= q == 0.f ? s : s + bend;
    }
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = rcp_fast(1.f + __expf(-z[i]));
      d[i] *= s * fmaf(z[i], 1.f - s, 1.f);
    }
  } else if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= z[i] > 0.f ? 1.f : z[i] == z[i] ? 0.f : z[i];
  } else if (act == MOE_ACT_RELU2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= z[i] < 0.f ? 0.f : 2.f * z[i];
  }
}

// Eight values at p, bf16 or fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[2 * q] = bf16_lo(w[q]);
    v[2 * q + 1] = bf16_hi(w[q]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = a[q];
    v[4 + q] = b[q];
  }
}
__device__ __forceinline__ u32x4 round8(const float (&v)[8]) {
  return u32x4{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
               cvt_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) = round8(v);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

// The same past the caches, for tensors that a pass reads or writes once: a
// stream that stays in the caches costs the others their place (65,536 x 7,168
// dropped and added, bf16: 0.49 ms through them, 0.46 to 0.47 past them).
__device__ __forceinline__ void load8_once(const uint16_t* p, float (&v)[8]) {
  const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[2 * q] = bf16_lo(w[q]);
    v[2 * q + 1] = bf16_hi(w[q]);
  }
}
__device__ __forceinline__ void load8_once(const float* p, float (&v)[8]) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = a[q];
    v[4 + q] = b[q];
  }
}
__device__ __forceinline__ void store8_once(uint16_t* p, const float (&v)[8]) {
  __builtin_nontemporal_store(round8(v), reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void store8_once(float* p, const float (&v)[8]) {
  __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(p + 4));
}

// One launch's epilogue.  All rows have N columns.
struct Epilogue {
  const float* bias;          // [E][N] or null
  const void* residual;       // [rows][N] of y's type, or null; may be y
  const int64_t* rng;         // seed and step; null without dropout
  void* y;                    // [rows][N], fp32 (f32) or bf16
  uint16_t* pre;              // [rows][N] or null: z, rounded
  const int32_t* slot_expert; // [R][B]
  int32_t act, f32, N;
  uint32_t cut;               // dropout in steps of 2^-16; 0: none
  float scale;
};

// Eight residual values as they lie in memory (bf16: the first half only).
struct Residual8 {
  u32x4 v[2];
};
__device__ __forceinline__ Residual8 residual8(const Epilogue& ep, int64_t at) {
  Residual8 r;
  if (ep.f32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(ep.residual) + at);
    r.v[0] = p[0];
    r.v[1] = p[1];
  } else {
    r.v[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(ep.residual) + at);
    r.v[1] = u32x4{0, 0, 0, 0};
  }
  return r;
}

// z + residual, rounded once, to y (8,192 x 2,048 x 7,168 with dropout and residual,
// one launch after another: 271 to 278 us with y through the caches, 261 to 268 past
// them; with new inputs each time 278 to 284 and 272 to 279).
__device__ __forceinline__ void finish8(const Epilogue& ep, float (&z)[8], const Residual8& r,
                                        int64_t at) {
  if (ep.f32) {
    if (ep.residual)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += __uint_as_float(r.v[i >> 2][i & 3]);
    store8_once(static_cast<float*>(ep.y) + at, z);
  } else {
    if (ep.residual)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z[2 * q] += bf16_lo(r.v[0][q]);
        z[2 * q + 1] += bf16_hi(r.v[0][q]);
      }
    store8_once(static_cast<uint16_t*>(ep.y) + at, z);
  }
}

// pre, activation and dropout of z = product + bias.
__device__ __forceinline__ void middle8(const Epilogue& ep, const DropKey& key, float (&z)[8],
                                        int64_t at) {
  if (ep.pre) store8_once(ep.pre + at, z);
  act8(z, ep.act);
  if (ep.cut) drop8(z, key, uint64_t(at) >> 3, ep.cut, ep.scale);
}

// Columns n .. n + 7 of row `row` from their products z and biases b.  The
// residual is asked for first: the rest covers its latency.
__device__ __forceinline__ void epilogue8(const Epilogue& ep, const DropKey& key, float (&z)[8],
                                          const float (&b)[8], int64_t row, int n) {
  const int64_t at = row * ep.N + n;
  Residual8 r{};
  if (ep.residual) r = residual8(ep, at);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
  middle8(ep, key, z, at);
  finish8(ep, z, r, at);
}

// A wave's block of z staged in LDS: groups 0 .. NG - 1 of this lane, group k at
// place(k, at) (its eight values; `at` the flat index of the first in y), null
// where there is none.  All residuals are asked for before the first group's
// arithmetic.  The activations are long code: a loop of their own, which leaves
// the values where they were.  Without one a group goes through in one piece
// (8,192 x 2,048 x 7,168 with dropout and residual, one launch after another: 267 to
// 273 us by two loops, 261 to 268; with new inputs 287 to 291, 272 to 279).
template <int NG, typename Place>
__device__ __forceinline__ void epilogue_block(const Epilogue& ep, const DropKey& key,
                                               Place&& place) {
  Residual8 r[NG];
  if (ep.residual)
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      int64_t at = 0;
      if (place(k, at)) r[k] = residual8(ep, at);
    }
  const bool plain = ep.act == MOE_ACT_NONE;
  if (!plain)
#pragma unroll 1
    for (int k = 0; k < NG; ++k) {
      int64_t at = 0;
      float* p = place(k, at);
      if (!p) continue;
      float z[8];
      load8(p, z);
      middle8(ep, key, z, at);
      store8(p, z);
    }
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    int64_t at = 0;
    float* p = place(k, at);
    if (!p) continue;
    float z[8];
    load8(p, z);
    if (plain && ep.pre) store8_once(ep.pre + at, z);
    if (plain && ep.cut) drop8(z, key, uint64_t(at) >> 3, ep.cut, ep.scale);
    finish8(ep, z, r[k], at);
  }
}

// Bias of column n of expert e, 0 without one.
__device__ __forceinline__ float bias1(const Epilogue& ep, int e, int E, int n) {
  return ep.bias && (unsigned)e < (unsigned)E && n < ep.N ? ep.bias[int64_t(e) * ep.N + n] : 0.f;
}

// Biases of columns n .. n + 7 of expert e; an id outside [0, E) has none.
__device__ __forceinline__ void bias8(const Epilogue& ep, int e, int E, int n, float (&b)[8]) {
  if (ep.bias && (unsigned)e < (unsigned)E && n < ep.N) load8(ep.bias + int64_t(e) * ep.N + n, b);
  else
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
}

// Expert whose weights row j of rank r holds.
__device__ __forceinline__ int expert_of(const Epilogue& ep, int r, int j, int E, int B) {
  return j < E || !ep.slot_expert ? j : ep.slot_expert[int64_t(r) * B + (j - E)];
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// Dropout of probability p in steps of 2^-16: whether p is one, the values
// below which a number drops its value, and the factor on the others.
inline bool drop_params(float p, uint32_t* cut, float* scale) {
  if (!(p >= 0.f && p <= 1.f)) return false;
  *cut = (uint32_t)(double(p) * 65536.0 + 0.5);
  *scale = *cut < 65536u ? (float)(65536.0 / (65536.0 - *cut)) : 0.f;
  return true;
}

// Whether rng can be read as two int64, or is not needed.
inline bool rng_ok(const int64_t* rng, uint32_t cut) {
  return cut == 0 || (rng && (reinterpret_cast<uintptr_t>(rng) & 7) == 0);
}

inline bool valid_epilogue(const moe_epilogue_cfg* ec) {
  uint32_t cut;
  float scale;
  return ec && ec->act >= MOE_ACT_NONE && ec->act <= MOE_ACT_RELU2 &&
         (ec->f32 == 0 || ec->f32 == 1) && drop_params(ec->p, &cut, &scale);
}

// Bytes of workspace of the epilogue's backward (epilogue.hip).
size_t epilogue_bwd_ws_bytes(const moe_cfg* c);

// The shape that a null plan stands for: every row belongs to one matrix.
inline bool one_matrix(const moe_cfg* c) { return c->R == 1 && c->E == 1; }

}  // namespace moonep
