// Dropout with a residual, alone and around the gate-weighted combine, and the
// combine's gradients through it.  The numbers come from a counter
// (epilogue.hpp); nothing is stored between the passes.  All three are bound by
// memory: every tensor is read or written once.
#include <algorithm>
#include <type_traits>

#include "epilogue.hpp"
#include "host.hpp"
#include "overlap.hpp"

namespace moonep {

// ---------------------------------------------------------------------------
// dst = residual + dropout(src): a lane takes groups of eight values, U of them
// with their loads in flight together.  dst may be src or residual.
// 65,536 rows of 7,168 with a residual, bf16: 0.46 to 0.48 ms (6.0 TB/s), 0.48 to 0.51
// in the first launches after a pause; 8 rows: 3 us.
// ---------------------------------------------------------------------------
template <typename T, int U>
__global__ __launch_bounds__(256) void k_dropout(const T* src, const T* residual,
                                                 const int64_t* rng, T* dst, int64_t groups,
                                                 uint32_t cut, float scale) {
  DropKey key{};
  if (cut) key = drop_key(rng);
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t g0 = int64_t(blockIdx.x) * 256 + threadIdx.x; g0 < groups; g0 += step * U) {
    float v[U][8], r[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = min(g0 + u * step, groups - 1);
      load8_once(src + g * 8, v[u]);
      if (residual) load8_once(residual + g * 8, r[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * step;
      if (g >= groups) break;
      if (cut) drop8(v[u], key, uint64_t(g), cut, scale);
      if (residual)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] += r[u][i];
      store8_once(dst + g * 8, v[u]);
    }
  }
}

// ---------------------------------------------------------------------------
// out[t] = residual[t] + dropout(sum_k gates[t][k] * y[route_k]): W waves per
// token, CU groups of eight columns a lane, KB rows in flight (as k_combine).
// A row of at most 1,024 columns is one pass of one wave, four tokens to a
// workgroup; a longer one is shared by the four waves of a workgroup, so that
// few tokens do not wait for passes one after the other and many read a row's
// bytes together (W = 1 in brackets, 8 routes): 8 tokens of 7,168 columns 6.3 us
// (18.2), 1,024 24 (33); 65,536 1.71 to 1.76 ms, 5.4 TB/s (1.82 ms); of 2,048 columns
// 0.43 ms, 6.2 TB/s (0.44; 0.49 with `out` kept in the caches).  At 4,096 rows of
// 1,000 columns four waves lose: 12.0 us against 10.0.
// ---------------------------------------------------------------------------
template <typename T, int CU, int KB, int W>
__global__ __launch_bounds__(256) void k_combine_drop(const u32x4* __restrict__ y,
                                                      const float* __restrict__ gates,
                                                      const int32_t* __restrict__ route,
                                                      const T* residual, const int64_t* rng, T* out,
                                                      int ntok, int K, int hv, uint32_t cut,
                                                      float scale) {
  const int wv = threadIdx.x / kWave;
  const int t = W == 1 ? blockIdx.x * 4 + wv : blockIdx.x;
  if (t >= ntok) return;                                  // whole waves leave together
  const int lane = lane_id();
  DropKey key{};
  if (cut) key = drop_key(rng);
  const int myroute = lane < K ? route[int64_t(t) * K + lane] : -1;
  const float mygate = lane < K ? gates[int64_t(t) * K + lane] : 0.f;
  for (int c0 = W == 1 ? 0 : wv * kWave * CU; c0 < hv; c0 += kWave * CU * W) {
    float acc[CU][8];
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[u][i] = 0.f;
    for (int k0 = 0; k0 < K; k0 += KB) {
      u32x4 v[KB][CU];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int src = wave_bcast(myroute, min(k0 + kb, K - 1));
        const bool ok = k0 + kb < K && src >= 0;
        const u32x4* row = y + int64_t(ok ? src : 0) * hv;
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int c = c0 + u * kWave + lane;
          // every y row is read exactly once: stream it past the caches
          v[kb][u] = (ok && c < hv) ? __builtin_nontemporal_load(row + c) : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (k0 + kb >= K || wave_bcast(myroute, k0 + kb) < 0) continue;   // uniform
        const float g = __int_as_float(wave_bcast(__float_as_int(mygate), k0 + kb));
#pragma unroll
        for (int u = 0; u < CU; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[u][2 * q] = fmaf(g, bf16_lo(v[kb][u][q]), acc[u][2 * q]);
            acc[u][2 * q + 1] = fmaf(g, bf16_hi(v[kb][u][q]), acc[u][2 * q + 1]);
          }
      }
    }
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int c = c0 + u * kWave + lane;
      if (c >= hv) continue;
      const int64_t g = int64_t(t) * hv + c;
      if (cut) drop8(acc[u], key, uint64_t(g), cut, scale);
      if (residual) {
        float r[8];
        load8(residual + g * 8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] += r[i];
      }
      store8_once(out + g * 8, acc[u]);
    }
  }
}

// ---------------------------------------------------------------------------
// Its gradients: the numbers of a row are drawn once and the masked gradient d
// stays in fp32 registers for the K rows (as k_combine_bwd); W as above, the
// gates' gradients of the waves added in their order.  8 routes: 8 tokens of
// 7,168 columns 7.4 us (W = 1: 23.5); 65,536 3.15 to 3.18 ms, 5.0 TB/s (3.17; 3.23 with dy
// through the caches); of 2,048 columns 0.87 ms, 5.2 TB/s (0.88; 0.92).
// ---------------------------------------------------------------------------
template <typename T, int CU, int KB, int W>
__global__ __launch_bounds__(256) void k_combine_drop_bwd(const T* __restrict__ dout,
                                                          const u32x4* __restrict__ y,
                                                          const float* gates,
                                                          const int32_t* __restrict__ route,
                                                          const int64_t* rng,
                                                          u32x4* __restrict__ dy, float* dgates,
                                                          int ntok, int K, int hv, uint32_t cut,
                                                          float scale) {
  __shared__ float s_dot[W][kWave];
  const int wv = threadIdx.x / kWave;
  const int t = W == 1 ? blockIdx.x * 4 + wv : blockIdx.x;
  if (t >= ntok) return;                                  // W > 1: never
  const int lane = lane_id();
  DropKey key{};
  if (cut) key = drop_key(rng);
  const int myroute = lane < K ? route[int64_t(t) * K + lane] : -1;
  const float mygate = lane < K ? gates[int64_t(t) * K + lane] : 0.f;
  float mydot = 0.f;                                      // lane k: dgates[t, k]
  for (int c0 = W == 1 ? 0 : wv * kWave * CU; c0 < hv; c0 += kWave * CU * W) {
    float d[CU][8];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int c = c0 + u * kWave + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[u][i] = 0.f;
      if (c < hv) load8(dout + (int64_t(t) * hv + c) * 8, d[u]);
    }
    if (cut)
#pragma unroll
      for (int u = 0; u < CU; ++u)
        drop8(d[u], key, uint64_t(int64_t(t) * hv + c0 + u * kWave + lane), cut, scale);
    for (int k0 = 0; k0 < K; k0 += KB) {
      u32x4 v[KB][CU];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int src = wave_bcast(myroute, min(k0 + kb, K - 1));
        const bool ok = k0 + kb < K && src >= 0;
        const u32x4* row = y + int64_t(ok ? src : 0) * hv;
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int c = c0 + u * kWave + lane;
          v[kb][u] = (ok && c < hv) ? __builtin_nontemporal_load(row + c) : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (k0 + kb >= K) break;                          // uniform
        const int dst = wave_bcast(myroute, k0 + kb);
        if (dst < 0) continue;
        const float g = __int_as_float(wave_bcast(__float_as_int(mygate), k0 + kb));
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int c = c0 + u * kWave + lane;
          float o[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            part = fmaf(d[u][2 * q], bf16_lo(v[kb][u][q]), part);
            part = fmaf(d[u][2 * q + 1], bf16_hi(v[kb][u][q]), part);
            o[2 * q] = g * d[u][2 * q];
            o[2 * q + 1] = g * d[u][2 * q + 1];
          }
          if (c < hv) __builtin_nontemporal_store(round8(o), dy + int64_t(dst) * hv + c);
        }
        const float s = wave_sum_f(part);
        if (lane == k0 + kb) mydot += s;
      }
    }
  }
  if constexpr (W > 1) {
    s_dot[wv][lane] = mydot;
    __syncthreads();                                      // gates are read: dgates may be gates
    if (wv > 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) mydot += s_dot[w][lane];
  }
  if (lane < K) dgates[int64_t(t) * K + lane] = mydot;
}

static bool valid_dropout(const moe_dropout_cfg* dc, uint32_t* cut, float* scale) {
  return dc && (dc->f32 == 0 || dc->f32 == 1) && drop_params(dc->p, cut, scale);
}

template <typename T>
static void run_dropout(const void* src, const void* residual, const int64_t* rng, void* dst,
                        int64_t groups, uint32_t cut, float scale, hipStream_t stream) {
  constexpr int U = 2;
  const int64_t wg = (groups + 256 * U - 1) / (256 * U);
  hipLaunchKernelGGL((k_dropout<T, U>), dim3((unsigned)std::min<int64_t>(wg, 1 << 20)), dim3(256), 0,
                     stream, static_cast<const T*>(src), static_cast<const T*>(residual), rng,
                     static_cast<T*>(dst), groups, cut, scale);
}

// Calls f(W, CU) as types of the kernels' choice for rows of hv groups.
template <int N> using Int = std::integral_constant<int, N>;
template <typename F>
static void with_shape(int hv, F f) {
  if (hv <= kWave) f(Int<1>{}, Int<1>{});
  else if (hv <= 2 * kWave) f(Int<1>{}, Int<2>{});
  else if (hv <= 4 * kWave) f(Int<4>{}, Int<1>{});
  else if (hv <= 8 * kWave) f(Int<4>{}, Int<2>{});
  else f(Int<4>{}, Int<4>{});
}

template <typename T>
static void run_combine(const moe_cfg* c, const moe_plan* plan, const moe_bf16* y,
                        const float* gates, const void* residual, const int64_t* rng, void* out,
                        uint32_t cut, float scale, hipStream_t stream) {
  const int ntok = c->R * c->S;
  with_shape(c->Hp / 8, [&](auto W, auto CU) {
    hipLaunchKernelGGL((k_combine_drop<T, CU(), 4, W()>), dim3(W() == 1 ? (ntok + 3) / 4 : ntok),
                       dim3(256), 0, stream, reinterpret_cast<const u32x4*>(y), gates, plan->route,
                       static_cast<const T*>(residual), rng, static_cast<T*>(out), ntok, c->K,
                       c->Hp / 8, cut, scale);
  });
}

template <typename T>
static void run_combine_bwd(const moe_cfg* c, const moe_plan* plan, const void* dout,
                            const moe_bf16* y, const float* gates, const int64_t* rng, moe_bf16* dy,
                            float* dgates, uint32_t cut, float scale, hipStream_t stream) {
  const int ntok = c->R * c->S;
  with_shape(c->Hp / 8, [&](auto W, auto CU) {
    hipLaunchKernelGGL((k_combine_drop_bwd<T, CU(), 4, W()>),
                       dim3(W() == 1 ? (ntok + 3) / 4 : ntok), dim3(256), 0, stream,
                       static_cast<const T*>(dout), reinterpret_cast<const u32x4*>(y), gates,
                       plan->route, rng, reinterpret_cast<u32x4*>(dy), dgates, ntok, c->K,
                       c->Hp / 8, cut, scale);
  });
}

}  // namespace moonep

using namespace moonep;

extern "C" int moe_dropout(const moe_dropout_cfg* dc, int64_t rows, int32_t width, const void* src,
                           const void* residual, const int64_t* rng, void* dst,
                           hipStream_t stream) {
  uint32_t cut;
  float scale;
  if (!valid_dropout(dc, &cut, &scale)) return MOE_EINVAL;
  if (rows < 0 || width < 8 || width % 8 != 0) return MOE_EINVAL;
  if (rows > ((int64_t(1) << 40) - 1) / width) return MOE_ELIMIT;
  if (rows == 0) return MOE_OK;
  if (!src || !dst || !rng_ok(rng, cut) || !aligned16(src, residual, dst)) return MOE_EINVAL;
  const int64_t bytes = rows * width * (dc->f32 ? 4 : 2);
  if (clash({{dst, bytes}}, {{dst == src ? nullptr : src, bytes},
                             {dst == residual ? nullptr : residual, bytes},
                             {cut ? rng : nullptr, 16}}))
    return MOE_EINVAL;
  const int64_t groups = rows * (width / 8);
  if (dc->f32) run_dropout<float>(src, residual, rng, dst, groups, cut, scale, stream);
  else run_dropout<uint16_t>(src, residual, rng, dst, groups, cut, scale, stream);
  return hip_status();
}

extern "C" int moe_combine_dropout(const moe_cfg* cfg, const moe_dropout_cfg* dc,
                                   const moe_plan* plan, const moe_bf16* y, const float* gates,
                                   const void* residual, const int64_t* rng, void* out,
                                   hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  uint32_t cut;
  float scale;
  if (!valid_dropout(dc, &cut, &scale)) return MOE_EINVAL;
  const int64_t ntok = int64_t(cfg->R) * cfg->S, rows = ntok * cfg->K;
  if (ntok == 0) return MOE_OK;
  if (!plan || !plan->route || !y || !gates || !out || !rng_ok(rng, cut)) return MOE_EINVAL;
  if (!aligned16(y, residual, out)) return MOE_EINVAL;
  const int64_t bytes = ntok * cfg->Hp * (dc->f32 ? 4 : 2);
  if (clash({{out, bytes}}, {{y, rows * cfg->Hp * 2},
                             {gates, rows * 4},
                             {plan->route, rows * 4},
                             {residual == out ? nullptr : residual, bytes},
                             {cut ? rng : nullptr, 16}}))
    return MOE_EINVAL;
  const auto run = dc->f32 ? run_combine<float> : run_combine<uint16_t>;
  run(cfg, plan, y, gates, residual, rng, out, cut, scale, stream);
  return hip_status();
}

extern "C" int moe_combine_dropout_backward(const moe_cfg* cfg, const moe_dropout_cfg* dc,
                                            const moe_plan* plan, const void* dout,
                                            const moe_bf16* y, const float* gates,
                                            const int64_t* rng, moe_bf16* dy, float* dgates,
                                            hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  uint32_t cut;
  float scale;
  if (!valid_dropout(dc, &cut, &scale)) return MOE_EINVAL;
  const int64_t ntok = int64_t(cfg->R) * cfg->S, rows = ntok * cfg->K;
  if (ntok == 0) return MOE_OK;
  if (!plan || !plan->route || !dout || !y || !gates || !dy || !dgates || !rng_ok(rng, cut))
    return MOE_EINVAL;
  if (!aligned16(dout, y, dy)) return MOE_EINVAL;
  if (clash({{dy, rows * cfg->Hp * 2}, {dgates, rows * 4}},
            {{dout, ntok * cfg->Hp * (dc->f32 ? 4 : 2)},
             {y, rows * cfg->Hp * 2},
             {dgates == gates ? nullptr : gates, rows * 4},
             {plan->route, rows * 4},
             {cut ? rng : nullptr, 16}}) ||
      overlap(dy, rows * cfg->Hp * 2, gates, rows * 4))
    return MOE_EINVAL;
  const auto run = dc->f32 ? run_combine_bwd<float> : run_combine_bwd<uint16_t>;
  run(cfg, plan, dout, y, gates, rng, dy, dgates, cut, scale, stream);
  return hip_status();
}
