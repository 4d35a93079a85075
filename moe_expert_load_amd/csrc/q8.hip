// Activation checkpoints in 8 bits and their use in the backward: rows to
// codes and back, the dispatch redone from the layer input's codes, and the
// backward of the SwiGLU activation and of combine from the codes of h13 and
// of y.  The format is in q8.hpp.  All of them stream: what they cost is the
// bytes of their tensors.
#include <algorithm>

#include "convert.hpp"
#include "overlap.hpp"
#include "host.hpp"
#include "q8.hpp"

namespace moonep {

constexpr int kQ8Threads = 256;
constexpr int kQ8Unroll = 4;                       // vectors of 8 values per thread
constexpr int kQ8Tile = kQ8Threads * kQ8Unroll;

// Where vector x of a tile lies.  Rows are padded to whole blocks (hvp vectors
// of which hv exist), so a block's four vectors are adjacent lanes of a wave.
struct Q8Place {
  int64_t row;
  int c;          // vector within the row
  bool real;      // not padding, not past the last row
};

template <bool FLAT>
__device__ __forceinline__ Q8Place q8_place(int64_t tile, int x, int64_t rows, int hv, int hvp) {
  Q8Place p;
  if constexpr (FLAT) {                            // hv == hvp: one row of rows * hv vectors
    p.row = 0;
    p.c = 0;
    p.real = tile * kQ8Tile + x < rows * hv;
  } else {
    const int64_t v0 = tile * kQ8Tile;
    const int64_t r0 = v0 / hvp;
    const uint32_t off = (uint32_t)(v0 - r0 * hvp) + (uint32_t)x;
    const uint32_t dr = off / (uint32_t)hvp;
    p.row = r0 + dr;
    p.c = (int)(off - dr * (uint32_t)hvp);
    p.real = p.row < rows && p.c < hv;
  }
  return p;
}

// Every value is read once and every code written once, past the caches:
// 0.507 ms for 524,288 rows of 2,048 values against 0.564 ms through them
// (6.4 TB/s; a device copy reaches 4.8, a fill 6.9).
template <bool FLAT>
__global__ __launch_bounds__(kQ8Threads) void k_q8_store(const u32x4* __restrict__ src,
                                                         q8_u32x2* __restrict__ q,
                                                         uint8_t* __restrict__ scale, int64_t rows,
                                                         int hv, int hvp) {
  const int64_t tile = blockIdx.x;
  u32x4 v[kQ8Unroll];
  int64_t at[kQ8Unroll], sat[kQ8Unroll];
  bool real[kQ8Unroll];
#pragma unroll
  for (int u = 0; u < kQ8Unroll; ++u) {
    const int x = u * kQ8Threads + threadIdx.x;
    const Q8Place p = q8_place<FLAT>(tile, x, rows, hv, hvp);
    real[u] = p.real;
    at[u] = FLAT ? tile * kQ8Tile + x : p.row * hv + p.c;
    sat[u] = FLAT ? at[u] >> 2 : p.row * (hvp >> 2) + (p.c >> 2);
    v[u] = p.real ? __builtin_nontemporal_load(src + at[u]) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int u = 0; u < kQ8Unroll; ++u) {
    const uint32_t b = q8_scale_byte(q8_group_max(q8_top(v[u])));
    const q8_u32x2 w = q8_encode(v[u], b);
    if (real[u]) {
      __builtin_nontemporal_store(w, q + at[u]);
      // a block's first vector always exists where one of its vectors does
      if ((threadIdx.x & 3) == 0) scale[sat[u]] = (uint8_t)b;
    }
  }
}

// 524,288 rows of 2,048 values in 0.549 ms, 5.9 TB/s (65,536 of 7,168 in 0.240).
template <bool FLAT>
__global__ __launch_bounds__(kQ8Threads) void k_q8_load(const q8_u32x2* __restrict__ q,
                                                        const uint8_t* __restrict__ scale,
                                                        u32x4* __restrict__ dst, int64_t rows,
                                                        int hv, int hvp) {
  const int64_t tile = blockIdx.x;
#pragma unroll
  for (int u = 0; u < kQ8Unroll; ++u) {
    const int x = u * kQ8Threads + threadIdx.x;
    const Q8Place p = q8_place<FLAT>(tile, x, rows, hv, hvp);
    const int64_t at = FLAT ? tile * kQ8Tile + x : p.row * hv + p.c;
    const int64_t sat = FLAT ? at >> 2 : p.row * (hvp >> 2) + (p.c >> 2);
    if (p.real) dst[at] = q8_decode_bf16(q[at], scale[sat]);
  }
}

// Dispatch from codes: one workgroup per token, its row decoded once and
// written to each of its K places.  Bound by the writes of scattered rows, as
// the dispatch of bf16 rows is: 65,536 rows of 7,168 to 8 places in 1.50 ms,
// 5.35 TB/s (non-temporal stores: 1.54 ms).
template <int Q>
__global__ __launch_bounds__(256) void k_dispatch_q8(const q8_u32x2* __restrict__ xq,
                                                     const uint8_t* __restrict__ xs,
                                                     u32x4* __restrict__ xperm,
                                                     const int32_t* __restrict__ route, int K,
                                                     int hv) {
  const int t = blockIdx.x;
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int myroute = lane < K ? route[int64_t(t) * K + lane] : -1;
  const q8_u32x2* src = xq + int64_t(t) * hv;
  const uint8_t* sc = xs + int64_t(t) * ((hv + 3) >> 2);
  for (int c0 = w * kWave * Q; c0 < hv; c0 += 4 * kWave * Q) {
    u32x4 v[Q];
#pragma unroll
    for (int u = 0; u < Q; ++u) {
      const int c = c0 + u * kWave + lane;
      if (c < hv) v[u] = q8_decode_bf16(src[c], sc[c >> 2]);
    }
    // each token starts at its own k, as in the dispatch of bf16 rows
    for (int kk = 0; kk < K; ++kk) {
      const int dst = wave_bcast(myroute, (kk + t) % K);
      if (dst < 0) continue;
      u32x4* d = xperm + int64_t(dst) * hv;
#pragma unroll
      for (int u = 0; u < Q; ++u) {
        const int c = c0 + u * kWave + lane;
        if (c < hv) d[c] = v[u];
      }
    }
  }
}

// Backward of act = silu(gate) * up from the codes of h13, with s = 1 / (1 + e^-gate):
//   d gate = d act * up * s * (1 + gate * (1 - s)),  d up = d act * gate * s,
// and act = gate * s * up again for the second projection's weight gradient.
// One workgroup per row; 65,536 rows of 2 x 2,048 in 0.209 ms, 6.5 TB/s (two
// thirds of it writes).  From bf16 h13, without act: 0.236 ms.  Rows below 64
// vectors share a workgroup: 262,144 of 2 x 256 values take 121 us, 196 with one
// each; wider ones do not gain (2 x 512: 231 and 226, 2 x 1,024: 460 and 431).
__global__ __launch_bounds__(kQ8Threads) void k_swiglu_bwd_q8(const q8_u32x2* __restrict__ hq,
                                                              const uint8_t* __restrict__ hs,
                                                              const u32x4* dact, u32x4* dh13,
                                                              u32x4* act,       // may be dact
                                                              int64_t rows, int hv, int per) {
  const int sb = (hv + 3) >> 2;                    // scale bytes of one half row
  const int sub = per > 1 ? (int)threadIdx.x / hv : 0;
  const int first = (int)threadIdx.x - sub * hv;
  if (sub >= per) return;
  for (int64_t r = int64_t(blockIdx.x) * per + sub; r < rows; r += int64_t(gridDim.x) * per) {
    const q8_u32x2* gq = hq + r * 2 * hv;
    const uint8_t* gs = hs + r * 2 * sb;
    for (int c = first; c < hv; c += kQ8Threads) {
      const u32x4 dw = dact[r * hv + c];
      float g[8], x[8];
      q8_decode(gq[c], gs[c >> 2], g);
      q8_decode(gq[hv + c], gs[sb + (c >> 2)], x);
      u32x4 og, ou, oa;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float dg[2], du[2], a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float gate = g[2 * q + i], up = x[2 * q + i];
          const float d = i ? bf16_hi(dw[q]) : bf16_lo(dw[q]);
          const float s = __builtin_amdgcn_rcpf(1.f + __expf(-gate));
          const float gs1 = gate * s;
          du[i] = d * gs1;
          dg[i] = d * up * s * (1.f + gate * (1.f - s));
          a[i] = gs1 * up;
        }
        og[q] = cvt_bf16x2(dg[0], dg[1]);
        ou[q] = cvt_bf16x2(du[0], du[1]);
        oa[q] = cvt_bf16x2(a[0], a[1]);
      }
      dh13[r * 2 * hv + c] = og;
      dh13[r * 2 * hv + hv + c] = ou;
      if (act) act[r * hv + c] = oa;
    }
  }
}

// Backward of combine from the codes of y: W = 4 waves, or 1, per token,
//   dy[route_k] = g_k * dout[t],  dgates[t, k] = sum_h dout[t, h] * y[route_k, h].
// Thread i takes vectors i + 64 W u of the row.  The codes of KB routes are in
// flight before the first is used; each wave sums its part of their KB dots,
// and the four waves' parts are added in LDS, pass after pass.  Bound by the
// scattered rows: 524,288 of 2,048 values in 0.70 ms, 5.0 TB/s (4 routes in
// flight: 0.71, 2: 0.76), of 7,168 in 2.57 ms, 4.8 TB/s.  One wave takes rows of
// up to 128 vectors, whose workgroups have too few loads in flight: 262,144 of 512
// values in 81 us, 1,024 in 189, against 220 and 232 with four waves; of 2,048 both
// take 0.70 ms.
template <int W, int CU, int KB>
__global__ __launch_bounds__(256) void k_combine_bwd_q8(const u32x4* __restrict__ dout,
                                                        const q8_u32x2* __restrict__ yq,
                                                        const uint8_t* __restrict__ ys,
                                                        const float* __restrict__ gates,
                                                        const int32_t* __restrict__ route,
                                                        u32x4* __restrict__ dy,
                                                        float* __restrict__ dgates, int ntok,
                                                        int K, int hv) {
  constexpr int NT = W * kWave;                         // threads of a token
  static_assert(W == 1 || W == 4);
  __shared__ float s_dot[W][MOE_MAX_K];
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = W == 1 ? (int)blockIdx.x * 4 + wv : (int)blockIdx.x;
  const int tid = W == 1 ? lane : (int)threadIdx.x;     // within the token
  if (W == 1 && t >= ntok) return;
  const int sb = (hv + 3) >> 2;
  const int myroute = lane < K ? route[int64_t(t) * K + lane] : -1;
  const float mygate = lane < K ? gates[int64_t(t) * K + lane] : 0.f;
  float mydot = 0.f;                                    // lane k: this wave's part of k's dot
  for (int c0 = 0; c0 < hv; c0 += NT * CU) {
    u32x4 d[CU];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      const int c = c0 + u * NT + tid;
      d[u] = c < hv ? __builtin_nontemporal_load(dout + int64_t(t) * hv + c) : u32x4{0, 0, 0, 0};
    }
    for (int k0 = 0; k0 < K; k0 += KB) {
      q8_u32x2 v[KB][CU];
      uint32_t b[KB][CU];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int src = wave_bcast(myroute, min(k0 + kb, K - 1));
        const bool ok = k0 + kb < K && src >= 0;
        const int64_t r = ok ? src : 0;
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int c = c0 + u * NT + tid;
          v[kb][u] = q8_u32x2{0, 0};
          b[kb][u] = 127;
          if (ok && c < hv) {
            v[kb][u] = __builtin_nontemporal_load(yq + r * hv + c);
            b[kb][u] = ys[r * sb + (c >> 2)];
          }
        }
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if (k0 + kb >= K) break;                        // uniform
        const int dst = wave_bcast(myroute, k0 + kb);
        const float g = __int_as_float(wave_bcast(__float_as_int(mygate), k0 + kb));
        float part = 0.f;
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int c = c0 + u * NT + tid;
          float y[8];
          q8_decode(v[kb][u], b[kb][u], y);
          u32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float dl = bf16_lo(d[u][q]), dh = bf16_hi(d[u][q]);
            part = fmaf(dl, y[2 * q], part);
            part = fmaf(dh, y[2 * q + 1], part);
            o[q] = mul_to_bf16(g, dl) | (mul_to_bf16(g, dh) << 16);
          }
          if (dst >= 0 && c < hv) dy[int64_t(dst) * hv + c] = o;
        }
        const float s = wave_sum_f(part);
        if (lane == k0 + kb && dst >= 0) mydot += s;
      }
    }
  }
  if constexpr (W == 1) {
    if (lane < K) dgates[int64_t(t) * K + lane] = mydot;
  } else {
    if (lane < K) s_dot[wv][lane] = mydot;
    __syncthreads();
    if (tid < K)
      dgates[int64_t(t) * K + tid] = s_dot[0][tid] + s_dot[1][tid] + s_dot[2][tid] + s_dot[3][tid];
  }
}

// rows x width of moe_q8_store and moe_q8_load, and their grid of tiles.
inline int check_q8(int64_t rows, int32_t width, int64_t* tiles) {
  if (rows < 0 || width < 8 || width % 8 != 0) return MOE_EINVAL;
  const int64_t hvp = (int64_t(width) + kQ8Block - 1) / kQ8Block * 4;
  if (rows > ((int64_t(1) << 40) / hvp)) return MOE_ELIMIT;
  *tiles = (rows * hvp + kQ8Tile - 1) / kQ8Tile;
  // one 256-thread workgroup per tile, fewer than 2^32 threads in a launch
  return *tiles >= (int64_t(1) << 24) ? MOE_ELIMIT : MOE_OK;
}

// Whether bf16 rows share memory with their codes or scales, or those with each
// other: a workgroup would write what another has yet to read.
inline bool q8_overlap(int64_t rows, int hv, int hvp, const void* x, const void* q,
                       const void* scale) {
  const int64_t n = rows * hv * 8, ns = rows * (hvp / 4);
  return overlap(x, 2 * n, q, n) || overlap(x, 2 * n, scale, ns) || overlap(q, n, scale, ns);
}

}  // namespace moonep

using namespace moonep;

extern "C" int moe_q8_store(int64_t rows, int32_t width, const moe_bf16* src, uint8_t* q,
                            uint8_t* scale, hipStream_t stream) {
  int64_t tiles = 0;
  const int rc = check_q8(rows, width, &tiles);
  if (rc != MOE_OK) return rc;
  if (rows == 0) return MOE_OK;
  if (!src || !q || !scale || !aligned16(src, q)) return MOE_EINVAL;
  const int hv = width / 8, hvp = (hv + 3) / 4 * 4;
  if (q8_overlap(rows, hv, hvp, src, q, scale)) return MOE_EINVAL;
  const u32x4* s = reinterpret_cast<const u32x4*>(src);
  q8_u32x2* d = reinterpret_cast<q8_u32x2*>(q);
  const dim3 grid((unsigned)tiles), block(kQ8Threads);
  if (hv == hvp)
    hipLaunchKernelGGL(k_q8_store<true>, grid, block, 0, stream, s, d, scale, rows, hv, hvp);
  else
    hipLaunchKernelGGL(k_q8_store<false>, grid, block, 0, stream, s, d, scale, rows, hv, hvp);
  return hip_status();
}

extern "C" int moe_q8_load(int64_t rows, int32_t width, const uint8_t* q, const uint8_t* scale,
                           moe_bf16* dst, hipStream_t stream) {
  int64_t tiles = 0;
  const int rc = check_q8(rows, width, &tiles);
  if (rc != MOE_OK) return rc;
  if (rows == 0) return MOE_OK;
  if (!dst || !q || !scale || !aligned16(dst, q)) return MOE_EINVAL;
  const int hv = width / 8, hvp = (hv + 3) / 4 * 4;
  if (q8_overlap(rows, hv, hvp, dst, q, scale)) return MOE_EINVAL;
  const q8_u32x2* s = reinterpret_cast<const q8_u32x2*>(q);
  u32x4* d = reinterpret_cast<u32x4*>(dst);
  const dim3 grid((unsigned)tiles), block(kQ8Threads);
  if (hv == hvp)
    hipLaunchKernelGGL(k_q8_load<true>, grid, block, 0, stream, s, scale, d, rows, hv, hvp);
  else
    hipLaunchKernelGGL(k_q8_load<false>, grid, block, 0, stream, s, scale, d, rows, hv, hvp);
  return hip_status();
}

extern "C" int moe_dispatch_q8(const moe_cfg* cfg, const moe_plan* plan, const uint8_t* xq,
                               const uint8_t* xscale, moe_bf16* xperm, hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  const int ntok = cfg->R * cfg->S;
  if (ntok == 0) return MOE_OK;
  if (!plan || !plan->route || !xq || !xscale || !xperm) return MOE_EINVAL;
  if (!aligned16(xq, xperm)) return MOE_EINVAL;
  const int hv = cfg->H / 8;
  const int64_t n = int64_t(ntok) * cfg->H;
  if (clash({{xperm, 2 * n * cfg->K}}, {{xq, n}, {xscale, int64_t(ntok) * ((hv + 3) / 4)}}))
    return MOE_EINVAL;
  const int q = (hv + 4 * kWave - 1) / (4 * kWave);
  const dim3 grid(ntok), block(256);
  const q8_u32x2* xs = reinterpret_cast<const q8_u32x2*>(xq);
  u32x4* xd = reinterpret_cast<u32x4*>(xperm);
#define MOE_DISPATCH(N)                                                                        \
  hipLaunchKernelGGL(k_dispatch_q8<N>, grid, block, 0, stream, xs, xscale, xd, plan->route, \
                     cfg->K, hv)
  if (q <= 1) MOE_DISPATCH(1);
  else if (q <= 2) MOE_DISPATCH(2);
  else MOE_DISPATCH(4);                                // larger rows take several passes
#undef MOE_DISPATCH
  return hip_status();
}

extern "C" int moe_swiglu_backward_q8(const moe_cfg* cfg, const uint8_t* h13q,
                                      const uint8_t* h13scale, const moe_bf16* dact,
                                      moe_bf16* dh13, moe_bf16* act, hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  const int64_t rows = int64_t(cfg->R) * cfg->S * cfg->K;
  if (rows == 0) return MOE_OK;
  if (!h13q || !h13scale || !dact || !dh13) return MOE_EINVAL;
  if (!aligned16(h13q) || !aligned16(dact, dh13, act)) return MOE_EINVAL;
  const int64_t n = rows * cfg->Hp, ns = 2 * rows * ((cfg->Hp + kQ8Block - 1) / kQ8Block);
  if (overlap(dh13, 4 * n, h13q, 2 * n) || overlap(dh13, 4 * n, h13scale, ns) ||
      overlap(dh13, 4 * n, dact, 2 * n) || overlap(dh13, 4 * n, act, 2 * n) ||
      overlap(act, 2 * n, h13q, 2 * n) || overlap(act, 2 * n, h13scale, ns) ||
      (act != dact && overlap(act, 2 * n, dact, 2 * n)))
    return MOE_EINVAL;
  const int hv = cfg->Hp / 8;
  const int per = hv < kWave ? kQ8Threads / hv : 1;               // rows of a workgroup
  const int64_t grid = std::min<int64_t>((rows + per - 1) / per, int64_t(1) << 20);
  hipLaunchKernelGGL(k_swiglu_bwd_q8, dim3((unsigned)grid), dim3(kQ8Threads), 0, stream,
                     reinterpret_cast<const q8_u32x2*>(h13q), h13scale,
                     reinterpret_cast<const u32x4*>(dact), reinterpret_cast<u32x4*>(dh13),
                     reinterpret_cast<u32x4*>(act), rows, hv, per);
  return hip_status();
}

extern "C" int moe_combine_backward_q8(const moe_cfg* cfg, const moe_plan* plan,
                                       const moe_bf16* dout, const uint8_t* yq,
                                       const uint8_t* yscale, const float* gates, moe_bf16* dy,
                                       float* dgates, hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  const int ntok = cfg->R * cfg->S;
  if (ntok == 0) return MOE_OK;
  if (!plan || !plan->route || !dout || !yq || !yscale || !gates || !dy || !dgates)
    return MOE_EINVAL;
  if (!aligned16(dout, dy) || !aligned16(yq) || !aligned16(gates, dgates)) return MOE_EINVAL;
  const int hv = cfg->Hp / 8;
  const int64_t rows = int64_t(ntok) * cfg->K, n = rows * cfg->Hp;
  const Range in[] = {{dout, 2 * int64_t(ntok) * cfg->Hp}, {yq, n}, {yscale, rows * ((hv + 3) / 4)}};
  // a token's gates are read before its dgates are written: in place is fine
  if (clash({{dy, 2 * n}, {dgates, 4 * rows}}, in) || overlap(dy, 2 * n, gates, 4 * rows) ||
      (dgates != gates && overlap(dgates, 4 * rows, gates, 4 * rows)))
    return MOE_EINVAL;
  const dim3 block(256);
  const u32x4* ds = reinterpret_cast<const u32x4*>(dout);
  const q8_u32x2* ysrc = reinterpret_cast<const q8_u32x2*>(yq);
  u32x4* dd = reinterpret_cast<u32x4*>(dy);
#define MOE_COMBINE_BWD(W, N)                                                                  \
  hipLaunchKernelGGL((k_combine_bwd_q8<W, N, 8>), dim3(W == 1 ? (ntok + 3) / 4 : ntok), block, 0, \
                     stream, ds, ysrc, yscale, gates, plan->route, dd, dgates, ntok, cfg->K, hv)
  if (hv <= 64) MOE_COMBINE_BWD(1, 1);
  else if (hv <= 128) MOE_COMBINE_BWD(1, 2);
  else if (hv <= 256) MOE_COMBINE_BWD(4, 1);
  else MOE_COMBINE_BWD(4, 2);                          // larger rows take several passes
#undef MOE_COMBINE_BWD
  return hip_status();
}
