// Router: the join of the loss's sums, the backward kernels and the entry
// points.  The formulas, the row layout and the forward are in router.hpp.
#include <algorithm>

#include "overlap.hpp"
#include "router.hpp"

namespace moonep {

// Joins a sequence's rows into counts, P and the loss, in a fixed order.
// k_router_join<true>: one workgroup has all `ns` slices of 64 experts of a
// sequence and writes the results.  k_router_join<false>: a workgroup has one
// slice and one of gridDim.z parts of the rows, and writes sums that
// k_router_total adds up.  Its 16 waves are 16 / ns groups that take the rows in
// turn, eight loads in flight each.  One sequence of 65,536 tokens of 384
// experts: 4.4 us and 2.5 for the total, against 123 in one workgroup and 8.7
// without the parts.
constexpr int kJoinThreads = 1024;
constexpr int kJoinWaves = kJoinThreads / kWave;

template <int N>
__device__ __forceinline__ void join_rows(const RouterArgs& a, int64_t at, int64_t stride, int n,
                                          double& p, int& c) {
  float fp[N];
  int fc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {                   // all loads go out before the first sum
    const int64_t x = at + min(j, n - 1) * stride;
    fp[j] = a.part_p[x];
    fc[j] = a.part_c[x];
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    p += j < n ? (double)fp[j] : 0.0;
    c += j < n ? fc[j] : 0;
  }
}

template <bool ONE>
__global__ __launch_bounds__(kJoinThreads) void k_router_join(RouterArgs a, int chunks, int ns,
                                                              int32_t* counts, float* prob,
                                                              float* loss) {
  __shared__ double s_p[kJoinWaves][kWave];
  __shared__ int s_c[kJoinWaves][kWave];
  const int seq = blockIdx.x, lane = lane_id(), wv = threadIdx.x / kWave;
  const int groups = kJoinWaves / ns, slice = wv % ns, group = wv / ns;
  const int lo = a.cu ? max(0, min(a.cu[seq], a.T)) : 0;
  const int hi = a.cu ? max(lo, min(a.cu[seq + 1], a.T)) : a.T;
  int c0 = hi > lo ? lo / a.chunk : 0, c1 = hi > lo ? min((hi - 1) / a.chunk + 1, chunks) : 0;
  if constexpr (!ONE) {
    const int part = (c1 - c0 + (int)gridDim.z - 1) / (int)gridDim.z;
    c0 += (int)blockIdx.z * part;
    c1 = min(c1, c0 + part);
  }
  const int e = (blockIdx.y * ns + slice) * kWave + lane;
  double p = 0.0;
  int c = 0;
  if (e < a.E && group < groups) {
    const int64_t stride = int64_t(groups) * a.E;
    for (int r = c0 + group; r < c1; r += 8 * groups) {
      const int64_t at = int64_t(r + seq) * a.E + e;
      const int n = (c1 - r + groups - 1) / groups;
      if (n > 2) join_rows<8>(a, at, stride, n, p, c);
      else join_rows<2>(a, at, stride, n, p, c);
    }
  }
  s_p[wv][lane] = p;
  s_c[wv][lane] = c;
  __syncthreads();
  double f = 0.0;
  if (group == 0 && e < a.E) {
#pragma unroll
    for (int g = 1; g < kJoinWaves; ++g) {        // LDS reads without a wait between them
      const int w = min(g * ns + slice, kJoinWaves - 1);
      const double gp = s_p[w][lane];
      const int gc = s_c[w][lane];
      p += g < groups ? gp : 0.0;
      c += g < groups ? gc : 0;
    }
    if constexpr (ONE) {
      const float mean = hi > lo ? (float)(p / (double)(hi - lo)) : 0.f;
      counts[int64_t(seq) * a.E + e] = c;
      prob[int64_t(seq) * a.E + e] = mean;
      f = (double)c * (double)mean;
    } else {
      const int64_t at = (int64_t(seq) * gridDim.z + blockIdx.z) * a.E + e;
      a.sum_p[at] = p;
      a.sum_c[at] = c;
    }
  }
  if constexpr (ONE) {
    __syncthreads();
    f = wave_sum_d(f);
    if (lane == 0) s_p[wv][0] = f;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < ns; ++w) f += s_p[w][0];
      loss[seq] = hi > lo ? (float)(f * a.E / ((double)a.K * (hi - lo))) : 0.f;
    }
  }
}

// A sequence's results from its Z parts' sums.
constexpr int kTotalThreads = 512;

template <int Z>
__global__ __launch_bounds__(kTotalThreads) void k_router_total(RouterArgs a, int32_t* counts,
                                                                float* prob, float* loss) {
  __shared__ double s_f[kTotalThreads / kWave];
  const int seq = blockIdx.x;
  const int lo = a.cu ? max(0, min(a.cu[seq], a.T)) : 0;
  const int hi = a.cu ? max(lo, min(a.cu[seq + 1], a.T)) : a.T;
  double f = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kTotalThreads) {
    const int64_t at = int64_t(seq) * Z * a.E + e;
    double p = 0.0;
    int c = 0;
#pragma unroll
    for (int z = 0; z < Z; ++z) {
      p += a.sum_p[at + int64_t(z) * a.E];
      c += a.sum_c[at + int64_t(z) * a.E];
    }
    const float mean = hi > lo ? (float)(p / (double)(hi - lo)) : 0.f;
    counts[int64_t(seq) * a.E + e] = c;
    prob[int64_t(seq) * a.E + e] = mean;
    f += (double)c * (double)mean;
  }
  f = wave_sum_d(f);
  if (lane_id() == 0) s_f[threadIdx.x / kWave] = f;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kTotalThreads / kWave; ++w) f += s_f[w];
    loss[seq] = hi > lo ? (float)(f * a.E / ((double)a.K * (hi - lo))) : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Backward.  A wave owns `chunk` consecutive tokens and keeps the loss's
// coefficient of every expert of the current sequence in registers,
//   u_e = dloss E c_e / (K L^2).
// With p' the softmax or the sigmoid's shares,
//   softmax  dz = p (u - sum u p),  sigmoid  dz = p (1 - s) (u - sum u p);
// the gates add, at the chosen experts only and with w_k = gate / scale,
//   softmax, not renormalised  scale dg_k joins u at the expert,
//   renormalised               scale w_k (dg_k - sum dg w) (1 - s_k for sigmoid),
//   sigmoid, not renormalised  scale dg_k s_k (1 - s_k).
// These K values reach the lanes that hold their experts through an LDS row.
//
// It streams: 65,536 fp32 tokens of 384 experts in 40 us (logits in, dlogits
// out: 5.0 TB/s), 262,144 bf16 tokens of 896 in 181 us (5.2 TB/s; a device copy
// reaches 4.8-4.9).  Five waves a SIMD for rows of 9 to 14 registers cost a few
// spills and hide more: 181 us against 198 with four, 294 with six.
// A gradient of renormalised gates alone reads only the K chosen logits.
// ---------------------------------------------------------------------------
template <int P, bool BF16, bool FULL, bool SOFT>
__global__ __launch_bounds__(kRtThreads, P > 8 && P <= 14 ? 5 : 1) void k_router_bwd(RouterArgs a) {
  extern __shared__ float lds[];                  // [waves][64 P]
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int E = a.E, K = a.K;
  float* row = lds + wv * (64 * P);
  const bool balance = a.dloss != nullptr, gates = a.dgates != nullptr;
  const bool into_u = SOFT && gates && !a.renorm;         // the gates' part goes through p
  if (gates) {
#pragma unroll
    for (int i = 0; i < P; i += 2) *reinterpret_cast<float2*>(row + expert_of(i)) = float2{0, 0};
  }
  const int64_t w0 = (int64_t(blockIdx.x) * kRtWaves + wv) * a.chunk;
  const int t0 = (int)min<int64_t>(w0, a.T), t1 = (int)min<int64_t>(w0 + a.chunk, a.T);
  if (t0 >= t1) return;
  const bool rows = balance || into_u;
  Row<P, BF16> next;
  int next_id = -1;
  float next_dg = 0.f;
  if (rows) load_row<P, BF16, FULL>(a.logits, t0, E, next);
  if (gates && lane < K) {
    next_id = a.ids[int64_t(t0) * K + lane];
    next_dg = a.dgates[int64_t(t0) * K + lane];
  }
  int end = t0, seq = -1;
  float u[P];
#pragma unroll
  for (int i = 0; i < P; ++i) u[i] = 0.f;
  for (int t = t0; t < t1; ++t) {
    float v[P], co[P], dz[P];
    float shift = 0.f, inv = 1.f;
    if (rows) {
      float z[P];
      unpack_row<P, BF16, FULL>(next, E, z);
      if (t + 1 < t1) load_row<P, BF16, FULL>(a.logits, t + 1, E, next);
      inv = row_shares<P, BF16, FULL, SOFT, !SOFT>(a, t, z, v, co, shift);
    }
    const int id = next_id;
    const bool on = (unsigned)id < (unsigned)E;
    float dg = on ? a.scale * next_dg : 0.f;
    if (gates && lane < K && t + 1 < t1) {
      next_id = a.ids[int64_t(t + 1) * K + lane];
      next_dg = a.dgates[int64_t(t + 1) * K + lane];
    }
    if (balance && t >= end) {
      seq = sequence_of(a, t, end);
      float c0 = 0.f;
      if (seq >= 0) {
        const int lo = a.cu ? a.cu[seq] : 0;
        const float len = (float)max(1, (a.cu ? a.cu[seq + 1] : a.T) - lo);
        c0 = a.dloss[seq] * (float)E / ((float)K * len) / len;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = expert_of(i);
        u[i] = seq >= 0 && e < E ? c0 * (float)a.counts[int64_t(seq) * E + e] : 0.f;
      }
    }
    if (gates) {
      if (!into_u) {
        const float zk = on ? logit_at<BF16>(a.logits, int64_t(t) * E + id) : 0.f;
        const float w = gate_share<SOFT>(zk, on, a.renorm, shift, inv);
        dg = w * (dg - (a.renorm ? wave_sum_f(dg * w) : 0.f));
        if constexpr (!SOFT) {
          float c;
          sigmoid_f(zk, c);
          dg *= c;
        }
      }
      if (on) atomicAdd(&row[id], dg);
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float2 g = *reinterpret_cast<const float2*>(row + expert_of(i));
        dz[i] = g.x;
        dz[i + 1] = g.y;
      }
      wave_lds_fence();
      if (on) row[id] = 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) dz[i] = 0.f;
    }
    if (into_u || (balance && seq >= 0)) {        // a row of no sequence may hold anything
      float mean = 0.f;
      if (into_u) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dz[i] += u[i];
          mean = fmaf(dz[i], v[i], mean);
        }
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) mean = fmaf(u[i], v[i], mean);
      }
      mean = wave_sum_f(mean) * inv;
      if (into_u) {
#pragma unroll
        for (int i = 0; i < P; ++i) dz[i] = v[i] * inv * (dz[i] - mean);
      } else if constexpr (SOFT) {
#pragma unroll
        for (int i = 0; i < P; ++i) dz[i] = fmaf(v[i] * inv, u[i] - mean, dz[i]);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) dz[i] = fmaf(v[i] * inv * co[i], u[i] - mean, dz[i]);
      }
    }
    const int64_t at = int64_t(t) * E;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const int e = expert_of(i);
      const bool sure = FULL || i < kSure<P>;
      if (FULL || (E & 1) == 0) {
        if (sure || e < E) {
          if constexpr (BF16)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.dlogits) + at + e) =
                cvt_bf16x2(dz[i], dz[i + 1]);
          else
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.dlogits) + at + e) =
                float2{dz[i], dz[i + 1]};
        }
      } else {
        const uint32_t w = BF16 ? cvt_bf16x2(dz[i], dz[i + 1]) : 0u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (sure || e + j < E) {
            if constexpr (BF16)
              reinterpret_cast<uint16_t*>(a.dlogits)[at + e + j] = (uint16_t)(w >> (16 * j));
            else
              reinterpret_cast<float*>(a.dlogits)[at + e + j] = dz[i + j];
          }
        }
      }
    }
  }
}

// Tokens per workgroup of a forward call of at most `most` workgroups: whole
// rounds of its waves.
inline int chunk_for(int T, int most) {
  const int rounds = (T + most * kRtWaves - 1) / (most * kRtWaves);
  return kRtWaves * (rounds > 1 ? rounds : 1);
}
inline int chunks_of(int T, int chunk) { return (T + chunk - 1) / chunk; }
inline int max_chunks(int T) { return chunks_of(T, chunk_for(T, kRtMaxChunks)); }

// Rows times slices of experts up to which one workgroup joins a sequence: at
// 512 rows of one slice it takes 4-5 us, as k_router_join<false> does alone,
// and a launch of 2.5-4.8 us less follows.
constexpr int kJoinOne = 512;
// Sequences from which on one workgroup joins each, whatever its rows: with
// workgroups for its slices too, most have a row or two.  The loss of 65,536
// bf16 tokens of 896 experts takes 35 us for 512 sequences and 271 for 16,384
// (63 and 1,118 with slices); 89 against 66 if one of the 512 has half of them.
constexpr int kJoinMany = 512;

// Parts into which a sequence's rows are joined first: several where a sequence
// has 256 rows or more on average (fewer leave a wave one round of loads).
constexpr int kJoinParts = 8;
inline int join_parts(int T, int nseq) {
  return max_chunks(T) >= int64_t(256) * nseq ? kJoinParts : 1;
}

// Workspace: joined sums, then the rows' sums, then both counts.
inline size_t part_rows(int T, int nseq) { return size_t(max_chunks(T)) + size_t(nseq); }
inline size_t sum_rows(int T, int nseq) { return size_t(nseq) * join_parts(T, nseq); }

inline int check_router(const moe_cfg* c, const moe_router_cfg* r) {
  const int rc = check_cfg(c);
  if (rc != MOE_OK) return rc;
  if (!r) return MOE_EINVAL;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if ((unsigned)r->renormalize > 1u || (unsigned)r->logits_bf16 > 1u || r->nseq < 1)
    return MOE_EINVAL;
  if (r->nseq > MOE_MAX_NSEQ) return MOE_ELIMIT;
  return MOE_OK;
}

inline size_t router_ws_bytes(const moe_cfg* c, int nseq) {
  const int T = c->R * c->S;
  return align256((part_rows(T, nseq) * 8 + sum_rows(T, nseq) * 12) * c->E);
}

// Whether a forward call's outputs share memory with what it reads or each other.
// ids and gates are null where they are not written; loss is null without one.
inline bool forward_clash(const moe_cfg* c, const moe_router_cfg* r, const RouterArgs& a,
                          const int32_t* ids_in, const int32_t* counts, const float* prob,
                          const float* loss, const void* workspace) {
  const int64_t T = int64_t(c->R) * c->S, row = int64_t(r->nseq) * c->E * 4, k = T * c->K * 4;
  const int64_t ws = loss ? (int64_t)router_ws_bytes(c, r->nseq) : 0;
  return clash({{ids_in ? nullptr : a.ids, k}, {a.gates, k}, {counts, row}, {prob, row},
                {loss, int64_t(r->nseq) * 4}, {workspace, ws}},
               {{a.logits, T * c->E * (r->logits_bf16 ? 2 : 4)}, {a.bias, int64_t(c->E) * 4},
                {ids_in, k}, {loss ? a.cu : nullptr, (int64_t(r->nseq) + 1) * 4}});
}

inline int run_forward(const moe_cfg* c, const moe_router_cfg* r, RouterArgs a, bool select,
                       int32_t* counts, float* prob, float* loss, void* workspace,
                       hipStream_t stream) {
  const bool stats = loss != nullptr;
  a.T = c->R * c->S;
  a.E = c->E;
  a.K = c->K;
  a.nseq = r->nseq;
  a.score = r->score;
  a.renorm = r->renormalize;
  a.scale = r->scale;
  int chunks = 0;
  if (stats) {
    a.chunk = chunk_for(a.T, select ? kRtSelectChunks : kRtMaxChunks);
    chunks = chunks_of(a.T, a.chunk);
    const size_t rows = part_rows(a.T, a.nseq) * a.E, sums = sum_rows(a.T, a.nseq) * a.E;
    a.sum_p = reinterpret_cast<double*>(workspace);
    a.part_p = reinterpret_cast<float*>(a.sum_p + sums);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + rows);
    a.sum_c = a.part_c + rows;
  } else {
    a.chunk = chunk_for(a.T, a.bias ? kRtSelectChunks : kRtMaxChunks);
  }
  if (a.T > 0) {
    const int grid = stats ? chunks : (a.T + a.chunk - 1) / a.chunk;
    const int rc = r->score == MOE_SCORE_SOFTMAX
                       ? launch_forward<true>(a, r->logits_bf16, select, stats, grid, stream)
                       : launch_forward<false>(a, r->logits_bf16, select, stats, grid, stream);
    if (rc != MOE_OK) return rc;
  }
  if (stats) {
    const int slices = (a.E + kWave - 1) / kWave;
    const dim3 t(kJoinThreads);
    if (slices <= kJoinWaves && (chunks * slices <= kJoinOne || a.nseq >= kJoinMany)) {
      hipLaunchKernelGGL(k_router_join<true>, dim3(a.nseq), t, 0, stream, a, chunks, slices,
                         counts, prob, loss);
      return hip_status();
    }
    const int z = join_parts(a.T, a.nseq);
    hipLaunchKernelGGL(k_router_join<false>, dim3(a.nseq, slices, z), t, 0, stream, a, chunks, 1,
                       counts, prob, loss);
    if (z > 1)
      hipLaunchKernelGGL(k_router_total<kJoinParts>, dim3(a.nseq), dim3(kTotalThreads), 0, stream,
                         a, counts, prob, loss);
    else
      hipLaunchKernelGGL(k_router_total<1>, dim3(a.nseq), dim3(kTotalThreads), 0, stream, a,
                         counts, prob, loss);
    return hip_status();
  }
  return MOE_OK;
}

}  // namespace moonep

using namespace moonep;

extern "C" int moe_router_workspace_size(const moe_cfg* cfg, const moe_router_cfg* rcfg,
                                         size_t* bytes_out) {
  const int rc = check_router(cfg, rcfg);
  if (rc != MOE_OK) return rc;
  if (!bytes_out) return MOE_EINVAL;
  *bytes_out = router_ws_bytes(cfg, rcfg->nseq);
  return MOE_OK;
}

extern "C" int moe_router(const moe_cfg* cfg, const moe_router_cfg* rcfg, const void* logits,
                          const float* bias, int32_t* topk_ids, float* gates,
                          const int32_t* cu_tokens, int32_t* counts, float* prob, float* loss,
                          void* workspace, hipStream_t stream) {
  const int rc = check_router(cfg, rcfg);
  if (rc != MOE_OK) return rc;
  const bool stats = loss != nullptr;
  if ((counts != nullptr) != stats || (prob != nullptr) != stats) return MOE_EINVAL;
  if (stats && (!workspace || (!cu_tokens && rcfg->nseq != 1))) return MOE_EINVAL;
  if (cfg->S > 0 && (!logits || !topk_ids || !gates)) return MOE_EINVAL;
  if (!aligned16(logits) || !aligned16(bias, gates, prob, loss) || !aligned16(workspace))
    return MOE_EINVAL;
  RouterArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.gates = gates;
  a.cu = cu_tokens;
  if (forward_clash(cfg, rcfg, a, nullptr, counts, prob, loss, workspace)) return MOE_EINVAL;
  return run_forward(cfg, rcfg, a, true, counts, prob, loss, workspace, stream);
}

extern "C" int moe_balance_loss(const moe_cfg* cfg, const moe_router_cfg* rcfg, const void* logits,
                                const int32_t* topk_ids, const int32_t* cu_tokens, int32_t* counts,
                                float* prob, float* loss, void* workspace, hipStream_t stream) {
  const int rc = check_router(cfg, rcfg);
  if (rc != MOE_OK) return rc;
  if (!counts || !prob || !loss || !workspace) return MOE_EINVAL;
  if (!cu_tokens && rcfg->nseq != 1) return MOE_EINVAL;
  if (cfg->S > 0 && (!logits || !topk_ids)) return MOE_EINVAL;
  if (!aligned16(logits) || !aligned16(prob, loss) || !aligned16(workspace)) return MOE_EINVAL;
  RouterArgs a{};
  a.logits = logits;
  a.ids = const_cast<int32_t*>(topk_ids);
  a.cu = cu_tokens;
  if (forward_clash(cfg, rcfg, a, topk_ids, counts, prob, loss, workspace)) return MOE_EINVAL;
  return run_forward(cfg, rcfg, a, false, counts, prob, loss, workspace, stream);
}

extern "C" int moe_router_backward(const moe_cfg* cfg, const moe_router_cfg* rcfg,
                                   const void* logits, const int32_t* topk_ids,
                                   const float* dgates, const int32_t* cu_tokens,
                                   const int32_t* counts, const float* dloss, void* dlogits,
                                   hipStream_t stream) {
  const int rc = check_router(cfg, rcfg);
  if (rc != MOE_OK) return rc;
  if (cfg->S == 0) return MOE_OK;                 // empty tensors may be null
  if (!dgates && !dloss) return MOE_EINVAL;
  if (dloss && (!counts || (!cu_tokens && rcfg->nseq != 1))) return MOE_EINVAL;
  if (!logits || !dlogits || (dgates && !topk_ids)) return MOE_EINVAL;
  if (!aligned16(logits, static_cast<const void*>(dlogits)) || !aligned16(dgates, dloss))
    return MOE_EINVAL;
  const int64_t bytes = int64_t(cfg->R) * cfg->S * cfg->E * (rcfg->logits_bf16 ? 2 : 4);
  if (dlogits != logits && overlap(logits, bytes, dlogits, bytes)) return MOE_EINVAL;
  const int64_t k = int64_t(cfg->R) * cfg->S * cfg->K * 4, n = rcfg->nseq;
  if (clash({{dlogits, bytes}},
            {{dgates ? topk_ids : nullptr, k}, {dgates, k}, {dloss, n * 4},
             {dloss ? cu_tokens : nullptr, (n + 1) * 4},
             {dloss ? counts : nullptr, n * cfg->E * 4}}))
    return MOE_EINVAL;
  RouterArgs a{};
  a.logits = logits;
  a.ids = const_cast<int32_t*>(topk_ids);
  a.dgates = dgates;
  a.cu = cu_tokens;
  a.counts = counts;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.T = cfg->R * cfg->S;
  a.E = cfg->E;
  a.K = cfg->K;
  a.nseq = rcfg->nseq;
  a.score = rcfg->score;
  a.renorm = rcfg->renormalize;
  a.scale = rcfg->scale;
  a.chunk = std::max(1, std::min(8, a.T >> 13));
  const int per = kRtWaves * a.chunk;
  return with_row(a.E, rcfg->logits_bf16, [&](auto p, auto b, auto full) {
    constexpr int P = decltype(p)::value;
    const size_t lds = dgates ? size_t(kRtWaves) * 64 * P * 4 : 0;
    constexpr bool BF = decltype(b)::value, FULL = decltype(full)::value;
    const dim3 grid((a.T + per - 1) / per), block(kRtThreads);
    if (a.score == MOE_SCORE_SOFTMAX)
      hipLaunchKernelGGL((k_router_bwd<P, BF, FULL, true>), grid, block, lds, stream, a);
    else
      hipLaunchKernelGGL((k_router_bwd<P, BF, FULL, false>), grid, block, lds, stream, a);
    return hip_status();
  });
}
