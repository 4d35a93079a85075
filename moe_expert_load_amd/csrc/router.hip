// Router: expert scores to top-k ids and gates, the balance loss of every
// sequence with its per-expert counts, and the gradient of both by the logits.
//
// With z one token's E logits, s = softmax(z) or 1 / (1 + e^-z):
//   ids    the K largest z (no bias) or s + bias (in float64), equal ones in
//          ascending id;
//   gates  scale * s_id, or scale * s_id / (sum of the K chosen s);
//   p      softmax(z), or s / (sum of the E s): what the loss averages.
// A sequence q of L tokens has counts c_e, f_e = E c_e / (K L), P_e = mean p_e
// and loss sum_e f_e P_e; f carries no gradient.
//
// One wave holds one token's row: lane l has experts 128 j + 2 l and
// 128 j + 2 l + 1, so a row of even E is read as pairs, and every reduction
// over the experts is a DPP tree.
#include <type_traits>

#include "common.hpp"
#include "host.hpp"

namespace moonep {

constexpr int kRtThreads = 256;
constexpr int kRtWaves = kRtThreads / kWave;
constexpr int kRtMaxChunks = 1024;              // workgroups whose sums are joined
constexpr int kKeyNone = -2147483647 - 1;       // below every key: taken, or past E

struct RouterArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;                  // written when selecting, read otherwise
  float* gates;
  const int32_t* cu;             // [nseq + 1], or null: one sequence of all tokens
  float* part_p;                 // [chunks + nseq][E] sums of p
  int32_t* part_c;               // [chunks + nseq][E] counts
  const float* dgates;
  const int32_t* counts;
  const float* dloss;
  void* dlogits;
  int32_t T, E, K, nseq, chunk, score, renorm;
  float scale;
};

__device__ __forceinline__ int expert_of(int i) {
  return ((i >> 1) << 7) + 2 * lane_id() + (i & 1);
}

// One logit, at any alignment.
template <bool BF16>
__device__ __forceinline__ float logit_at(const void* z, int64_t i) {
  if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(z)[i]);
  else return reinterpret_cast<const float*>(z)[i];
}

// A row into P registers per lane; -inf (score 0) past E.
template <int P, bool BF16>
__device__ __forceinline__ void load_row(const void* z, int64_t t, int E, float (&v)[P]) {
  const int64_t at = t * E;
  if ((E & 1) == 0) {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const int e = expert_of(i);
      v[i] = v[i + 1] = -INFINITY;
      if (e < E) {
        if constexpr (BF16) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(
              reinterpret_cast<const uint16_t*>(z) + at + e);
          v[i] = bf16_lo(w);
          v[i + 1] = bf16_hi(w);
        } else {
          const float2 w = *reinterpret_cast<const float2*>(
              reinterpret_cast<const float*>(z) + at + e);
          v[i] = w.x;
          v[i + 1] = w.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = expert_of(i);
      v[i] = e < E ? logit_at<BF16>(z, at + e) : -INFINITY;
    }
  }
}

// Order of floats as order of ints: -0 equals +0, NaN comes below -inf.
__device__ __forceinline__ int order_key(float f) {
  const int b = __float_as_int(f + 0.f);
  return f != f ? kKeyNone + 1 : b ^ ((b >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float wave_max_f(float v) {        // NaN is passed over
  const int k = wave_max(v != v ? kKeyNone : order_key(v));
  if (k == kKeyNone) return -INFINITY;
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

__device__ __forceinline__ double wave_sum_d(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

__device__ __forceinline__ float sigmoid_f(float z) {
  const float t = __expf(-fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.f + t);
  return z != z ? z : z >= 0.f ? r : t * r;
}

// 1 - sigmoid(z) without cancellation.
__device__ __forceinline__ float co_sigmoid_f(float z) { return sigmoid_f(-z); }

// Below this logit a sigmoid is e^z to fp32's last bit, and ratios of scores
// are taken from e^(z - max) so that they survive the scores' underflow.
constexpr float kDeep = -60.f;

// Unnormalised p of a row: s (or its multiple) in v, and the factor 1 / sum.
// A row whose every logit is -inf has p = 0.
template <int P>
__device__ __forceinline__ float row_shares(const float (&z)[P], float (&v)[P], int score,
                                            float m) {
  const bool soft = score == MOE_SCORE_SOFTMAX || m < kDeep;
  float sum = 0.f;
  if (soft) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = m == -INFINITY && !(z[i] != z[i]) ? 0.f : __expf(z[i] - m);
      sum += v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = sigmoid_f(z[i]);
      sum += v[i];
    }
  }
  sum = wave_sum_f(sum);
  return sum == 0.f ? 0.f : 1.f / sum;
}

// The K largest keys in order, equal ones in ascending expert; lane k returns
// the k-th id.  key is consumed.
template <int P>
__device__ __forceinline__ int take_top(int (&key)[P], int K) {
  const int lane = lane_id();
  int mine = 0;
  for (int k = 0; k < K; ++k) {
    int best = key[0], bi = 0;
#pragma unroll
    for (int i = 1; i < P; ++i) {
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    }
    const int m = wave_max(best);
    const int e = expert_of(bi);
    uint64_t tied = __ballot(best == m);
    int id = wave_bcast(e, __ffsll((unsigned long long)tied) - 1);
    if (tied & (tied - 1)) id = -wave_max(best == m ? -e : kKeyNone);
    if (best == m && e == id) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i == bi) key[i] = kKeyNone;
    }
    if (lane == k) mine = id;
  }
  return mine;
}

// Scores s + bias of one expert in float64.
template <bool BF16>
__device__ __forceinline__ double key64(const RouterArgs& a, int64_t at, int e, double m,
                                        double sum) {
  const double z = (double)logit_at<BF16>(a.logits, at + e);
  double s;
  if (a.score == MOE_SCORE_SOFTMAX) s = m == -INFINITY && z == z ? 0.0 : exp(z - m) / sum;
  else s = 1.0 / (1.0 + exp(-z));
  return s + (double)a.bias[e];
}

// take_top on the float64 scores plus bias, for a row whose fp32 ones are too
// near each other to order.  Rare, so nothing is kept in registers between
// rounds: the scores are computed anew.
template <int P, bool BF16>
__device__ int take_top64(const RouterArgs& a, int64_t t, float mf) {
  const int lane = lane_id();
  const int64_t at = t * a.E;
  const double m = (double)mf;
  double sum = 1.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    sum = 0.0;
    for (int i = 0; i < P; ++i) {
      const int e = expert_of(i);
      if (e < a.E) {
        const double z = (double)logit_at<BF16>(a.logits, at + e);
        if (!(m == -INFINITY && z == z)) sum += exp(z - m);
      }
    }
    sum = wave_sum_d(sum);
  }
  uint32_t taken = 0;                            // P <= 32 bits
  int mine = 0;
  for (int k = 0; k < a.K; ++k) {
    // rank of a candidate: numbers by value, then NaN, then nothing
    double best = 0.0;
    int cls = 0, id = 0x7fffffff, bi = 0;
    for (int i = 0; i < P; ++i) {
      const int e = expert_of(i);
      if (e >= a.E || (taken >> i & 1)) continue;
      const double d = key64<BF16>(a, at, e, m, sum);
      const int c = d == d ? 2 : 1;
      if (c > cls || (c == cls && c == 2 && d > best)) {
        cls = c;
        best = d;
        id = e;
        bi = i;
      }
    }
    const int mybi = bi, myid = id;
    for (int o = 32; o > 0; o >>= 1) {
      const double od = __shfl_xor(best, o, kWave);
      const int oc = __shfl_xor(cls, o, kWave), oi = __shfl_xor(id, o, kWave);
      const bool equal = oc == cls && (cls < 2 || od == best);
      if (oc > cls || (oc == cls && cls == 2 && od > best) || (equal && oi < id)) {
        best = od;
        cls = oc;
        id = oi;
      }
    }
    if (id == myid && cls > 0) taken |= 1u << mybi;
    if (lane == k) mine = id;
  }
  return mine;
}

// Lane k < K: the k-th chosen expert of token t.  m is the row's largest
// logit.
//
// With a bias the order is that of float64 s + bias.  fp32 keys order all rows
// but those where two neighbours among the K + 1 largest are nearer than the
// keys' errors: s from v_exp_f32 and v_rcp_f32 (1 ulp each) is off by
//   sigmoid  s (1 - s) |z| 2^-24 + 2.5 ulp  <=  1.4e-8 + 2.5 * 2^-23 s,
//   softmax  s (|z - m| 2^-24 + the sum's) <= 8e-6 s  (s > 0 needs |z - m| < 104),
// and the sum with the bias by 2^-24 |key|.  Such rows are taken again in
// float64; equal logits with equal biases need no second look.
template <int P, bool BF16>
__device__ __forceinline__ int choose(const RouterArgs& a, int64_t t, const float (&z)[P],
                                      const float (&v)[P], float inv, float m) {
  int key[P];
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = expert_of(i) < a.E ? order_key(z[i]) : kKeyNone;
    return take_top<P>(key, a.K);
  }
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  const int n = a.K < a.E ? a.K + 1 : a.K;
  if (n <= kWave) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = expert_of(i);
      key[i] = e < a.E ? order_key((soft ? v[i] * inv : sigmoid_f(z[i])) + a.bias[e]) : kKeyNone;
    }
    const int id = take_top<P>(key, n);
    const int lane = lane_id();
    const int at = lane < n ? id : 0;
    const float zi = logit_at<BF16>(a.logits, t * a.E + at), bi = a.bias[at];
    const float s = soft ? (m == -INFINITY ? 0.f : __expf(zi - m) * inv) : sigmoid_f(zi);
    const float k = s + bi;
    const float zo = __shfl_down(zi, 1, kWave), bo = __shfl_down(bi, 1, kWave);
    const float so = __shfl_down(s, 1, kWave), ko = __shfl_down(k, 1, kWave);
    const float tol = (soft ? 8e-6f * (s + so) : 4e-7f * (s + so) + 4e-8f) +
                      1.2e-7f * (fabsf(k) + fabsf(ko));
    const bool same = zi == zo && bi == bo;
    const bool clear = same || k - ko > tol;             // NaN is never clear
    if (__all(lane >= n - 1 || clear)) return id;
  }
  return take_top64<P, BF16>(a, t, m);
}

// Lane k < K: score of the chosen logit zk relative to `total`, such that the
// gate is scale * w.
__device__ __forceinline__ float gate_share(float zk, bool on, int score, bool renorm, float m,
                                            float inv) {
  if (!renorm) {
    if (!on) return 0.f;
    if (score == MOE_SCORE_SIGMOID) return sigmoid_f(zk);
    return m == -INFINITY && zk == zk ? 0.f : __expf(zk - m) * inv;
  }
  const float mk = wave_max_f(on ? zk : -INFINITY);
  float s = 0.f;
  if (on) {
    if (score == MOE_SCORE_SOFTMAX || mk < kDeep)
      s = mk == -INFINITY && zk == zk ? 0.f : __expf(zk - mk);
    else
      s = sigmoid_f(zk);
  }
  const float sum = wave_sum_f(s);
  return sum == 0.f ? 0.f : s / sum;
}

// The sequence that holds token t (the last one with cu[s] <= t), or -1, and
// where its tokens, or those of no sequence, end.
__device__ __forceinline__ int sequence_of(const RouterArgs& a, int t, int& end) {
  if (!a.cu) {
    end = a.T;
    return 0;
  }
  int lo = -1, hi = a.nseq;                       // cu[lo] <= t < cu[hi], as if cu[-1] = -inf
  if (a.cu[hi] <= t) {
    end = a.T;
    return -1;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  end = max(t + 1, min(a.cu[hi], a.T));
  return lo;                                      // -1: before the first sequence
}

// ---------------------------------------------------------------------------
// Forward.  A workgroup owns `chunk` consecutive tokens, its waves take them in
// turn.  Where the loss is wanted, each wave keeps the sums of p in registers
// and the workgroup the counts in LDS; both go to row (workgroup + sequence)
// of the workspace when the sequence or the chunk ends.  Along the tokens
// either number grows, so no two pieces share a row.
// ---------------------------------------------------------------------------
template <int P, bool BF16, bool SELECT, bool STATS>
__global__ __launch_bounds__(kRtThreads) void k_router(RouterArgs a) {
  extern __shared__ float lds[];                  // [waves][E] sums, [E] counts
  const int lane = lane_id(), wv = threadIdx.x / kWave;
  const int E = a.E, K = a.K;
  int* cnt = reinterpret_cast<int*>(lds + kRtWaves * E);
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  float acc[P];
  for (int lo = t0; lo < t1;) {
    int hi = t1, seq = -1;
    if constexpr (STATS) {
      seq = sequence_of(a, lo, hi);
      hi = min(hi, t1);
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] = 0.f;
      for (int e = threadIdx.x; e < E; e += kRtThreads) cnt[e] = 0;
      __syncthreads();
    }
    if (SELECT || seq >= 0) {
      for (int t = lo + wv; t < hi; t += kRtWaves) {
        float z[P], v[P];
        load_row<P, BF16>(a.logits, t, E, z);
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < P; ++i) m = fmaxf(m, z[i]);
        m = wave_max_f(m);
        float inv = 0.f;
        const bool shares = STATS || (SELECT && a.score == MOE_SCORE_SOFTMAX &&
                                      (a.bias || !a.renorm));
        if (shares) inv = row_shares<P>(z, v, a.score, m);
        int id = -1;
        if constexpr (SELECT) {
          id = choose<P, BF16>(a, t, z, v, inv, m);
          const bool on = lane < K;
          const float zk = on ? logit_at<BF16>(a.logits, int64_t(t) * E + id) : 0.f;
          const float w = gate_share(zk, on, a.score, a.renorm, m, inv);
          if (on) {
            a.ids[int64_t(t) * K + lane] = id;
            a.gates[int64_t(t) * K + lane] = a.scale * w;
          }
        } else {
          if (lane < K) id = a.ids[int64_t(t) * K + lane];
        }
        if constexpr (STATS) {
          if (seq >= 0) {
            if (lane < K && (unsigned)id < (unsigned)E) atomicAdd(&cnt[id], 1);
#pragma unroll
            for (int i = 0; i < P; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
          }
        }
      }
    }
    if constexpr (STATS) {
      if (seq >= 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int e = expert_of(i);
          if (e < E) lds[wv * E + e] = acc[i];
        }
      }
      __syncthreads();
      if (seq >= 0) {
        const int64_t row = int64_t(blockIdx.x + seq) * E;
        for (int e = threadIdx.x; e < E; e += kRtThreads) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < kRtWaves; ++w) s += lds[w * E + e];
          a.part_p[row + e] = s;
          a.part_c[row + e] = cnt[e];
        }
      }
      __syncthreads();                            // cnt is cleared next
    }
    lo = hi;
  }
}

// Joins a sequence's rows, in the order of its chunks, into counts, P and the
// loss.  One workgroup per sequence.
constexpr int kFinThreads = 1024;

__global__ __launch_bounds__(kFinThreads) void k_router_finish(RouterArgs a, int chunks,
                                                              int32_t* counts, float* prob,
                                                              float* loss) {
  constexpr int W = kFinThreads / kWave;
  __shared__ double s_p[W][kWave];
  __shared__ int s_c[W][kWave];
  const int seq = blockIdx.x, lane = lane_id(), wv = threadIdx.x / kWave;
  const int lo = a.cu ? max(0, min(a.cu[seq], a.T)) : 0;
  const int hi = a.cu ? max(lo, min(a.cu[seq + 1], a.T)) : a.T;
  const int c0 = hi > lo ? lo / a.chunk : 0, c1 = hi > lo ? min((hi - 1) / a.chunk + 1, chunks) : 0;
  const double len = hi > lo ? (double)(hi - lo) : 1.0;
  double total = 0.0;
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    const int e = e0 + lane;
    double p = 0.0;
    int c = 0;
    if (e < a.E) {
      for (int r = c0 + wv; r < c1; r += W) {
        const int64_t at = int64_t(r + seq) * a.E + e;
        p += (double)a.part_p[at];
        c += a.part_c[at];
      }
    }
    s_p[wv][lane] = p;
    s_c[wv][lane] = c;
    __syncthreads();
    if (wv == 0 && e < a.E) {
      for (int w = 1; w < W; ++w) {
        p += s_p[w][lane];
        c += s_c[w][lane];
      }
      const double mean = p / len;
      counts[int64_t(seq) * a.E + e] = c;
      prob[int64_t(seq) * a.E + e] = (float)mean;
      total += (double)a.E * c / (a.K * len) * mean;
    }
    __syncthreads();
  }
  if (wv == 0) {
    total = wave_sum_d(total);
    if (lane == 0) loss[seq] = (float)total;
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
// ---------------------------------------------------------------------------
template <int P, bool BF16>
__global__ __launch_bounds__(kRtThreads) void k_router_bwd(RouterArgs a) {
  extern __shared__ float lds[];                  // [waves][E]
  const int lane = lane_id(), wv = threadIdx.x / kWave;
  const int E = a.E, K = a.K;
  float* row = lds + wv * E;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  const bool balance = a.dloss != nullptr, gates = a.dgates != nullptr;
  const bool into_u = soft && gates && !a.renorm;         // the gates' part goes through p
  for (int e = lane; e < E; e += kWave) row[e] = 0.f;
  const int64_t w0 = (int64_t(blockIdx.x) * kRtWaves + wv) * a.chunk;
  const int t0 = (int)min<int64_t>(w0, a.T), t1 = (int)min<int64_t>(w0 + a.chunk, a.T);
  int end = t0, seq = -1;
  float u[P];
#pragma unroll
  for (int i = 0; i < P; ++i) u[i] = 0.f;
  for (int t = t0; t < t1; ++t) {
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
    const bool bal = balance && seq >= 0;
    float z[P], v[P], dz[P];
    float m = -INFINITY, inv = 0.f;
    if (bal || into_u) {
      load_row<P, BF16>(a.logits, t, E, z);
#pragma unroll
      for (int i = 0; i < P; ++i) m = fmaxf(m, z[i]);
      m = wave_max_f(m);
      inv = row_shares<P>(z, v, a.score, m);
    }
    int id = -1;
    if (gates) {
      if (lane < K) id = a.ids[int64_t(t) * K + lane];
      const bool on = (unsigned)id < (unsigned)E;
      const float zk = on ? logit_at<BF16>(a.logits, int64_t(t) * E + id) : 0.f;
      const float dg = on ? a.scale * a.dgates[int64_t(t) * K + lane] : 0.f;
      float val = dg;
      if (!into_u) {
        const float w = gate_share(zk, on, a.score, a.renorm, m, inv);
        const float mean = a.renorm ? wave_sum_f(dg * w) : 0.f;
        val = w * (dg - mean);
        if (!soft) val *= co_sigmoid_f(zk);
      }
      if (on) atomicAdd(&row[id], val);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < P; ++i) dz[i] = gates && expert_of(i) < E ? row[expert_of(i)] : 0.f;
    if (gates) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if ((unsigned)id < (unsigned)E) row[id] = 0.f;
    }
    if (bal || into_u) {
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v[i] *= inv;
        const float ui = (bal ? u[i] : 0.f) + (into_u ? dz[i] : 0.f);
        mean = fmaf(ui, v[i], mean);
      }
      mean = wave_sum_f(mean);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float ui = (bal ? u[i] : 0.f) + (into_u ? dz[i] : 0.f);
        const float g = v[i] * (ui - mean) * (soft ? 1.f : co_sigmoid_f(z[i]));
        dz[i] = (into_u ? 0.f : dz[i]) + g;
      }
    }
    const int64_t at = int64_t(t) * E;
    if ((E & 1) == 0) {
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const int e = expert_of(i);
        if (e < E) {
          if constexpr (BF16)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.dlogits) + at + e) =
                pack_bf16x2(dz[i], dz[i + 1]);
          else
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.dlogits) + at + e) =
                float2{dz[i], dz[i + 1]};
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = expert_of(i);
        if (e < E) {
          if constexpr (BF16)
            reinterpret_cast<uint16_t*>(a.dlogits)[at + e] = (uint16_t)f32_to_bf16(dz[i]);
          else
            reinterpret_cast<float*>(a.dlogits)[at + e] = dz[i];
        }
      }
    }
  }
}

// Tokens per workgroup and workgroups of a forward call that keeps sums.
inline int stats_chunk(int T) { return T > 0 ? (T + kRtMaxChunks - 1) / kRtMaxChunks : 1; }
inline int stats_chunks(int T) { return T > 0 ? (T + stats_chunk(T) - 1) / stats_chunk(T) : 0; }

inline size_t part_rows(int T, int nseq) { return size_t(stats_chunks(T)) + size_t(nseq); }

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

// Calls f with the registers per lane of a row of E experts and the type.
template <typename F>
inline int with_row(int E, bool bf16, F f) {
  const int p = 2 * ((E + 127) / 128);
#define MOE_ROW(N)                                                       \
  if (p <= N)                                                            \
  return bf16 ? f(std::integral_constant<int, N>(), std::true_type())    \
              : f(std::integral_constant<int, N>(), std::false_type())
  MOE_ROW(2);
  MOE_ROW(4);
  MOE_ROW(6);
  MOE_ROW(8);
  MOE_ROW(14);
  MOE_ROW(20);
  MOE_ROW(32);
#undef MOE_ROW
  return MOE_ELIMIT;
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
    a.chunk = stats_chunk(a.T);
    chunks = stats_chunks(a.T);
    a.part_p = reinterpret_cast<float*>(workspace);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + part_rows(a.T, a.nseq) * a.E);
  } else {
    a.chunk = kRtWaves;
  }
  if (a.T > 0) {
    const int grid = stats ? chunks : (a.T + a.chunk - 1) / a.chunk;
    const size_t lds = stats ? size_t(kRtWaves + 1) * a.E * 4 : 0;
    const int rc = with_row(a.E, r->logits_bf16, [&](auto p, auto b) {
      constexpr int P = decltype(p)::value;
      constexpr bool BF = decltype(b)::value;
      const dim3 g(grid), t(kRtThreads);
      if (select && stats) hipLaunchKernelGGL((k_router<P, BF, true, true>), g, t, lds, stream, a);
      else if (select) hipLaunchKernelGGL((k_router<P, BF, true, false>), g, t, lds, stream, a);
      else hipLaunchKernelGGL((k_router<P, BF, false, true>), g, t, lds, stream, a);
      return hip_status();
    });
    if (rc != MOE_OK) return rc;
  }
  if (stats) {
    hipLaunchKernelGGL(k_router_finish, dim3(a.nseq), dim3(kFinThreads), 0, stream, a, chunks,
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
  *bytes_out = align256(part_rows(cfg->R * cfg->S, rcfg->nseq) * cfg->E * 8);
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
  a.chunk = a.T >= (1 << 15) ? 8 : 1;
  const int per = kRtWaves * a.chunk;
  const size_t lds = size_t(kRtWaves) * a.E * 4;
  return with_row(a.E, rcfg->logits_bf16, [&](auto p, auto b) {
    hipLaunchKernelGGL((k_router_bwd<decltype(p)::value, decltype(b)::value>),
                       dim3((a.T + per - 1) / per), dim3(kRtThreads), lds, stream, a);
    return hip_status();
  });
}
