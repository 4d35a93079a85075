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
#pragma once

#include <type_traits>

#include "common.hpp"
#include "convert.hpp"
#include "host.hpp"

namespace moonep {

constexpr int kRtThreads = 512;
constexpr int kRtWaves = kRtThreads / kWave;
// Workgroups whose sums are joined, at most; and how many a call that chooses
// makes of its tokens: its registers leave two workgroups a CU, and a second
// round of workgroups costs more than it evens out (65,536 tokens of 384
// experts: 50.3 us in 512 workgroups, 55.9 in 1,024).
constexpr int kRtMaxChunks = 1024;
constexpr int kRtSelectChunks = 512;
constexpr int kKeyNone = -2147483647 - 1;       // below every key: taken, or past E

struct RouterArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;                  // written when selecting, read otherwise
  float* gates;
  const int32_t* cu;             // [nseq + 1], or null: one sequence of all tokens
  float* part_p;                 // [chunks + nseq][E] sums of p
  int32_t* part_c;               // [chunks + nseq][E] counts
  double* sum_p;                 // [nseq][parts][E] the same, joined in part
  int32_t* sum_c;
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

// A token's row as loaded: P / 2 pairs per lane.  FULL: E == 64 P, every lane
// holds P experts and nothing is masked.
template <int P, bool BF16>
struct Row {
  uint32_t w[BF16 ? P / 2 : P];
};

// The registers of a row that hold experts in every lane: a row of P has more
// than 64 kSure<P> experts (with_row).
template <int P>
constexpr int kSure = P <= 8 ? P - 2 : P == 12 ? 8 : P <= 16 ? P - 2 : P == 20 ? 16 : 20;

// Lanes past E load experts before it, which unpack_row replaces: a load under a
// condition costs more (32,768 fp32 rows of 704 experts: routes 24 us, 21 so).
template <int P, bool BF16, bool FULL>
__device__ __forceinline__ void load_row(const void* z, int64_t t, int E, Row<P, BF16>& r) {
  using T = std::conditional_t<BF16, uint16_t, uint32_t>;
  using Pair = std::conditional_t<BF16, uint32_t, uint2>;
  const T* p = reinterpret_cast<const T*>(z) + t * E;
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const int e = expert_of(i);
    const bool sure = FULL || i < kSure<P>;
    if (FULL || (E & 1) == 0) {
      const Pair v = *reinterpret_cast<const Pair*>(p + (sure ? e : min(e, E - 2)));
      if constexpr (BF16) {
        r.w[i / 2] = v;
      } else {
        r.w[i] = v.x;
        r.w[i + 1] = v.y;
      }
    } else {
      const uint32_t lo = p[sure ? e : min(e, E - 1)], hi = p[sure ? e + 1 : min(e + 1, E - 1)];
      if constexpr (BF16) {
        r.w[i / 2] = lo | (hi << 16);
      } else {
        r.w[i] = lo;
        r.w[i + 1] = hi;
      }
    }
  }
}

// The row's logits, -inf past E.
template <int P, bool BF16, bool FULL>
__device__ __forceinline__ void unpack_row(const Row<P, BF16>& r, int E, float (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (BF16) v[i] = (i & 1) ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
    else v[i] = __uint_as_float(r.w[i]);
    if (!FULL && i >= kSure<P>) v[i] = expert_of(i) < E ? v[i] : -INFINITY;
  }
}

// Order of floats as order of ints: -0 equals +0, NaN comes below -inf.
__device__ __forceinline__ int order_key(float f) {
  const int b = __float_as_int(f + 0.f);
  return f != f ? kKeyNone + 1 : b ^ ((b >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float key_value(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

__device__ __forceinline__ uint64_t ballot(bool b) { return __builtin_amdgcn_ballot_w64(b); }

// order_key of the largest of the 64 lanes' values; NaN is passed over.
__device__ __forceinline__ int wave_max_key(float v) {
  return wave_max(v != v ? kKeyNone : order_key(v));
}

// That value, -inf if there is none.
__device__ __forceinline__ float wave_max_f(float v) {
  const int k = wave_max_key(v);
  return k == kKeyNone ? -INFINITY : key_value(k);
}

template <int P>
__device__ __forceinline__ float lane_max(const float (&v)[P]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < P; ++i) m = fmaxf(m, v[i]);
  return m;
}

__device__ __forceinline__ double wave_sum_d(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

__device__ __forceinline__ double lane_bcast_d(double v, int l) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)wave_bcast((int)b, l);
  const uint32_t hi = (uint32_t)wave_bcast((int)(b >> 32), l);
  return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ float exp_f(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// sigmoid(z) and 1 - sigmoid(z), neither by cancellation; NaN stays NaN.
__device__ __forceinline__ float sigmoid_f(float z, float& co) {
  const float t = exp_f(-fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.f + t), q = t * r;
  co = z >= 0.f ? q : r;
  return z >= 0.f ? r : q;
}

__device__ __forceinline__ float sigmoid_f(float z) {
  float co;
  return sigmoid_f(z, co);
}

// Below this logit a sigmoid is e^z to fp32's last bit, and ratios of scores
// are taken from e^(z - max) so that they survive the scores' underflow.
constexpr float kDeep = -60.f;

// Sums of exponentials in this range are taken as they are: the largest logit
// is then between -8 and 13, so nothing overflows, a share that underflows is
// below 2^-126 itself, and the exponentials' arguments are longer than those of
// z - max by 13 at most.  Other sums (far logits, a masked row's 0, NaN) are
// taken again from z - max.
constexpr float kPlainLo = 1.f, kPlainHi = 0x1p18f;
// The same for sums of sigmoids: none of their terms that count has underflowed.
constexpr float kSigmoidLo = 0x1p-60f;

__device__ __forceinline__ float recip(float sum) {          // 0 for an empty sum
  return sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum);
}

// Unnormalised shares p of token t in v (co: 1 - s for sigmoids) and their
// factor, from its logits z.  The scores of a softmax are e^(z - shift) times
// that factor.  A row whose every logit is -inf has p = 0.
template <int P, bool BF16, bool FULL, bool SOFT, bool CO>
__device__ __forceinline__ float row_shares(const RouterArgs& a, int64_t t, const float (&z)[P],
                                            float (&v)[P], float (&co)[P], float& shift) {
  float sum = 0.f;
  shift = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (SOFT) {
      v[i] = exp_f(z[i]);
    } else {
      float c;
      v[i] = sigmoid_f(z[i], c);
      if constexpr (CO) co[i] = c;
    }
    sum += v[i];
  }
  sum = wave_sum_f(sum);
  if (SOFT ? sum >= kPlainLo && sum <= kPlainHi : sum >= kSigmoidLo) return recip(sum);
  // the row is loaded again, so that z need not be kept for this
  Row<P, BF16> again;
  load_row<P, BF16, FULL>(a.logits, t, a.E, again);
  float x[P];
  unpack_row<P, BF16, FULL>(again, a.E, x);
  const float m = wave_max_f(lane_max<P>(x));
  if (!SOFT && !(m < kDeep)) return recip(sum);              // NaN, for one
  sum = 0.f;
  if (m > -INFINITY) shift = m;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    v[i] = exp_f(x[i] - shift);
    if constexpr (CO) co[i] = 1.f;                           // a deep row's 1 - s
    sum += v[i];
  }
  return recip(wave_sum_f(sum));
}

// The K largest keys in order, equal ones in ascending expert; lane k returns
// the k-th id.  key is consumed.  Any keys: K rounds of a maximum of the wave.
// For rows that sort_top leaves: NaN, masks, many equal keys, and with K above 24
// ordinary rows, whose 64 lanes cannot bound so many keys (65,536 bf16 rows of 384
// experts: routes 26 us with K = 8, 43 with 24, 70 with 28, 153 with 32, 327 with
// 64).  Used for all rows of 896 experts and K = 16 it takes 1,174 us where
// sort_top takes 205.
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

// A bound t such that the K largest keys are among those >= t, and few others
// are.  `top` is the lane's largest key, `hi` the order_key of the row's.  The
// K-th largest of the 64 lanes' largest keys is such a bound; any bound that K
// to 3 K / 2 + 1 lanes reach is taken.  It is searched for on the scalar unit,
// one comparison of the wave a step: from the bound of the wave's last token
// (`probe`), whose row was much like this one, outwards by doubled steps and
// then by halves.  -inf where there is none above it (fewer than K lanes have
// a finite key).  The choice that follows does not depend on which is taken.
__device__ __forceinline__ float key_bound(float top, int hi, int K, int& probe) {
  const int most = K + (K >> 1) + 1;
  const int low = order_key(-INFINITY);
  const auto reach = [&](int k) { return (int)__popcll(ballot(top >= key_value(k))); };
  const bool fresh = probe == kKeyNone;                      // no token before
  const int step = fresh ? 1 << 20 : 1 << 18;
  int lo = fresh ? max(hi - step, low + 1) : min(probe, hi), up = hi + 1, n = reach(lo);
  if (n < K) {
    for (int d = step; n < K; d <<= 1) {
      if (d < 0 || (int64_t)lo - d <= (int64_t)low) return -INFINITY;
      up = lo;
      lo -= d;
      n = reach(lo);
    }
  } else if (n > most) {
    for (int d = step; d > 0 && (uint32_t)hi - (uint32_t)lo > (uint32_t)d; d <<= 1) {
      const int c = reach(lo + d);
      if (c < K) {
        up = lo + d;
        break;
      }
      lo += d;
      n = c;
      if (n <= most) break;
    }
  }
  while (n > most && (uint32_t)up - (uint32_t)lo > 1u) {
    const int mid = lo + (int)(((uint32_t)up - (uint32_t)lo) >> 1);
    const int c = reach(mid);
    if (c >= K) {
      lo = mid;
      n = c;
    } else {
      up = mid;
    }
  }
  probe = lo;
  return key_value(lo);
}

// Lanes whose i-th key reaches t, for every i, and their number.
template <int P>
__device__ __forceinline__ int reaching(const float (&key)[P], float t, uint64_t (&m)[P]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    m[i] = ballot(key[i] >= t);
    n += (int)__popcll(m[i]);
  }
  return n;
}

// A wave's list of up to 64 keys and their experts.
struct KeyList {
  float key[kWave];
  int id[kWave];
};

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Number of listed keys that come before key k, the one at place `cand`: larger
// ones, and equal ones at earlier places.  The G groups of 64 / G lanes hold
// the same candidates (cand = lane modulo the group) and look at a G-th of the
// list each, four keys a read.
template <int G>
__device__ __forceinline__ int count_before(const KeyList& list, int cnt, float k) {
  constexpr int L = kWave / G;
  const int per = (cnt + 4 * G - 1) / (4 * G) * 4;           // places per group, G * per <= 64
  const int first = lane_id() / L * per;
  int ahead = lane_id() % L - first;                         // cand - place
  int rank = 0;
  for (int j = 0; j < per; j += 4, ahead -= 4) {
    const f32x4 o = *reinterpret_cast<const f32x4*>(list.key + first + j);
#pragma unroll
    for (int q = 0; q < 4; ++q) rank += (o[q] > k) | ((o[q] == k) & (ahead > q)) ? 1 : 0;
  }
  if constexpr (G == 4) rank += __shfl_xor(rank, 16, kWave);
  if constexpr (G >= 2) rank += __shfl_xor(rank, 32, kWave);
  return rank;
}

// Sorts the cnt <= 64 keys that m marks across the lanes, largest first, equal
// ones in ascending expert: lane k < cnt gets the k-th key and its expert.
// They are written to the list in ascending expert, each one's place in the
// order is counted, and that is where its lane sends it.  (Inserting one key
// after the other into a list across the lanes, a median of three a key, took
// 316 us where this takes 205: a chain of 20 steps with their scalar loop.)
template <int P>
__device__ __forceinline__ void sort_marked(const float (&key)[P], const uint64_t (&m)[P],
                                            int cnt, KeyList& list, float& mykey, int& mine) {
  const int lane = lane_id();
  int base = 0;
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    if ((m[i] | m[i + 1]) == 0) continue;
    int at = base;
    at = __builtin_amdgcn_mbcnt_lo((uint32_t)m[i], at);
    at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m[i] >> 32), at);
    at = __builtin_amdgcn_mbcnt_lo((uint32_t)m[i + 1], at);
    at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m[i + 1] >> 32), at);
    const bool first = __builtin_amdgcn_inverse_ballot_w64(m[i]);
    if (first) {
      list.key[at] = key[i];
      list.id[at] = expert_of(i);
    }
    if (__builtin_amdgcn_inverse_ballot_w64(m[i + 1])) {
      const int to = at + (first ? 1 : 0);
      list.key[to] = key[i + 1];
      list.id[to] = expert_of(i + 1);
    }
    base += (int)__popcll(m[i]) + (int)__popcll(m[i + 1]);
  }
  if (lane >= cnt) list.key[lane] = -INFINITY;
  wave_lds_fence();
  const int groups = cnt <= 16 ? 4 : cnt <= 32 ? 2 : 1;
  const float k = list.key[lane & (kWave / groups - 1)];
  const int id = list.id[lane];
  const int rank = groups == 4   ? count_before<4>(list, cnt, k)
                   : groups == 2 ? count_before<2>(list, cnt, k)
                                 : count_before<1>(list, cnt, k);
  wave_lds_fence();                              // the list is written again
  const int to = 4 * (lane < cnt ? rank : lane);
  // (lanes past the first group send what they hold of the list, behind cnt)
  mykey = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(k)));
  mine = __builtin_amdgcn_ds_permute(to, id);
}

// take_top through key_bound and sort_marked: the largest keys, K at least.
// False, and nothing done, where a key is NaN, more than 64 keys reach the
// bound, or fewer than K keys are finite.
template <int P>
__device__ __forceinline__ bool sort_top(const float (&key)[P], bool no_nan, int K, int& probe,
                                         KeyList& list, float& mykey, int& mine) {
  if (!no_nan) {
    uint64_t bad = 0;
#pragma unroll
    for (int i = 0; i < P; i += 2) bad |= ballot(__builtin_isunordered(key[i], key[i + 1]));
    if (bad) return false;
  }
  const float top = lane_max<P>(key);
  float t = key_bound(top, wave_max_key(top), K, probe);
  if (t == -INFINITY) t = -3.402823466e38f;      // every finite key: 64 experts, or a mask
  uint64_t m[P];
  const int cnt = reaching<P>(key, t, m);
  if (cnt < K || cnt > kWave) return false;
  sort_marked<P>(key, m, cnt, list, mykey, mine);
  return true;
}

// Score plus bias of one expert in float64; at: the row's first logit.
template <bool BF16, bool SOFT>
__device__ __forceinline__ double key64(const RouterArgs& a, int64_t at, int e, double m,
                                        double sum) {
  const double z = (double)logit_at<BF16>(a.logits, at + e);
  if (z == -INFINITY) return -INFINITY;          // masked, whatever its bias
  double s;
  if constexpr (SOFT) s = exp(z - m) / sum;
  else s = 1.0 / (1.0 + exp(-z));
  return s + (double)a.bias[e];
}

// Sum of a row's e^(z - m) in float64.
template <bool BF16>
__device__ __forceinline__ double sum64(const RouterArgs& a, int64_t at, double m) {
  double sum = 0.0;
#pragma unroll 1
  for (int e = lane_id(); e < a.E; e += kWave) {
    const double z = (double)logit_at<BF16>(a.logits, at + e);
    if (z != -INFINITY) sum += exp(z - m);
  }
  return wave_sum_d(sum);
}

// Orders the cnt experts `id` of lanes 0 .. cnt - 1 by float64 score plus bias.
template <bool BF16, bool SOFT>
__device__ __forceinline__ int order64(const RouterArgs& a, int64_t at, float mf, int cnt, int id) {
  const int lane = lane_id();
  const double m = (double)mf, sum = SOFT ? sum64<BF16>(a, at, m) : 1.0;
  const double mine = lane < cnt ? key64<BF16, SOFT>(a, at, id, m, sum) : 0.0;
  int rank = 0;
  for (int j = 0; j < cnt; ++j) {
    const double kj = lane_bcast_d(mine, j);
    const int ij = wave_bcast(id, j);
    rank += kj > mine || (kj == mine && ij < id) ? 1 : 0;
  }
  return __builtin_amdgcn_ds_permute(4 * (lane < cnt ? rank : lane), id);
}

// take_top on the float64 scores plus bias: the K largest, equal ones in
// ascending expert; after all numbers the sums that are NaN (a NaN bias, a softmax
// row with NaN or +inf), then the masked experts, NaN logits last, each of these
// in ascending expert.  For rows that sort_top leaves, K of them finite or fewer
// among them, and for every row of K = 64 below E.  Nothing is kept in registers
// between rounds: the scores are computed anew, K times E of them.  Ordinary rows
// with a bias come here from K = 28 on: 65,536 of 384 experts take 40 us with
// K = 8, 2.1 ms with 32 and 4.8 with 64; of 896, 56 us, 4.8 and 10 ms.
template <bool BF16, bool SOFT>
__device__ __forceinline__ int take_top64(const RouterArgs& a, int64_t at, float mf) {
  const int lane = lane_id();
  const double m = (double)mf, sum = SOFT ? sum64<BF16>(a, at, m) : 1.0;
  uint32_t taken = 0;                            // at most 32 experts a lane
  int mine = 0;
  for (int k = 0; k < a.K; ++k) {
    // class of a candidate: 4 a number, 3 NaN, 2 masked, 1 a NaN logit, 0 none
    double best = 0.0;
    int cls = 0, id = 0x7fffffff;
#pragma unroll 1
    for (int i = 0, e = lane; e < a.E; ++i, e += kWave) {
      if (taken >> i & 1) continue;
      const float z = logit_at<BF16>(a.logits, at + e);
      const double d = key64<BF16, SOFT>(a, at, e, m, sum);
      const int c = z != z ? 1 : z == -INFINITY ? 2 : d == d ? 4 : 3;
      if (c > cls || (c == cls && c == 4 && d > best)) {
        cls = c;
        best = d;
        id = e;
      }
    }
    const int myid = id;
    for (int o = 32; o > 0; o >>= 1) {
      const double od = __shfl_xor(best, o, kWave);
      const int oc = __shfl_xor(cls, o, kWave), oi = __shfl_xor(id, o, kWave);
      const bool equal = oc == cls && (cls < 4 || od == best);
      if (oc > cls || (oc == cls && cls == 4 && od > best) || (equal && oi < id)) {
        best = od;
        cls = oc;
        id = oi;
      }
    }
    if (id == myid && cls > 0) taken |= 1u << (id / kWave);
    if (lane == k) mine = id;
  }
  return mine;
}

// Lane k < K: the k-th expert by score plus bias (fp32 in key), and its logit
// zk; m is the row's largest logit (softmax).
//
// The order is that of float64 scores plus bias; fp32 keys give it wherever
// neighbours among the K + 1 largest keys are further apart than two keys'
// errors.  With h = 2^-24 a sigmoid key is off by the argument's rounding,
//   s (1 - s) |z| 2.2 h  <=  2.9e-8,
// and by the exponential's, the sum's and the reciprocal's, at most 2^-22 of a
// score above 1/2 and 3 * 2^-23 of one below, 2.4e-7: 3.2e-7 covers both.  A
// softmax key is off by
//   s (|z - shift| 2.2 h + the sum's relative error), where
//   s |z - max| <= 0.37 p_max and the sum's error is at most
//   (2.2 ln E + 48 + 33) h:  <= 8e-6 p_max,
// and both by h |key| from the addition.  Other rows list every key that may be
// among the K largest, at most 64, and order those in float64, a lane each.
// Equal logits under equal biases are such rows: bf16 logits with a bias of zeros
// and the loss, 65,536 tokens, take 70 us at E = 384, K = 8 (sigmoid; with a random
// bias 50) and 217 at E = 896, K = 16 (softmax, whose sum is taken again; 82).
template <int P, bool BF16, bool SOFT>
__device__ __forceinline__ int choose_biased(const RouterArgs& a, int64_t t, float m,
                                             const float (&key)[P], float inv, float shift,
                                             int& probe, KeyList& list, float& zk) {
  const int lane = lane_id();
  const int64_t at = t * a.E;
  const int n = a.K < a.E ? a.K + 1 : a.K;
  float lk = 0.f;
  int id = 0;
  bool listed = n <= kWave && sort_top<P>(key, false, n, probe, list, lk, id);
  if (listed) {
    const float err = SOFT ? 8e-6f * exp_f(m - shift) * inv : 3.2e-7f;
    const float ko = __shfl_down(lk, 1, kWave);
    const bool apart = lk - ko > 2.f * err + 1.2e-7f * (fabsf(lk) + fabsf(ko));
    if (ballot(lane < n - 1 && !apart)) {
      const float last = __int_as_float(wave_bcast(__float_as_int(lk), a.K - 1));
      const float reach = last - (2.f * err + 2.4e-7f * fabsf(last) + 1e-12f);
      uint64_t in[P];
      const int cnt = reaching<P>(key, reach, in);
      listed = reach > -INFINITY && cnt <= kWave;
      if (listed) {
        sort_marked<P>(key, in, cnt, list, lk, id);
        id = order64<BF16, SOFT>(a, at, m, cnt, id);
      }
    }
  }
  if (!listed) id = take_top64<BF16, SOFT>(a, at, m);
  zk = logit_at<BF16>(a.logits, at + (lane < a.K ? id : 0));
  return id;
}

// Lane k < K: the k-th expert by logit, and its logit zk.
template <int P, bool BF16, bool FULL>
__device__ __forceinline__ int choose(const RouterArgs& a, int64_t t, const float (&z)[P],
                                      bool no_nan, int& probe, KeyList& list, float& zk) {
  int id = 0;
  if (sort_top<P>(z, no_nan, a.K, probe, list, zk, id)) return id;
  int key[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    key[i] = FULL || i < kSure<P> || expert_of(i) < a.E ? order_key(z[i]) : kKeyNone;
  id = take_top<P>(key, a.K);
  zk = logit_at<BF16>(a.logits, t * a.E + (lane_id() < a.K ? id : 0));
  return id;
}

// Lane k < K (`on`): the gate of the chosen logit zk, over scale.
template <bool SOFT>
__device__ __forceinline__ float gate_share(float zk, bool on, bool renorm, float shift,
                                            float inv) {
  if (!renorm) {
    if (!on) return 0.f;
    return SOFT ? exp_f(zk - shift) * inv : sigmoid_f(zk);
  }
  float s = on ? SOFT ? exp_f(zk) : sigmoid_f(zk) : 0.f;
  float sum = wave_sum_f(s);
  const bool plain = SOFT ? sum >= kPlainLo && sum <= kPlainHi : sum >= kSigmoidLo;
  if (!plain) {
    const float mk = wave_max_f(on ? zk : -INFINITY);
    if (SOFT || mk < kDeep) {
      s = on ? exp_f(mk > -INFINITY ? zk - mk : zk) : 0.f;
      sum = wave_sum_f(s);
    }
  }
  return s * recip(sum);
}

// The sequence that holds token t (the last one with cu[s] <= t), or -1, and
// where its tokens, or those of no sequence, end.  The lanes look at 64 places
// of cu at once: up to 63 sequences take one load instead of a chain of them.
__device__ __forceinline__ int sequence_of(const RouterArgs& a, int t, int& end) {
  end = a.T;
  if (!a.cu) return 0;
  int lo = -1, hi = a.nseq + 1;                   // cu[lo] <= t < cu[hi], as if cu[hi] = inf
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + (lane_id() + 1) * step;   // below 2^21 + 64 * 2^14
    const bool in = at < hi;
    const int c = in ? a.cu[at] : 0;
    const int n = (int)__popcll(ballot(in && c <= t));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  lo = min(lo, a.nseq);
  if (lo >= a.nseq) return -1;                    // behind the last sequence
  end = max(t + 1, min(a.cu[lo + 1], a.T));
  return lo;                                      // -1: before the first sequence
}

// ---------------------------------------------------------------------------
// Forward.  A workgroup owns `chunk` consecutive tokens, its waves take them in
// turn, each loading its next row before it works on the present one.  Where
// the loss is wanted, each wave keeps the sums of p in registers and the
// workgroup the counts in LDS; both go to row (workgroup + sequence) of the
// workspace when the sequence or the chunk ends.  Along the tokens either
// number grows, so no two pieces share a row.
//
// Bound by the vector units: 65,536 tokens of 384 experts (sigmoid, bias, K 8,
// loss) take 46 us, 282 vector instructions a token, where reading the logits
// takes 20; 262,144 bf16 tokens of 896 (softmax, K 16, loss) 205 us, 308 a token
// in 80 % of the cycles, reading 97.  Without a choice (given ids) it streams:
// 65,536 bf16 tokens of 384 in 11 us, 4.6 TB/s.  One wave a row, rather than 16
// lanes and four rows a wave, keeps the K-independent work (scores, sums) at one
// instruction per 64 experts and the row in P registers.
// ---------------------------------------------------------------------------
// Waves a SIMD.  Two leave 256 registers: 32,768 sigmoid rows of 1,024 experts
// with bias take 62-65 us with two, 65-76 with four and their spills; of a
// softmax 61-66 and 47-57.
template <int P, bool SOFT, bool BIAS>
constexpr int kForwardWaves = P < 16 || (P == 16 && (SOFT || !BIAS)) ? 4 : 2;

template <int P, bool BF16, bool FULL, bool SOFT, bool SELECT, bool BIAS, bool STATS>
__global__ __launch_bounds__(kRtThreads, (kForwardWaves<P, SOFT, BIAS>)) void k_router(RouterArgs a) {
  // BIAS: [64 P] bias, -inf past E (in registers it cost rows of 896 experts
  // spills: 81 us for 32,768 tokens, 51 so); STATS: [waves][E] sums, [E] counts
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int E = a.E, K = a.K;
  __shared__ __attribute__((aligned(16))) KeyList lists[SELECT ? kRtWaves : 1];
  KeyList& list = lists[SELECT ? wv : 0];
  int probe = kKeyNone;
  float* sum = lds + (BIAS ? 64 * P : 0);
  int* cnt = reinterpret_cast<int*>(sum + kRtWaves * E);
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  float acc[P];
  Row<P, BF16> next;
  if (t0 + wv < t1) load_row<P, BF16, FULL>(a.logits, t0 + wv, E, next);
  if constexpr (BIAS) {
    for (int e = threadIdx.x; e < 64 * P; e += kRtThreads) lds[e] = e < E ? a.bias[e] : -INFINITY;
    if constexpr (!STATS) __syncthreads();
  }
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
      if (lo != t0 && lo + wv < hi) load_row<P, BF16, FULL>(a.logits, lo + wv, E, next);
      for (int t = lo + wv; t < hi; t += kRtWaves) {
        float z[P], v[P], co[P];
        unpack_row<P, BF16, FULL>(next, E, z);
        if (t + kRtWaves < hi) load_row<P, BF16, FULL>(a.logits, t + kRtWaves, E, next);
        int id = -1;
        if constexpr (!SELECT) {
          if (lane < K) id = a.ids[int64_t(t) * K + lane];
        }
        float inv = 1.f, shift = 0.f;
        if (STATS || (SELECT && SOFT && (BIAS || !a.renorm)))
          inv = row_shares<P, BF16, FULL, SOFT, false>(a, t, z, v, co, shift);
        if constexpr (STATS) {
          if (seq >= 0) {
#pragma unroll
            for (int i = 0; i < P; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
          }
        }
        if constexpr (SELECT) {
          float zk;
          if constexpr (BIAS) {
            float m = 0.f;
            if constexpr (SOFT) m = wave_max_f(lane_max<P>(z));
            if (!SOFT && (!STATS || shift != 0.f)) {      // v holds no sigmoids
#pragma unroll
              for (int i = 0; i < P; ++i) v[i] = sigmoid_f(z[i]);
            }
            float least = z[0];
#pragma unroll
            for (int i = 0; i < P; i += 2) {
              const float2 b = *reinterpret_cast<const float2*>(lds + expert_of(i));
              least = fminf(least, fminf(z[i], z[i + 1]));
              v[i] = SOFT ? fmaf(v[i], inv, b.x) : v[i] + b.x;
              v[i + 1] = SOFT ? fmaf(v[i + 1], inv, b.y) : v[i + 1] + b.y;
            }
            if (ballot(least == -INFINITY)) {             // masked, whatever their bias
#pragma unroll
              for (int i = 0; i < P; ++i) v[i] = z[i] == -INFINITY ? -INFINITY : v[i];
            }
            id = choose_biased<P, BF16, SOFT>(a, t, m, v, inv, shift, probe, list, zk);
          } else {
            // a sum of shares that is a number has no NaN in it
            id = choose<P, BF16, FULL>(a, t, z, STATS && inv > 0.f, probe, list, zk);
          }
          const bool on = lane < K;
          const float w = gate_share<SOFT>(zk, on, a.renorm, shift, inv);
          if (on) {
            a.ids[int64_t(t) * K + lane] = id;
            a.gates[int64_t(t) * K + lane] = a.scale * w;
          }
        }
        if constexpr (STATS) {
          if (seq >= 0 && lane < K && (unsigned)id < (unsigned)E) atomicAdd(&cnt[id], 1);
        }
      }
    }
    if constexpr (STATS) {
      if (seq >= 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int e = expert_of(i);
          if (FULL || i < kSure<P> || e < E) sum[wv * E + e] = acc[i];
        }
      }
      __syncthreads();
      if (seq >= 0) {
        const int64_t row = int64_t(blockIdx.x + seq) * E;
        for (int e = threadIdx.x; e < E; e += kRtThreads) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < kRtWaves; ++w) s += sum[w * E + e];
          a.part_p[row + e] = s;
          a.part_c[row + e] = cnt[e];
        }
      }
      __syncthreads();                            // cnt is cleared next
    }
    lo = hi;
  }
}

// Calls f with the registers per lane of a row of E experts, the type, and
// whether the row fills all lanes.  The counts are close where experts are
// many: 32,768 rows of 1,024 experts take 38 us in 16 registers, 98 in 20.
template <typename F>
inline int with_row(int E, bool bf16, F f) {
  const int p = 2 * ((E + 127) / 128);
#define MOE_ROW(N)                                                                      \
  if (p <= N) {                                                                         \
    constexpr std::integral_constant<int, N> n;                                         \
    if (E == 64 * N)                                                                    \
      return bf16 ? f(n, std::true_type(), std::true_type())                            \
                  : f(n, std::false_type(), std::true_type());                          \
    return bf16 ? f(n, std::true_type(), std::false_type())                             \
                : f(n, std::false_type(), std::false_type());                           \
  }
  MOE_ROW(2)
  MOE_ROW(4)
  MOE_ROW(6)
  MOE_ROW(8)
  MOE_ROW(12)
  MOE_ROW(14)
  MOE_ROW(16)
  MOE_ROW(20)
  MOE_ROW(32)
#undef MOE_ROW
  return MOE_ELIMIT;
}

// Launches the forward for one score function (instantiated in
// router_softmax.hip and router_sigmoid.hip, which compile side by side).
template <bool SOFT>
int launch_forward(const RouterArgs& a, bool bf16, bool select, bool stats, int grid,
                   hipStream_t stream) {
  const size_t stats_lds = stats ? size_t(kRtWaves + 1) * a.E * 4 : 0;
  return with_row(a.E, bf16, [&](auto p, auto b, auto full) {
    constexpr int P = decltype(p)::value;
    constexpr bool BF = decltype(b)::value, FULL = decltype(full)::value;
    const dim3 g(grid), t(kRtThreads);
    const size_t lds = stats_lds + (select && a.bias ? size_t(64) * P * 4 : 0);
    int rc = MOE_OK;
#define MOE_ROUTER(SEL, BIAS, STATS)                                         \
  do {                                                                       \
    auto* k = k_router<P, BF, FULL, SOFT, SEL, BIAS, STATS>;                 \
    rc = allow_lds(k, lds + (SEL ? sizeof(KeyList) * kRtWaves : 0));         \
    if (rc == MOE_OK) hipLaunchKernelGGL(k, g, t, lds, stream, a);           \
  } while (0)
    if (!select) MOE_ROUTER(false, false, true);
    else if (stats && a.bias) MOE_ROUTER(true, true, true);
    else if (stats) MOE_ROUTER(true, false, true);
    else if (a.bias) MOE_ROUTER(true, true, false);
    else MOE_ROUTER(true, false, false);
#undef MOE_ROUTER
    return rc == MOE_OK ? hip_status() : rc;
  });
}

extern template int launch_forward<true>(const RouterArgs&, bool, bool, bool, int, hipStream_t);
extern template int launch_forward<false>(const RouterArgs&, bool, bool, bool, int, hipStream_t);

}  // namespace moonep
