// Backward of the product's epilogue (epilogue.hpp): dz = act'(pre) times what
// dropout leaves of dy, and the biases' gradients, the sums of dz over the rows
// of each expert.
//
// One pass over dy and pre, bound by memory.  The rows are cut into chunks; a
// workgroup takes a chunk and 512 columns, a lane eight columns (16-byte loads, 1
// KB a wave), its four waves the rows in turn, and the sums over the rows of one
// segment stay in registers.  Where a segment or the chunk ends they are joined
// over the waves in LDS and written: segment s (counted over all ranks) has its
// part of chunk c at place c + s, which no other pair has and which needs no
// list.  A second kernel adds an expert's parts in a fixed order (rank by rank,
// rows in order): no atomics.
#include <algorithm>

#include "epilogue.hpp"
#include "host.hpp"
#include "overlap.hpp"

namespace moonep {

constexpr int kEbCols = 512;

struct EbArgs {
  const void* dy;
  const uint16_t* pre;
  const int64_t* rng;
  uint16_t* dz;
  float* dbias;
  const int32_t* cu;           // null: one matrix, or no sums wanted
  const int32_t* slot_expert;
  float* part;                 // [chunks + segments][N]
  int64_t rows;
  int32_t R, E, B, SK, N, act, chunk_rows, chunks, col_tiles;
  uint32_t cut;
  float scale;
};

// Rows of a chunk: enough workgroups to fill the chip several times over, and at
// most 256 rows, where the parts' own traffic is below half a percent.
static int eb_chunk_rows(int64_t rows, int col_tiles) {
  int p = 16;
  while (p < 256 && rows / p * col_tiles > 4096) p *= 2;
  return p;
}

// The segment of row `row` of its rank's buffer (cu its prefix over n segments):
// the number of segments that end at or before it, n for a row after the last.
// One look by the whole wave.
__device__ __forceinline__ int segment_of(const int32_t* cu, int n, int row) {
  int before = 0;
  for (int j = lane_id(); j < n; j += kWave) before += cu[j + 1] <= row ? 1 : 0;
  return wave_sum(before);
}

// Blocks of 4 U rows, U a wave: their loads go out first, before the block's
// segments are known and before any of them is stored, so dz may be what is read.
// 524,288 rows of 2,048 over 384 experts, gelu, bf16, in cold memory 1.24 to 1.32
// ms with dropout (5.2 to 4.9 TB/s), up to 1.5 in the first ten launches after a pause;
// 3 % more through the caches.
template <typename D, int U>
__global__ __launch_bounds__(256) void k_eb(EbArgs a) {
  __shared__ f32x4 s_sum[3][2][kWave];
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int64_t work = int64_t(a.chunks) * a.col_tiles;
  const int segs = a.E + a.B;
  DropKey key{};
  if (a.cut) key = drop_key(a.rng);
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int chunk = int(w / a.col_tiles), n = int(w % a.col_tiles) * kEbCols + lane * 8;
    const bool on = n < a.N;
    const int64_t from = int64_t(chunk) * a.chunk_rows;
    const int64_t end = min(from + a.chunk_rows, a.rows);
    // the segment of row `row` and the row after its last (always ahead of
    // `row`, whatever cu holds: the loops end)
    int seg = 0;
    int64_t stop = end + 1;
    auto find = [&](int64_t row) {
      if (!a.cu) return;
      const int r = int(row / a.SK);
      const int32_t* cu = a.cu + int64_t(r) * (segs + 1);
      const int j = segment_of(cu, segs, int(row - int64_t(r) * a.SK));
      seg = r * (segs + 1) + j;
      stop = max(row + 1, int64_t(r) * a.SK + (j < segs ? cu[j + 1] : a.SK));
    };
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    // the waves' sums joined and written; the next segment starts from zero
    auto flush = [&]() {
      if (wv > 0) {
        s_sum[wv - 1][0][lane] = f32x4{sum[0], sum[1], sum[2], sum[3]};
        s_sum[wv - 1][1][lane] = f32x4{sum[4], sum[5], sum[6], sum[7]};
      }
      __syncthreads();
      if (wv == 0 && on) {
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const f32x4 lo = s_sum[u][0][lane], hi = s_sum[u][1][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[i] += lo[i];
            sum[4 + i] += hi[i];
          }
        }
        store8(a.part + (int64_t(chunk) + seg) * a.N + n, sum);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    };
    for (int64_t row = from; row < end; row += 4 * U) {
      const int have = int(min(int64_t(4 * U), end - row));
      float d[U][8], z[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[u][i] = z[u][i] = 0.f;
        // a row past the last is the last again, and is left out below
        const int64_t at = (row + min(wv + 4 * u, have - 1)) * a.N + n;
        if (on) {
          load8_once(static_cast<const D*>(a.dy) + at, d[u]);
          if (a.act != MOE_ACT_NONE) load8_once(a.pre + at, z[u]);
        }
      }
      if (a.dbias && row == from) find(row);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (wv + 4 * u >= have) break;                    // uniform
        const int64_t at = (row + wv + 4 * u) * a.N + n;
        if (a.cut) drop8(d[u], key, uint64_t(at) >> 3, a.cut, a.scale);
        if (a.act != MOE_ACT_NONE) act_grad8(d[u], z[u], a.act);
        if (a.dz && on) store8_once(a.dz + at, d[u]);
      }
      if (!a.dbias) continue;
      // the block's rows segment by segment
      for (int done = 0; done < have;) {
        const int lim = (int)min(int64_t(have), stop - row);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (wv + 4 * u >= done && wv + 4 * u < lim)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += d[u][i];
        done = lim;
        if (row + done == stop) {
          flush();
          if (stop < end) find(stop);
        }
      }
    }
    if (a.dbias && stop > end) flush();
  }
}

// dbias[e]: workgroup (64 columns, expert), 16 lanes of four columns, 16 rows of
// lanes taking the expert's parts in turn.  Bound by reading the parts: 22 us for
// the 524,288 rows above, 4 us (latency) for 4,100 of 520.
__global__ __launch_bounds__(256) void k_eb_bias(EbArgs a) {
  __shared__ int2 s_seg[MOE_MAX_E + MOE_MAX_R];     // first part, parts
  __shared__ int s_part[4];
  __shared__ f32x4 s_sum[16][16];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int e = blockIdx.y;
  int segs = 0;
  if (a.cu) {
    // the segments that hold rows of expert e, rank by rank
    const int per = a.E + a.B + 1, cand = a.R * (a.B + 1);
    for (int c0 = 0; c0 < cand; c0 += 256) {
      const int i = c0 + tid;
      int2 seg{0, 0};
      if (i < cand) {
        const int r = i / (a.B + 1), b = i % (a.B + 1);
        if (b == 0 || a.slot_expert[int64_t(r) * a.B + b - 1] == e) {
          const int j = b == 0 ? e : a.E + b - 1;
          const int32_t* cu = a.cu + int64_t(r) * per + j;
          const int64_t lo = int64_t(r) * a.SK + cu[0], hi = int64_t(r) * a.SK + cu[1];
          if (lo < hi) {
            const int c = int(lo / a.chunk_rows);
            seg = int2{c + r * per + j, int((hi - 1) / a.chunk_rows) - c + 1};
          }
        }
      }
      const uint64_t any = __ballot(seg.y > 0);
      if (lane == 0) s_part[wave] = (int)__popcll(any);
      __syncthreads();
      int at = segs + (int)__popcll(any & lanemask_lt());
      for (int q = 0; q < 4; ++q) {
        if (q < wave) at += s_part[q];
        segs += s_part[q];
      }
      if (seg.y > 0) s_seg[at] = seg;
      __syncthreads();
    }
  } else {
    segs = 1;
    if (tid == 0) s_seg[0] = int2{0, a.chunks};
    __syncthreads();
  }
  const int y = tid >> 4;
  for (int64_t c0 = int64_t(blockIdx.x) * 64; c0 < a.N; c0 += int64_t(gridDim.x) * 64) {
    const int n = int(c0) + (tid & 15) * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (n < a.N) {
      for (int s = 0; s < segs; ++s) {
        const int2 seg = s_seg[s];
#pragma unroll 4
        for (int p = y; p < seg.y; p += 16) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + int64_t(seg.x + p) * a.N + n);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] += v[i];
        }
      }
    }
    s_sum[y][tid & 15] = sum;
    __syncthreads();
    if (y == 0 && n < a.N) {
#pragma unroll
      for (int u = 1; u < 16; ++u) {
        const f32x4 v = s_sum[u][tid];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[i];
      }
      *reinterpret_cast<f32x4*>(a.dbias + int64_t(e) * a.N + n) = sum;
    }
    __syncthreads();
  }
}

static int eb_col_tiles(const moe_cfg* c) { return (c->Hp + kEbCols - 1) / kEbCols; }

static int64_t eb_chunks(const moe_cfg* c) {
  const int64_t rows = int64_t(c->R) * c->S * c->K, p = eb_chunk_rows(rows, eb_col_tiles(c));
  return (rows + p - 1) / p;
}

size_t epilogue_bwd_ws_bytes(const moe_cfg* c) {
  return size_t(eb_chunks(c) + int64_t(c->R) * (c->E + c->B + 1)) * c->Hp * 4;
}

}  // namespace moonep

using namespace moonep;

extern "C" int moe_epilogue_backward(const moe_cfg* cfg, const moe_epilogue_cfg* ec,
                                     const moe_plan* plan, const void* dy, const moe_bf16* pre,
                                     const int64_t* rng, moe_bf16* dz, float* dbias,
                                     void* workspace, hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  if (!valid_epilogue(ec) || (!dz && !dbias)) return MOE_EINVAL;
  if (dbias && !plan && !one_matrix(cfg)) return MOE_EINVAL;
  const int64_t rows = int64_t(cfg->R) * cfg->S * cfg->K;
  EbArgs a{};
  drop_params(ec->p, &a.cut, &a.scale);
  if (rows > 0) {
    if (!dy || !rng_ok(rng, a.cut) || (ec->act != MOE_ACT_NONE && !pre)) return MOE_EINVAL;
  }
  if (dbias && !workspace) return MOE_EINVAL;
  if (dbias && plan && (!plan->cu_seqlens || (cfg->B > 0 && !plan->slot_expert))) return MOE_EINVAL;
  if (!aligned16(dy, pre, dz, dbias, dbias ? workspace : nullptr)) return MOE_EINVAL;
  const int64_t n = rows * cfg->Hp, ein = n * (ec->f32 ? 4 : 2);
  const int64_t sums = int64_t(cfg->E) * cfg->Hp * 4, ws = dbias ? epilogue_bwd_ws_bytes(cfg) : 0;
  const bool lists = dbias && plan;
  const bool on_dy = static_cast<const void*>(dz) == dy && !ec->f32;
  if (clash({{dz, n * 2}, {dbias, sums}, {workspace, ws}},
            {{on_dy ? nullptr : dy, ein},
             {dz == pre ? nullptr : pre, n * 2},
             {a.cut ? rng : nullptr, 16},
             {lists ? plan->cu_seqlens : nullptr, int64_t(cfg->R) * (cfg->E + cfg->B + 1) * 4},
             {lists && cfg->B ? plan->slot_expert : nullptr, int64_t(cfg->R) * cfg->B * 4}}) ||
      clash({{dbias, sums}, {workspace, ws}}, {{dy, ein}, {pre, n * 2}}))
    return MOE_EINVAL;
  a.dy = dy; a.pre = pre; a.rng = rng; a.dz = dz; a.dbias = dbias;
  a.cu = lists ? plan->cu_seqlens : nullptr;
  a.slot_expert = lists ? plan->slot_expert : nullptr;
  a.rows = rows; a.R = cfg->R; a.E = cfg->E; a.B = cfg->B; a.SK = cfg->S * cfg->K;
  a.N = cfg->Hp; a.act = ec->act;
  a.col_tiles = eb_col_tiles(cfg);
  a.chunk_rows = eb_chunk_rows(rows, a.col_tiles);
  a.chunks = (int32_t)eb_chunks(cfg);
  a.part = static_cast<float*>(workspace);
  if (rows > 0) {
    // (a launch holds fewer than 2^32 threads)
    const dim3 grid((unsigned)std::min<int64_t>(int64_t(a.chunks) * a.col_tiles, 1 << 20)),
        block(256);
    // all rows of the smallest chunk at once: its time is the latency of one look
    // (4,100 rows of 520: 12.5 us by two rows a wave, 10.7 by four); in long chunks
    // fewer registers pay (1.27 against 1.30 ms)
    if (a.chunk_rows == 16) {
      if (ec->f32) hipLaunchKernelGGL((k_eb<float, 4>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_eb<uint16_t, 4>), grid, block, 0, stream, a);
    } else {
      if (ec->f32) hipLaunchKernelGGL((k_eb<float, 2>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_eb<uint16_t, 2>), grid, block, 0, stream, a);
    }
  } else {
    a.cu = nullptr;                                    // no parts: zeros
  }
  if (dbias)
    hipLaunchKernelGGL(k_eb_bias, dim3(std::min(4096, (cfg->Hp + 63) / 64), cfg->E), dim3(256), 0,
                       stream, a);
  return hip_status();
}
