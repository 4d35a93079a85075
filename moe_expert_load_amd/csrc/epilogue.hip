// Backward of the product's epilogue (epilogue.hpp): dz = act'(pre) times what
// dropout leaves of dy, and the biases' gradients, the sums of dz over the rows
// of each expert.
//
// One pass over dy and pre.  The rows are cut into pieces of at most kEbRows
// rows of one segment; a workgroup takes a piece and 512 columns, a lane eight
// columns (16-byte loads, 1 KB a wave), its four waves the piece's rows in turn,
// and the sums over the piece's rows stay in registers.  They are joined over
// the waves in LDS and written once per piece, 1/kEbRows of the traffic; a
// second kernel adds an expert's pieces in a fixed order (rank by rank, rows in
// order), so no atomics.  The list of pieces comes from cu_seqlens on the device.
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
  int32_t* base;               // [segs * R + R + 1] first piece of each segment
  int2* pieces;                // row, rows
  float* part;                 // [pieces][N]
  int64_t rows;
  int32_t R, E, B, SK, N, act, piece_rows, max_pieces, col_tiles;
  uint32_t cut;
  float scale;
};

// Rows of a piece: enough pieces to fill the chip several times, and at 256
// the sums' own traffic is below half a percent.
static int eb_piece_rows(int64_t rows) {
  int p = 16;
  while (p < 256 && rows / p > 4096) p *= 2;
  return p;
}

// Pieces of all segments, rank by rank; a rank's rows after its last segment
// (all of them if its plan failed) follow as one more, which no expert owns.
__global__ __launch_bounds__(1024) void k_eb_pieces(EbArgs a) {
  __shared__ int s_part[17];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int per = a.E + a.B + 1, total = a.R * per;
  int carry = 0;
  for (int c0 = 0; c0 < total; c0 += 1024) {
    const int i = c0 + tid;
    int row0 = 0, len = 0;
    if (i < total) {
      const int r = i / per, j = i % per;
      const int32_t* cu = a.cu + int64_t(r) * per;
      const int lo = cu[j], hi = j + 1 < per ? cu[j + 1] : a.SK;
      row0 = r * a.SK + lo;
      len = max(0, hi - lo);
    }
    const int n = (len + a.piece_rows - 1) / a.piece_rows;
    const int incl = wave_incl_scan(n);
    if (lane == kWave - 1) s_part[wave] = incl;
    __syncthreads();
    if (wave == 0) {
      const int x = lane < 16 ? s_part[lane] : 0;
      const int xi = wave_incl_scan(x);
      if (lane < 16) s_part[lane] = xi - x;
      if (lane == 15) s_part[16] = xi;
    }
    __syncthreads();
    const int at = carry + s_part[wave] + incl - n;
    carry += s_part[16];
    if (i < total) a.base[i] = at;
    for (int m = 0; m < n; ++m)
      if (at + m < a.max_pieces)
        a.pieces[at + m] = int2{row0 + m * a.piece_rows, min(a.piece_rows, len - m * a.piece_rows)};
    __syncthreads();
  }
  if (tid == 0) a.base[total] = min(carry, a.max_pieces);
}

// Loads of U rows go out before the first of them is used or stored, so dz may
// be what is read.
template <typename D, int U>
__global__ __launch_bounds__(256) void k_eb(EbArgs a) {
  __shared__ f32x4 s_sum[3][2][kWave];
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int pieces = a.cu ? a.base[a.R * (a.E + a.B + 1)] : a.max_pieces;
  const int64_t work = int64_t(pieces) * a.col_tiles;
  DropKey key{};
  if (a.cut) key = drop_key(a.rng);
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int piece = int(w / a.col_tiles), ct = int(w % a.col_tiles);
    int64_t row0 = int64_t(piece) * a.piece_rows;
    int rows = (int)min(int64_t(a.piece_rows), a.rows - row0);
    if (a.cu) {
      const int2 p = a.pieces[piece];
      row0 = p.x;
      rows = p.y;
    }
    const int n = ct * kEbCols + lane * 8;
    const bool on = n < a.N;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    for (int m0 = on ? wv : rows; m0 < rows; m0 += 4 * U) {
      float d[U][8], z[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // a row past the piece is its last one again, and is left out below
        const int64_t at = (row0 + min(m0 + 4 * u, rows - 1)) * a.N + n;
        load8(static_cast<const D*>(a.dy) + at, d[u]);
        if (a.act != MOE_ACT_NONE) load8(a.pre + at, z[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (m0 + 4 * u >= rows) break;
        const int64_t at = (row0 + m0 + 4 * u) * a.N + n;
        if (a.cut) drop8(d[u], key, uint64_t(at) >> 3, a.cut, a.scale);
        if (a.act != MOE_ACT_NONE) act_grad8(d[u], z[u], a.act);
        if (a.dz) store8(a.dz + at, d[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += d[u][i];
      }
    }
    if (!a.dbias) continue;
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
      store8(a.part + int64_t(piece) * a.N + n, sum);
    }
    __syncthreads();
  }
}

// dbias[e]: workgroup (columns, expert), 32 lanes of four columns, eight rows of
// lanes taking the expert's pieces in turn.
__global__ __launch_bounds__(256) void k_eb_bias(EbArgs a) {
  __shared__ int2 s_seg[MOE_MAX_E + MOE_MAX_R];     // first piece, pieces
  __shared__ int s_part[4];
  __shared__ f32x4 s_sum[8][32];
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
          const int at = r * per + (b == 0 ? e : a.E + b - 1);
          seg = int2{a.base[at], a.base[at + 1] - a.base[at]};
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
    if (tid == 0) s_seg[0] = int2{0, a.max_pieces};
    __syncthreads();
  }
  const int n = blockIdx.x * 128 + (tid & 31) * 4, y = tid >> 5;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (n < a.N) {
    for (int s = 0; s < segs; ++s) {
      const int2 seg = s_seg[s];
#pragma unroll 4
      for (int p = y; p < seg.y; p += 8) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + int64_t(seg.x + p) * a.N + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[i];
      }
    }
  }
  s_sum[y][tid & 31] = sum;
  __syncthreads();
  if (y > 0 || n >= a.N) return;
#pragma unroll
  for (int u = 1; u < 8; ++u) {
    const f32x4 v = s_sum[u][tid];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += v[i];
  }
  *reinterpret_cast<f32x4*>(a.dbias + int64_t(e) * a.N + n) = sum;
}

static int64_t eb_max_pieces(const moe_cfg* c) {
  const int64_t rows = int64_t(c->R) * c->S * c->K, p = eb_piece_rows(rows);
  return (rows + p - 1) / p + int64_t(c->R) * (c->E + c->B + 1);
}

static size_t eb_list_bytes(const moe_cfg* c) {
  return align256((size_t(c->R) * (c->E + c->B + 1) + 1) * 4) + align256(size_t(eb_max_pieces(c)) * 8);
}

size_t epilogue_bwd_ws_bytes(const moe_cfg* c) {
  return eb_list_bytes(c) + size_t(eb_max_pieces(c)) * c->Hp * 4;
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
    if (!dy || (a.cut && !rng) || (ec->act != MOE_ACT_NONE && !pre)) return MOE_EINVAL;
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
  a.piece_rows = eb_piece_rows(rows);
  a.col_tiles = (cfg->Hp + kEbCols - 1) / kEbCols;
  a.max_pieces = (int32_t)(lists ? eb_max_pieces(cfg) : (rows + a.piece_rows - 1) / a.piece_rows);
  if (dbias) {
    char* w = static_cast<char*>(workspace);
    a.base = reinterpret_cast<int32_t*>(w);
    a.pieces = reinterpret_cast<int2*>(w + align256((size_t(cfg->R) * (cfg->E + cfg->B + 1) + 1) * 4));
    a.part = reinterpret_cast<float*>(w + eb_list_bytes(cfg));
  }
  if (rows > 0) {
    // (a launch holds fewer than 2^32 threads)
    const dim3 grid((unsigned)std::min<int64_t>(int64_t(a.max_pieces) * a.col_tiles, 1 << 20)),
        block(256);
    if (lists) hipLaunchKernelGGL(k_eb_pieces, dim3(1), dim3(1024), 0, stream, a);
    if (ec->f32) hipLaunchKernelGGL((k_eb<float, 2>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_eb<uint16_t, 2>), grid, block, 0, stream, a);
  } else {
    a.cu = nullptr;                                    // no pieces: zeros
    a.max_pieces = 0;
  }
  if (dbias)
    hipLaunchKernelGGL(k_eb_bias, dim3((cfg->Hp + 127) / 128, cfg->E), dim3(256), 0, stream, a);
  return hip_status();
}
