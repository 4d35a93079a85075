// Product of few rows with large weights, and the epilogue (epilogue.hpp): the
// single tokens of decoding, and row counts whose 256 x 256 tiles would leave
// most of the chip idle.  The time is that of reading the weights once, so they
// go from memory to registers and nowhere else, and every wave of the chip
// takes part in every matrix:
//
//  * a wave takes 128 columns and steps of 32 k.  Lane l loads rows k0 + 8 (l /
//    16) + 0 .. 7 of columns n0 + 8 (l % 16) + 0 .. 7, eight 16-byte loads of
//    which every 16 lanes cover 256 contiguous bytes.  A matrix instruction
//    wants eight consecutive k of one column per lane; a lane has an 8 x 8
//    block, whose transposition is 32 byte permutes (pairs of rows; larger
//    strides only rename registers).  Instruction i then multiplies columns
//    n0 + 8 (l % 16) + i, and a lane ends with eight consecutive columns of a
//    row: one group of the epilogue.  No LDS on the way.
//  * the k axis is cut over the four waves of a workgroup (joined in LDS) and
//    over workgroups until there are about kFewItems of them; their sums go to
//    the workspace in fp32 and a second launch adds them in a fixed order and
//    applies the epilogue.
#include "few.hpp"

#include <algorithm>

#include "host.hpp"

namespace moonep {

typedef __bf16 few_bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kFewCols = 128;        // columns of a wave
constexpr int kFewStep = 32;         // k of a step
constexpr int kFewItems = 512;       // workgroups wanted: two on every compute unit
constexpr int kFewSteps = 8;         // least steps of a workgroup: two per wave
constexpr int kFewMaxBlocks = 1024;  // row blocks of a grouped call
constexpr int kFewGrid = 1024;       // workgroups of a grouped call

struct FewArgs {
  const uint16_t* x;
  const uint16_t* w_home;
  const uint16_t* w_pref;
  const int32_t* cu;         // null: one matrix
  float* partial;            // [splits][rows][N]
  int32_t* hdr;              // [0]: splits
  int32_t* row_expert;       // [rows], grouped
  int32_t H, E, B, SK, first_rank, nranks;
  int32_t rows, strips, steps;
  int32_t blocks, splits;    // of one matrix; grouped: splits is the most there may be
  Epilogue ep;
};

// Splits of the k axis for this many row blocks.
__host__ __device__ inline int few_splits(int blocks, int strips, int steps, int most) {
  const int want = kFewItems / max(1, blocks * strips), room = (steps + kFewSteps - 1) / kFewSteps;
  return max(1, min(most, min(want, room)));
}

// Columns 2j and 2j + 1 of an 8 x 8 block as eight consecutive k each.
__device__ __forceinline__ void column_pair(const u32x4 (&w)[8], int j, few_bf16x8& even,
                                            few_bf16x8& odd) {
  u32x4 e, o;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    e[q] = __builtin_amdgcn_perm(w[2 * q + 1][j], w[2 * q][j], 0x05040100u);
    o[q] = __builtin_amdgcn_perm(w[2 * q + 1][j], w[2 * q][j], 0x07060302u);
  }
  even = __builtin_bit_cast(few_bf16x8, e);
  odd = __builtin_bit_cast(few_bf16x8, o);
}

// RB: blocks of 16 rows that a workgroup takes.
template <int RB>
__global__ __launch_bounds__(256, RB == 4 ? 1 : 2) void k_few(FewArgs a) {
  __shared__ int4 s_list[kFewMaxBlocks];
  __shared__ int s_part[5];
  __shared__ f32x4 s_sum[4 * 3 * RB * kWave * 2];
  const int tid = threadIdx.x, lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int H = a.H, N = a.ep.N;
  int blocks = a.blocks;
  if (a.cu) {
    // the listed ranks' segments as row blocks, in layout order
    const int per = a.E + a.B, total = a.nranks * per;
    blocks = 0;
    for (int c0 = 0; c0 < total; c0 += 256) {
      const int i = c0 + tid;
      int r = 0, j = 0, lo = 0, len = 0;
      if (i < total) {
        r = a.first_rank + i / per;
        j = i % per;
        const int32_t* cu = a.cu + int64_t(r) * (per + 1);
        lo = cu[j];
        len = cu[j + 1] - lo;
      }
      const int n = (len + 16 * RB - 1) / (16 * RB);
      const int incl = wave_incl_scan(n);
      if (lane == kWave - 1) s_part[wv] = incl;
      __syncthreads();
      int at = blocks + incl - n;
      for (int q = 0; q < 4; ++q) {
        if (q < wv) at += s_part[q];
        blocks += s_part[q];
      }
      for (int m = 0; m < n; ++m)
        if (at + m < kFewMaxBlocks)
          s_list[at + m] = int4{r, j, r * a.SK + lo + m * 16 * RB, min(16 * RB, len - m * 16 * RB)};
      __syncthreads();
    }
    blocks = min(blocks, kFewMaxBlocks);
  }
  const int units = blocks * a.strips;
  const int splits = a.cu ? few_splits(blocks, a.strips, a.steps, a.splits) : a.splits;
  if (a.cu && blockIdx.x == 0 && tid == 0) a.hdr[0] = splits;
  const int items = units * splits;
  DropKey key{};
  if (a.ep.cut && splits == 1) key = drop_key(a.ep.rng);

  // Neighbouring items (the row blocks of one piece of the weights) go to one
  // XCD, whose L2 then reads it once.
  const int per = (items + 7) / 8;
  for (int q = blockIdx.x / 8; q < per; q += gridDim.x / 8) {
    const int item = (blockIdx.x % 8) * per + q;
    if (item >= items) break;
    const int blk = item % blocks, rest = item / blocks;
    const int n0 = (rest % a.strips) * kFewCols, split = rest / a.strips;
    int r = 0, j = 0, row0 = blk * 16 * RB, rows = min(16 * RB, a.rows - row0);
    if (a.cu) {
      const int4 it = s_list[blk];
      r = __builtin_amdgcn_readfirstlane(it.x);
      j = __builtin_amdgcn_readfirstlane(it.y);
      row0 = __builtin_amdgcn_readfirstlane(it.z);
      rows = __builtin_amdgcn_readfirstlane(it.w);
    }
    const int n = n0 + 8 * (lane & 15);
    const char* w = reinterpret_cast<const char*>(
        j < a.E ? a.w_home + int64_t(j) * H * N : a.w_pref + (int64_t(r) * a.B + (j - a.E)) * H * N);
    const char* x = reinterpret_cast<const char*>(a.x + int64_t(row0) * H);
    // rows past the block's and columns past the matrix read the first ones:
    // what they give is not stored
    const uint32_t wcol = 2u * (n < N ? n : 0);
    uint32_t xrow[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int m = 16 * b + (lane & 15);
      xrow[b] = 2u * uint32_t(m < rows ? m : 0) * H;
    }
    f32x4 acc[8][RB];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int t0 = int(int64_t(split) * a.steps / splits);
    const int t1 = int(int64_t(split + 1) * a.steps / splits);
    auto load = [&](int t, u32x4 (&wr)[8], u32x4 (&xr)[RB]) {
      const int k = t * kFewStep + 8 * (lane >> 4);
      const bool in = k < H;
      const uint32_t wk = wcol + 2u * uint32_t(in ? k : 0) * N;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        wr[q] = *reinterpret_cast<const u32x4*>(w + (wk + 2u * uint32_t(q) * N));
#pragma unroll
      for (int b = 0; b < RB; ++b)
        xr[b] = *reinterpret_cast<const u32x4*>(x + (xrow[b] + 2u * uint32_t(in ? k : 0)));
    };
    auto multiply = [&](int t, u32x4 (&wr)[8], u32x4 (&xr)[RB]) {
      if ((t + 1) * kFewStep > H && t * kFewStep + 8 * (lane >> 4) >= H) {
        // k past the end: zeros on both sides (0 times infinity is none)
#pragma unroll
        for (int q = 0; q < 8; ++q) wr[q] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < RB; ++b) xr[b] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        few_bf16x8 even, odd;
        column_pair(wr, jj, even, odd);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const few_bf16x8 xa = __builtin_bit_cast(few_bf16x8, xr[b]);
          acc[2 * jj][b] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, even, acc[2 * jj][b], 0, 0, 0);
          acc[2 * jj + 1][b] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, odd, acc[2 * jj + 1][b], 0, 0, 0);
        }
      }
    };
    // two steps in flight
    u32x4 w0[8], w1[8], x0[RB], x1[RB];
    int t = t0 + wv;
    if (t < t1) load(t, w0, x0);
    for (; t < t1; t += 8) {
      if (t + 4 < t1) load(t + 4, w1, x1);
      multiply(t, w0, x0);
      if (t + 4 >= t1) break;
      if (t + 8 < t1) load(t + 8, w0, x0);
      multiply(t + 4, w1, x1);
    }

    // Register v of an accumulator is row 4 (l / 16) + v of its block: wave v
    // sums those rows of the four waves.
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (v == wv) continue;
      f32x4* to = s_sum + (v * 3 + (wv < v ? wv : wv - 1)) * RB * kWave * 2;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        to[(b * 2 + 0) * kWave + lane] = f32x4{acc[0][b][v], acc[1][b][v], acc[2][b][v], acc[3][b][v]};
        to[(b * 2 + 1) * kWave + lane] = f32x4{acc[4][b][v], acc[5][b][v], acc[6][b][v], acc[7][b][v]};
      }
    }
    __syncthreads();
    float bias[8];
    if (splits == 1) bias8(a.ep, expert_of(a.ep, r, j, a.E, a.B), a.E, n, bias);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float z[8];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v == wv)
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = acc[i][b][v];
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const f32x4* from = s_sum + ((wv * 3 + u) * RB + b) * kWave * 2;
        const f32x4 lo = from[lane], hi = from[kWave + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[i] += lo[i];
          z[4 + i] += hi[i];
        }
      }
      const int m = 16 * b + 4 * (lane >> 4) + wv;
      if (m >= rows || n >= N) continue;
      const int64_t row = int64_t(row0) + m;
      if (splits == 1) {
        epilogue8(a.ep, key, z, bias, row, n);
      } else {
        const int64_t at = row - int64_t(a.first_rank) * a.SK;
        store8(a.partial + (int64_t(split) * a.rows + at) * N + n, z);
        if (a.cu && n == 0 && split == 0) a.row_expert[at] = expert_of(a.ep, r, j, a.E, a.B);
      }
    }
    __syncthreads();
  }
}

// Sums of the splits in ascending order, and the epilogue.
__global__ __launch_bounds__(256) void k_few_join(FewArgs a) {
  const int splits = a.cu ? a.hdr[0] : a.splits;
  if (splits <= 1) return;                          // done already
  const int64_t nv = a.ep.N / 8, g = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (g >= nv * a.rows) return;
  const int64_t at = g / nv;
  const int n = int(g % nv) * 8;
  DropKey key{};
  if (a.ep.cut) key = drop_key(a.ep.rng);
  float b[8];
  bias8(a.ep, a.cu ? a.row_expert[at] : 0, a.E, n, b);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0.f;
  const float* p = a.partial + at * a.ep.N + n;
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    float v[8];
    load8(p + int64_t(s) * a.rows * a.ep.N, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += v[i];
  }
  epilogue8(a.ep, key, z, b, at + int64_t(a.first_rank) * a.SK, n);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int64_t kFewGroupedRows = 512;

static int few_block_rows(const moe_cfg* c, bool dense, int64_t rows) {
  const int64_t ranks = rows / (int64_t(c->S) * c->K);
  const int64_t mean = dense ? rows : rows / (ranks * (c->E + c->B));
  return mean <= 16 ? 16 : mean <= 32 ? 32 : 64;
}

bool few_rows(const moe_cfg* c, bool dense, int64_t nranks, int cus) {
  const int64_t rows = nranks * c->S * c->K;
  if (rows == 0) return false;
  if (!dense) return rows <= kFewGroupedRows;
  return rows <= 1024;
}

// The most splits that a call of `rows` rows can have, and its bytes.
static int few_most_splits(const moe_cfg* c, bool dense, int64_t rows) {
  const int bm = few_block_rows(c, dense, rows);
  return few_splits(int((rows + bm - 1) / bm), (c->Hp + kFewCols - 1) / kFewCols,
                    (c->H + kFewStep - 1) / kFewStep, 1 << 30);
}

static size_t few_bytes(const moe_cfg* c, bool dense, int64_t rows) {
  const int splits = few_most_splits(c, dense, rows);
  return 256 + align256(size_t(rows) * 4) + (splits > 1 ? size_t(splits) * rows * c->Hp * 4 : 0);
}

size_t few_ws_bytes(const moe_cfg* c) {
  size_t most = 0;
  if (c->S == 0) return most;
  for (int64_t n = 1; n <= c->R && few_rows(c, false, n, 0); ++n)
    most = std::max(most, few_bytes(c, false, n * c->S * c->K));
  if (one_matrix(c)) most = std::max(most, few_bytes(c, true, c->S));
  return most;
}

int launch_few(const moe_cfg* c, const uint16_t* x, const uint16_t* w_home, const uint16_t* w_pref,
               const int32_t* cu, const Epilogue& ep, int rank_begin, int rank_end, void* workspace,
               hipStream_t stream) {
  FewArgs a{};
  const bool dense = !cu;
  a.x = x; a.w_home = w_home; a.w_pref = w_pref; a.cu = cu; a.ep = ep;
  a.H = c->H; a.E = c->E; a.B = c->B; a.SK = c->S * c->K;
  a.first_rank = rank_begin; a.nranks = rank_end - rank_begin;
  a.rows = a.nranks * a.SK;
  a.strips = (c->Hp + kFewCols - 1) / kFewCols;
  a.steps = (c->H + kFewStep - 1) / kFewStep;
  const int bm = few_block_rows(c, dense, a.rows);
  a.blocks = (a.rows + bm - 1) / bm;
  a.splits = few_most_splits(c, dense, a.rows);
  char* ws = static_cast<char*>(workspace);
  a.hdr = reinterpret_cast<int32_t*>(ws);
  a.row_expert = reinterpret_cast<int32_t*>(ws + 256);
  a.partial = reinterpret_cast<float*>(ws + 256 + align256(size_t(a.rows) * 4));
  const int grid = dense ? (a.blocks * a.strips * a.splits + 7) / 8 * 8 : kFewGrid;
  if (bm == 16) hipLaunchKernelGGL(k_few<1>, dim3(grid), dim3(256), 0, stream, a);
  else if (bm == 32) hipLaunchKernelGGL(k_few<2>, dim3(grid), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(k_few<4>, dim3(grid), dim3(256), 0, stream, a);
  if (a.splits > 1) {
    const int64_t groups = int64_t(a.rows) * (c->Hp / 8);
    hipLaunchKernelGGL(k_few_join, dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, stream, a);
  }
  return hip_status();
}

}  // namespace moonep
