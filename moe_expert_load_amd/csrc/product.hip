// Products of rows with one matrix or with one per expert, and the epilogue
// (epilogue.hpp), in four kernels by the height of their tiles; the time of each
// is modelled on the host (kTiles) and the shortest taken.  The grid covers the
// tiles that a configuration can have; which there are is found on the device from
// cu_seqlens (my_block).  Where the tiles would leave units idle the k
// axis is cut into parts whose sums go to the workspace in fp32; k_join adds them
// in a fixed order and applies the epilogue.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "epilogue.hpp"

#include "host.hpp"
#include "lds.hpp"
#include "overlap.hpp"

namespace moonep {

constexpr int kFewCols = 128;        // columns of a wave
constexpr int kFewStep = 32;         // k of a step
constexpr int kBand = 8;             // row blocks of a band, about
constexpr int kScan = 8;             // segments a lane looks at, without a list

struct RowItem {
  int32_t seg;               // segment, counted from the first listed rank's first
  int32_t first, cnt;        // the segment's first item, and how many there are
};

struct ProductArgs {
  const uint16_t* x;
  const uint16_t* w_home;
  const uint16_t* w_pref;
  const int32_t* cu;         // null: one matrix
  float* partial;            // [splits][rows][N]
  int32_t* nblocks;          // grouped: how many of `list` there are
  int32_t* row_expert;       // [rows], grouped
  RowItem* list;             // grouped, over more than 64 kScan segments
  int32_t H, E, B, SK, first_rank, nranks;
  int32_t rows, height, cols, strips, steps, splits;
  int32_t blocks;            // grouped: the most there may be
  int32_t once;              // about one block for each segment, all weights too many to be kept
  Epilogue ep;
};

// The listed ranks' segments as blocks of at most a.height rows, in layout order.
__global__ __launch_bounds__(1024) void k_row_blocks(ProductArgs a) {
  __shared__ int s_part[17];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int per = a.E + a.B, total = a.nranks * per;
  int carry = 0;
  for (int c0 = 0; c0 < total; c0 += 1024) {
    const int i = c0 + tid;
    int len = 0;
    if (i < total) {
      const int32_t* cu = a.cu + int64_t(a.first_rank + i / per) * (per + 1) + i % per;
      len = cu[1] - cu[0];
    }
    const int n = (len + a.height - 1) / a.height;
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
    for (int m = 0; m < n && at + m < a.blocks; ++m)
      a.list[at + m] = RowItem{i, at, n};
    __syncthreads();
  }
  if (tid == 0) *a.nblocks = min(carry, a.blocks);
}

struct RowBlock {
  int r, j, row0, rows;                       // rank, weight row, first row (absolute), rows
  int n0, split;                              // first column, part of the k axis
};

// What this workgroup multiplies; false: nothing.  Neighbouring items go to one
// XCD: the row blocks of a band of a segment under one strip of columns, then the
// next strip, so that what an XCD's units work on at a time is about square and
// its L2 reads the fewest rows and columns for it.  A segment is cut into bands of
// 6 to 11 blocks, all of one size but the last, which has what is left: one block
// at least (65,536 rows of 7,168 onto 2,048: bands of 4, 8, 16 and 32 blocks take
// 1.70, 1.69, 1.73 and 1.95 ms; over 48 experts of 11 blocks each, bands of 8 that
// straddle them 1.95 ms, of 11 1.89).  Bands that differ by one block at most, in
// place of a short last one, change nothing: segments of 33 to 257 blocks with a
// last band of 1 to 6, both ways round of 7,168 x 2,048, within 1 % on either side.
//
// Where the segments are few every wave counts their blocks itself, kScan
// segments a lane: 1 us, where the list of k_row_blocks costs 4 and a launch.
__device__ __forceinline__ bool my_block(const ProductArgs& a, RowBlock& b) {
  const int lane = lane_id(), per = a.E + a.B, total = a.nranks * per;
  const bool scan = a.cu && !a.list;
  int start[kScan], n[kScan], blocks = a.blocks;
  if (scan) {
    blocks = 0;
#pragma unroll
    for (int q = 0; q < kScan; ++q) {
      const int i = q * kWave + lane;
      n[q] = 0;
      if (i < total) {
        const int32_t* cu = a.cu + int64_t(a.first_rank + i / per) * (per + 1) + i % per;
        n[q] = (cu[1] - cu[0] + a.height - 1) / a.height;
      }
    }
#pragma unroll
    for (int q = 0; q < kScan; ++q) {
      const int incl = wave_incl_scan(n[q]);
      start[q] = blocks + incl - n[q];
      blocks += wave_bcast(incl, kWave - 1);
    }
  } else if (a.cu) {
    blocks = *a.nblocks;
  }
  const int units = blocks * a.strips, items = units * a.splits, share = (items + 7) / 8;
  const int place = blockIdx.x / 8, item = (blockIdx.x % 8) * share + place;
  if (place >= share || item >= items) return false;
  b.split = item / units;
  int u = item % units;
  // few rows of many experts: strip by strip over the experts, not expert by expert
  if (a.once) u = u % blocks * a.strips + u / blocks;
  const int near = u / a.strips;                           // a block of the same segment
  int first = 0, cnt = blocks, seg = 0;
  if (scan) {
#pragma unroll
    for (int q = 0; q < kScan; ++q) {
      const uint64_t hit = __ballot(near >= start[q] && near < start[q] + n[q]);
      if (hit) {
        const int src = __ffsll((unsigned long long)hit) - 1;
        first = wave_bcast(start[q], src);
        cnt = wave_bcast(n[q], src);
        seg = q * kWave + src;
      }
    }
  } else if (a.cu) {
    first = __builtin_amdgcn_readfirstlane(a.list[near].first);
    cnt = __builtin_amdgcn_readfirstlane(a.list[near].cnt);
    seg = __builtin_amdgcn_readfirstlane(a.list[near].seg);
  }
  const int bands = max(1, (2 * cnt + kBand) / (2 * kBand));
  const int size = (cnt + bands - 1) / bands, in = u - first * a.strips;
  const int band = in / (size * a.strips), at = in % (size * a.strips);
  const int high = min(size, cnt - band * size), m = (band * size + at % high) * a.height;
  b.n0 = (at / high) * a.cols;
  if (a.cu) {
    b.r = a.first_rank + seg / per;
    b.j = seg % per;
    const int32_t* cu = a.cu + int64_t(b.r) * (per + 1) + b.j;
    const int lo = cu[0], len = cu[1] - lo;
    b.row0 = b.r * a.SK + lo + m;
    b.rows = min(a.height, len - m);
  } else {
    b.r = b.j = 0;
    b.row0 = m;
    b.rows = min(a.height, a.rows - m);
  }
  return true;
}

// Weights of the block's segment, and its share of the steps.
__device__ __forceinline__ const uint16_t* weights_of(const ProductArgs& a, const RowBlock& b) {
  const int64_t size = int64_t(a.H) * a.ep.N;
  return b.j < a.E ? a.w_home + b.j * size : a.w_pref + (int64_t(b.r) * a.B + (b.j - a.E)) * size;
}
__device__ __forceinline__ int first_step(const ProductArgs& a, int split) {
  return int(int64_t(split) * a.steps / a.splits);
}

// A lane's eight columns of one row: to the workspace, or through the epilogue.
template <bool SPLIT>
__device__ __forceinline__ void give8(const ProductArgs& a, const RowBlock& rb, const DropKey& key,
                                      float (&z)[8], const float (&bias)[8], int m, int n) {
  const int64_t row = int64_t(rb.row0) + m;
  if constexpr (SPLIT) {
    const int64_t at = row - int64_t(a.first_rank) * a.SK;
    store8(a.partial + (int64_t(rb.split) * a.rows + at) * a.ep.N + n, z);
    if (a.cu && n == 0 && rb.split == 0)
      a.row_expert[at] = expert_of(a.ep, rb.r, rb.j, a.E, a.B);
  } else {
    epilogue8(a.ep, key, z, bias, row, n);
  }
}

// ---------------------------------------------------------------------------
// Few rows: the single tokens of decoding, one matrix or an expert each.  The time
// is that of reading the weights once, so they go from memory to registers and
// nowhere else.
// A wave takes 128 columns and steps of 32 k.  Lane l loads rows k0 + 8 (l / 16) +
// 0 .. 7 of columns n0 + 8 (l % 16) + 0 .. 7, eight 16-byte loads of which every 16
// lanes cover 256 contiguous bytes.  A matrix instruction wants eight consecutive
// k of one column per lane; a lane has an 8 x 8 block, whose transposition is 32
// byte permutes (pairs of rows; larger strides only rename registers).
// Instruction i then multiplies columns n0 + 8 (l % 16) + i, and a lane ends with
// eight consecutive columns of a row: one group of the epilogue.  The four waves
// of a workgroup share its steps and are joined in LDS.
// ---------------------------------------------------------------------------

// Columns 2j and 2j + 1 of an 8 x 8 block as eight consecutive k each.
__device__ __forceinline__ void column_pair(const u32x4 (&w)[8], int j, bf16x8& even,
                                            bf16x8& odd) {
  u32x4 e, o;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    e[q] = __builtin_amdgcn_perm(w[2 * q + 1][j], w[2 * q][j], 0x05040100u);
    o[q] = __builtin_amdgcn_perm(w[2 * q + 1][j], w[2 * q][j], 0x07060302u);
  }
  even = __builtin_bit_cast(bf16x8, e);
  odd = __builtin_bit_cast(bf16x8, o);
}

// RB: blocks of 16 rows that a workgroup takes.  ONCE: where the experts' weights
// are too many for the last cache, and read by about one block each, they pass it
// by, and strips are taken over the experts in turn (my_block).  One token on each
// of 8 ranks, 41 experts of 7,168 x 2,048 met: 224 us through the caches expert by
// expert, 209 strip by strip, 201 past them, 189 both (6.3 TB/s).  Not so where
// blocks share weights (568 rows over 60 experts of 880 x 6,576: 116, 154, 133, 171)
// or where the last cache holds them from call to call (64 experts of 1,024 x 512:
// 10, 10, 13, 12).  All experts' weights count, not only those that a call meets: a
// later call meets others, or comes after other layers.  One token on 8 of 384
// experts of 1,024 x 512 (8 MB of 403) after other work 16 us (through the caches
// 17), with other experts from call to call 12 (13.6), with the same ones 8 to 12 (8);
// on 8 of 24 of 2,648 x 2,160 (92 MB of 275) 28 (42), 25 (22), 25 (20).
template <int RB, bool SPLIT, bool ONCE>
__global__ __launch_bounds__(256, 2) void k_few(ProductArgs a) {
  __shared__ f32x4 s_sum[4 * 3 * RB * kWave * 2];
  RowBlock rb;
  if (!my_block(a, rb)) return;
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int H = a.H, N = a.ep.N, rows = rb.rows;
  const int n = rb.n0 + 8 * (lane & 15);
  const char* w = reinterpret_cast<const char*>(weights_of(a, rb));
  const char* x = reinterpret_cast<const char*>(a.x + int64_t(rb.row0) * H);
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

  const int t0 = first_step(a, rb.split), t1 = first_step(a, rb.split + 1);
  auto load = [&](int t, u32x4 (&wr)[8], u32x4 (&xr)[RB]) {
    const int k = t * kFewStep + 8 * (lane >> 4);
    const bool in = k < H;
    const uint32_t wk = wcol + 2u * uint32_t(in ? k : 0) * N;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const u32x4* p = reinterpret_cast<const u32x4*>(w + (wk + 2u * uint32_t(q) * N));
      wr[q] = ONCE ? __builtin_nontemporal_load(p) : *p;
    }
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
      bf16x8 even, odd;
      column_pair(wr, jj, even, odd);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const bf16x8 xa = __builtin_bit_cast(bf16x8, xr[b]);
        acc[2 * jj][b] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, even, acc[2 * jj][b], 0, 0, 0);
        acc[2 * jj + 1][b] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, odd, acc[2 * jj + 1][b], 0, 0, 0);
      }
    }
  };
  // three steps ahead, four buffers (one token, 7,168 x 2,048 cold: 14.0 us with one
  // step ahead, 13.3)
  u32x4 wr[4][8], xr[4][RB];
  int t = t0 + wv;
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (t + 4 * u < t1) load(t + 4 * u, wr[u], xr[u]);
#pragma unroll 1
  for (; t < t1; t += 16) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int now = t + 4 * u, ahead = now + 12;
      if (now >= t1) break;
      if (ahead < t1) load(ahead, wr[(u + 3) & 3], xr[(u + 3) & 3]);
      multiply(now, wr[u], xr[u]);
    }
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
  DropKey key{};
  if constexpr (!SPLIT) {
    bias8(a.ep, expert_of(a.ep, rb.r, rb.j, a.E, a.B), a.E, n, bias);
    if (a.ep.cut) key = drop_key(a.ep.rng);
  }
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
    if (m < rows && n < N) give8<SPLIT>(a, rb, key, z, bias, m, n);
  }
}

// ---------------------------------------------------------------------------
// More rows than weights should be read again for, and fewer than fill the chip
// with larger tiles: 128 x 128 tiles, four waves of 64 x 64 (2 x 2 blocks of 32 x
// 32), operands straight into LDS in stages of 64 k, the k axis cut over
// workgroups as above.  Both operands' rows are whole 128- or 256-byte lines: x
// [128 rows][64 k] is read with 16-byte LDS reads (chunk kc of row m at kc ^ (m /
// 2) % 8), the weights [64 k][128 columns] with the transposing read (chunk c of
// row k at c ^ 4 (k % 4)); neither has a bank conflict.  A unit holds eight waves
// with two stages for each four, which together ask LDS for 96 KB a step and four
// waves: LDS sets the pace (more stages for fewer waves, or one ring of stages for
// all eight, are no faster).  With G = 1 they are two workgroups, whose loads and
// epilogues cover each other's products; with G = 2 one, whose groups of four waves
// share the tile's k axis, add their sums in LDS and do half of its epilogue each:
// nearly half the steps' time where there are no more tiles than units (2,048 rows of
// 7,168 onto 384 in 4 parts, in fp32: 29.7 us, 27.3 by two groups, joins included;
// 4,100 rows over 8 experts of 1,000 x 520 with everything in the epilogue: 23.9,
// 20.6; both replayed.  Bare, 188 shapes of up to 256 tiles: 0.91 of the time on
// average, 1.15 at worst; of 257 to 320 tiles 1.31 to 1.50).
// ---------------------------------------------------------------------------
constexpr int kMidTile = 128, kMidStep = 64;
constexpr int kMidHalf = kMidTile * kMidStep * 2;      // bytes of one operand's stage

template <bool SPLIT, int G>
__global__ __launch_bounds__(256 * G, 2) void k_mid(ProductArgs a) {
  constexpr int NST = 2;
  static_assert(2 * kMidHalf * NST >= 4 * 64 * 256, "the epilogue's staging fits the stages");
  __shared__ __attribute__((aligned(1024))) unsigned char s_all[G * NST * 2 * kMidHalf];
  RowBlock rb;
  if (!my_block(a, rb)) return;
  const int lane = lane_id(), w8 = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wv = w8 & 3, grp = w8 >> 2;
  unsigned char* s_st = s_all + grp * NST * 2 * kMidHalf;
  const int wm = wv >> 1, wn = wv & 1;
  const int H = a.H, N = a.ep.N, n0 = rb.n0;

  // Fragment reads: x rows 64 wm + 32 i + lane % 32, chunk 2 s + lane / 32; the
  // weights' pieces as lds_tr wants them (lane / 16 picks k half and column half).
  const int G4 = lane >> 4, li = lane & 15;
  int xo[4], wo[2];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int row = wm * 64 + (lane & 31), kc = 2 * s + (lane >> 5);
    xo[s] = row * 128 + ((kc ^ ((row >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = (4 * (2 * wn + j) + 2 * (G4 & 1) + ((li & 3) >> 1)) ^ (4 * (li >> 2));
    wo[j] = (8 * (G4 >> 1) + (li >> 2)) * 256 + c * 16 + 8 * (li & 1);
  }

  const u32x4 rx = make_rsrc(a.x + int64_t(rb.row0) * H, uint32_t(rb.rows) * H * 2);
  const u32x4 rw = make_rsrc(weights_of(a, rb), uint32_t(H) * N * 2);
  const int from = first_step(a, rb.split), to = first_step(a, rb.split + 1);
  const int turns = (to - from + G - 1) / G;              // of the first group, the other's less one
  const int t0 = from + grp * turns, t1 = min(to, t0 + turns);

  // Load u of this wave: x rows 8 (4 wv + u) + lane / 8, weight rows 4 (4 wv +
  // u) + lane / 16.  Past the rows, or past k in the last step, an offset
  // beyond every tensor: zeros.
  auto issue = [&](int t) {
    unsigned char* st = s_st + (t % NST) * 2 * kMidHalf;
    const bool ragged = (t + 1) * kMidStep > H;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = wv * 4 + u;
      const int row = 8 * p + (lane >> 3), kc = (lane & 7) ^ ((row >> 1) & 7);
      uint32_t vx = 2u * uint32_t(row) * H + kc * 16;
      const int k = 4 * p + G4, c = li ^ (4 * G4);
      uint32_t vw = 2u * (uint32_t(k) * N + n0 + 8 * c);
      if (ragged) {
        if (t * kMidStep + 8 * kc >= H) vx = 0xfffffff0u;
        if (t * kMidStep + k >= H) vw = 0xfffffff0u;
      }
      if (row >= rb.rows) vx = 0xfffffff0u;
      load_lds16(rx, st + p * 1024, vx, uint32_t(t) * kMidStep * 2);
      load_lds16(rw, st + kMidHalf + p * 1024, vw, uint32_t(t) * kMidStep * 2 * N);
    }
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (t0 + s < t1) issue(t0 + s);
#pragma unroll 1
  for (int t = t0; t < t0 + turns; ++t) {
    // this wave's loads of stage t have landed; the barrier makes every wave's
    // visible, and says that all are done with the stage that is filled next
    wait_vm<0>();
    // its own LDS reads of the last step are done too, not only asked for
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + NST - 1 < t1) issue(t + NST - 1);
    if (G > 1 && t >= t1) break;                          // the last turn: no barrier follows
    const unsigned char* xs = s_st + (t % NST) * 2 * kMidHalf;
    const unsigned char* ws = xs + kMidHalf;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 xa[2], wb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        xa[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(xs + xo[s] + i * 4096));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned char* p = ws + wo[j] + s * 16 * 256;
        wb[j] = join(lds_tr(p), lds_tr(p + 4 * 256));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[i], wb[j], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();

  // 32 x 32 accumulators: lane l holds column l % 32, rows 8 (v / 4) + 4 (l /
  // 32) + v % 4.  Staged in the wave's own 16 KB as 64 rows of 256 bytes (the
  // lane halves, 4 rows apart, swap the row's two column blocks: other banks).
  unsigned char* cs = s_all + w8 * 16384;
  const int half = lane >> 5;
  float bias[2] = {0.f, 0.f};
  DropKey key{};
  if constexpr (!SPLIT) {
    const int e = expert_of(a.ep, rb.r, rb.j, a.E, a.B);
#pragma unroll
    for (int j = 0; j < 2; ++j) bias[j] = bias1(a.ep, e, a.E, n0 + wn * 64 + 32 * j + (lane & 31));
    if (a.ep.cut) key = drop_key(a.ep.rng);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        *reinterpret_cast<float*>(cs + (32 * i + 8 * (v >> 2) + 4 * half + (v & 3)) * 256 +
                                  ((j ^ half) * 128) + (lane & 31) * 4) =
            G == 1 || grp == 0 ? acc[i][j][v] + bias[j] : acc[i][j][v];
  if constexpr (G > 1) {
    // the groups' sums added: each takes half of the rows
    __syncthreads();
    cs = s_all + wv * 16384 + grp * 32 * 256;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f32x4* p = reinterpret_cast<f32x4*>(cs + (k * kWave + lane) * 16);
      const f32x4 o = *reinterpret_cast<const f32x4*>(cs + 4 * 16384 + (k * kWave + lane) * 16);
      const f32x4 m = *p;
      *p = f32x4{m[0] + o[0], m[1] + o[1], m[2] + o[2], m[3] + o[3]};
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int n = n0 + wn * 64 + (lane & 7) * 8;
  auto place = [&](int k, int64_t& at) -> float* {
    const int rr = 8 * k + (lane >> 3), m = wm * 64 + grp * 32 + rr;
    if (m >= rb.rows || n >= N) return nullptr;
    at = (int64_t(rb.row0) + m) * N + n;
    const int blk = ((lane & 7) >> 2) ^ ((rr >> 2) & 1);
    return reinterpret_cast<float*>(cs + rr * 256 + blk * 128 + (lane & 3) * 32);
  };
  if constexpr (SPLIT) {
    const int64_t first = int64_t(a.first_rank) * a.SK;
    float* dst = a.partial + (int64_t(rb.split) * a.rows - first) * N;
#pragma unroll
    for (int k = 0; k < 8 / G; ++k) {
      int64_t at = 0;
      const float* p = place(k, at);
      if (!p) continue;
      float z[8];
      load8(p, z);
      store8(dst + at, z);
    }
    if (a.cu && rb.split == 0 && n0 == 0 && wn == 0 && grp == 0 && wm * 64 + lane < rb.rows)
      a.row_expert[rb.row0 - first + wm * 64 + lane] = expert_of(a.ep, rb.r, rb.j, a.E, a.B);
  } else {
    epilogue_block<8 / G>(a.ep, key, place);
  }
}

// ---------------------------------------------------------------------------
// Many rows: 128 x 256 tiles, four waves of 64 x 128 (2 x 4 blocks), two
// workgroups on a unit, so that one's loads and epilogue are covered by the
// other's products.  A tile of this shape asks LDS for 72 KB every 32 k, 0.75 of
// what 128 x 128 tiles ask for the same products.  The matrix pipe is 59 % busy at
// 1.5 GHz (counters, 65,536 rows of 7,168 onto 2,048): power sets the pace, as of
// the library's product.  That case takes 1.69 to 1.75 ms, 1.1 PFLOP/s (the
// library's bare product 1.55 to 1.63); 8,192 rows of 2,048 onto 7,168 223 to 242
// us bare (the library's 200 to 213), 250 to 268 with dropout and residual.  Those
// are launches one after another; the first 40 or so after a pause take 270 to 310
// while the clock settles, and a call among others with new inputs 272 to 281.  The
// weights go through three stages of 32 k (rows of 512 bytes); x, whose rows of 32 k
// would be half lines, in pairs of steps through two buffers: 80 KB a workgroup.
// ---------------------------------------------------------------------------
constexpr int kWideCols = 256, kWideStep = 32;
constexpr int kWidePair = 128 * 64 * 2, kWideW = kWideStep * kWideCols * 2;

template <bool SPLIT>
__global__ __launch_bounds__(256, 2) void k_wide(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char s_x[2 * kWidePair];
  __shared__ __attribute__((aligned(1024))) unsigned char s_w[3 * kWideW];
  RowBlock rb;
  if (!my_block(a, rb)) return;
  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = wv >> 1, wn = wv & 1;
  const int H = a.H, N = a.ep.N, n0 = rb.n0;
  const int G4 = lane >> 4, li = lane & 15;
  int xo[4], wo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int row = wm * 64 + (lane & 31), kc = 2 * s + (lane >> 5);
    xo[s] = row * 128 + ((kc ^ ((row >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = (4 * (4 * wn + j) + 2 * (G4 & 1) + ((li & 3) >> 1)) ^ (4 * (li >> 2));
    wo[j] = (8 * (G4 >> 1) + (li >> 2)) * 512 + c * 16 + 8 * (li & 1);
  }
  const u32x4 rx = make_rsrc(a.x + int64_t(rb.row0) * H, uint32_t(rb.rows) * H * 2);
  const u32x4 rw = make_rsrc(weights_of(a, rb), uint32_t(H) * N * 2);
  // whole pairs of steps: the parts of the k axis are cut at multiples of 64
  const int p0 = first_step(a, rb.split), p1 = first_step(a, rb.split + 1);
  const int t0 = 2 * p0, t1 = min(2 * p1, (H + kWideStep - 1) / kWideStep);

  // Load u of this wave: x rows 8 (4 wv + u) + lane / 8, weight rows 2 (4 wv + u)
  // + lane / 32 of a step.  Past the rows or past k an offset beyond every
  // tensor: zeros.
  uint32_t vx[4], vw[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int p = wv * 4 + u;
    const int row = 8 * p + (lane >> 3), kc = (lane & 7) ^ ((row >> 1) & 7);
    vx[u] = row < rb.rows ? 2u * uint32_t(row) * H + kc * 16 : 0xfffffff0u;
    const int k = 2 * p + (lane >> 5), c = (lane & 31) ^ (4 * (k & 3));
    vw[u] = 2u * (uint32_t(k) * N + n0 + 8 * c);
  }
  auto issue_x = [&](int pair) {
    unsigned char* to = s_x + (pair & 1) * kWidePair + wv * 4096;
    const bool ragged = (pair + 1) * 64 > H;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = 8 * (wv * 4 + u) + (lane >> 3), kc = (lane & 7) ^ ((row >> 1) & 7);
      const uint32_t v = ragged && pair * 64 + 8 * kc >= H ? 0xfffffff0u : vx[u];
      load_lds16(rx, to + u * 1024, v, uint32_t(pair) * 128);
    }
  };
  auto issue_w = [&](int t) {
    unsigned char* to = s_w + (t % 3) * kWideW + wv * 4096;
    const bool ragged = (t + 1) * kWideStep > H;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = 2 * (wv * 4 + u) + (lane >> 5);
      const uint32_t v = ragged && t * kWideStep + k >= H ? 0xfffffff0u : vw[u];
      load_lds16(rw, to + u * 1024, v, uint32_t(t) * kWideStep * 2 * N);
    }
  };
  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // Order of the loads: x0 w0 w1 | w2 x1 | w3 | w4 x2 | w5 ...: at an even step the
  // weights of one more step may be in flight, at an odd one those and a pair of x.
  auto step = [&](int t, auto ODD_) {
    constexpr int ODD = decltype(ODD_)::value;
    if (t + 1 >= t1) wait_vm<0>();
    else if (ODD) wait_vm<8>();
    else wait_vm<4>();
    // every wave's loads are visible and its LDS reads of the last step done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + 2 < t1) {
      issue_w(t + 2);
      if (!ODD) issue_x(t / 2 + 1);
    }
    const unsigned char* xs = s_x + ((t >> 1) & 1) * kWidePair;
    const unsigned char* ws = s_w + (t % 3) * kWideW;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8 xa[2], wb[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        xa[i] = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4*>(xs + xo[2 * ODD + s] + i * 4096));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned char* p = ws + wo[j] + s * 16 * 512;
        wb[j] = join(lds_tr(p), lds_tr(p + 4 * 512));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[i], wb[j], acc[i][j], 0, 0, 0);
    }
  };
  if (t0 < t1) {
    issue_x(t0 / 2);
    issue_w(t0);
    if (t0 + 1 < t1) issue_w(t0 + 1);
  }
#pragma unroll 1
  for (int t = t0; t < t1; t += 2) {
    step(t, std::integral_constant<int, 0>());
    if (t + 1 < t1) step(t + 1, std::integral_constant<int, 1>());
  }
  __syncthreads();

  // Two passes of 32 rows x 128 columns staged in the wave's own 16 KB, rows of
  // 512 bytes (of two neighbouring blocks of 32 columns the lane halves write one
  // each: other banks).
  unsigned char* cs = wv < 2 ? s_x + wv * 16384 : s_w + (wv - 2) * 16384;
  const int half = lane >> 5, n = n0 + wn * 128 + li * 8;
  const int e = expert_of(a.ep, rb.r, rb.j, a.E, a.B);
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  DropKey key{};
  if constexpr (!SPLIT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = bias1(a.ep, e, a.E, n0 + wn * 128 + 32 * j + (lane & 31));
    if (a.ep.cut) key = drop_key(a.ep.rng);
  }
  const int64_t first = int64_t(a.first_rank) * a.SK;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (wm * 64 + 32 * i >= rb.rows) break;                // uniform: no row is left
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        *reinterpret_cast<float*>(cs + (8 * (v >> 2) + 4 * half + (v & 3)) * 512 +
                                  ((j ^ half) * 128) + (lane & 31) * 4) = acc[i][j][v] + bias[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    auto place = [&](int k, int64_t& at) -> float* {
      const int rr = 4 * k + G4, m = wm * 64 + 32 * i + rr;
      if (m >= rb.rows || n >= N) return nullptr;
      at = (int64_t(rb.row0) + m) * N + n;
      const int blk = (li >> 2) ^ ((rr >> 2) & 1);
      return reinterpret_cast<float*>(cs + rr * 512 + blk * 128 + (lane & 3) * 32);
    };
    if constexpr (SPLIT) {
      float* to = a.partial + (int64_t(rb.split) * a.rows - first) * N;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        int64_t at = 0;
        const float* p = place(k, at);
        if (!p) continue;
        float z[8];
        load8(p, z);
        store8(to + at, z);
      }
    } else {
      epilogue_block<8>(a.ep, key, place);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  if (SPLIT && a.cu && rb.split == 0 && n0 == 0 && wn == 0 && wm * 64 + lane < rb.rows)
    a.row_expert[rb.row0 - first + wm * 64 + lane] = e;
}

// Sums of the splits in ascending order, and the epilogue.  Workgroups of one
// wave: a token's few outputs are spread over the units (14.6 -> 14.0 us there).
__global__ __launch_bounds__(64) void k_join(ProductArgs a) {
  const int64_t nv = a.ep.N / 8, g = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (g >= nv * a.rows) return;
  const int64_t at = g / nv;
  const int n = int(g % nv) * 8;
  DropKey key{};
  if (a.ep.cut) key = drop_key(a.ep.rng);
  float b[8];
  // grouped: rows behind the rank's last segment (all, of a failed plan) have no
  // sums and stay as they were
  bool live = true;
  if (a.cu) {
    const int64_t r = a.first_rank + at / a.SK, per = a.E + a.B;
    live = at % a.SK < a.cu[r * (per + 1) + per];
  }
  bias8(a.ep, a.cu ? a.row_expert[at] : 0, a.E, n, b);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0.f;
  const float* p = a.partial + at * a.ep.N + n;
  for (int s0 = 0; s0 < a.splits; s0 += 8) {
    float v[8][8];                                  // eight parts in flight
#pragma unroll
    for (int s = 0; s < 8; ++s)
      load8(p + int64_t(min(s0 + s, a.splits - 1)) * a.rows * a.ep.N, v[s]);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < a.splits)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += v[s][i];
  }
  if (live) epilogue8(a.ep, key, z, b, at + int64_t(a.first_rank) * a.SK, n);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// The four kernels: rows and columns of a workgroup's tile, k of a step, the
// waves that share the steps, the workgroups that the chip holds at a time, and
// the terms of a call's time in microseconds: with n steps of a wave,
//   start + rounds * (n * step + round) + halves * (n * half + round)
//     + n * items / at_once * filled + outputs / 2^20 * store
// where `halves` is 1 for a last round of at most half as many workgroups as fit
// (tiles in LDS; the others count it whole), and
//   + join + parts * part + parts * outputs / 2^20 * sums    if k is cut into parts,
//   + list + weights of the segments with rows / 2^20 * weight    for experts.
// Fitted (non-negative least squares of the relative error) to 8,384 timings of
// 416 shapes on one MI355X: one to 16,384 rows (a few to 65,536), widths of 8 to
// 7,168, one to 384 experts; of products with a bias and nothing else, replayed with
// the same inputs, and of 128 x 128 tiles by one group of waves only, also where two
// are launched now.  Against the kernels as they are, 169 other shapes (3,135
// timings): the median error is 3.4, 3.9, 8.3 and 5.1 % in the order of the rows,
// what the model picks is 2.6 % slower than the best of them on average, 61 % at
// worst.  With gelu, dropout, residual and z kept (120 shapes, 2,414 timings) times
// are 10 % longer than modelled, all kernels' alike but for the last one's 6 %, and
// the pick costs 2.7 % on average, 54 % at worst.  Large calls, which power holds
// back, take longer too: 8,192 rows of 2,048 onto 7,168 with dropout and residual 250
// to 281 us, by the model 199; 65,536 of 7,168 onto 2,048 over 48 experts 2.0 to 2.2
// ms, by the model 1.4.
struct Tile {
  int height, cols, step_k, waves, at_once;
  float start, step, half, round, filled, join, part, sums, store, list, weight;
};
constexpr Tile kTiles[4] = {
    {16, kFewCols, kFewStep, 4, 512,
     3.80f, 0.284f, 0.f, 0.678f, 0.491f, 1.77f, 0.070f, 2.64f, 1.09f, 1.11f, 0.027f},
    {32, kFewCols, kFewStep, 4, 512,
     4.19f, 0.335f, 0.f, 0.737f, 0.630f, 1.73f, 0.069f, 2.28f, 0.767f, 1.04f, 0.001f},
    {kMidTile, kMidTile, kMidStep, 1, 512,
     5.06f, 0.738f, 0.620f, 0.f, 0.f, 1.77f, 0.073f, 2.50f, 0.696f, 1.30f, 0.f},
    {kMidTile, kWideCols, kMidStep, 1, 512,
     6.43f, 1.31f, 1.07f, 0.f, 0.f, 1.55f, 0.077f, 2.02f, 0.574f, 1.05f, 0.f},
};
constexpr int kMostSplits = 32;          // parts of the k axis
constexpr int64_t kMostItems = (1 << 24) - 8;  // a launch holds fewer than 2^32 threads
constexpr int64_t kUnits = 256;          // compute units
constexpr int64_t kSplitItems = 512;     // a split call fills the chip about once
constexpr int64_t kCached = 256 << 20;   // bytes that the last cache holds
constexpr int64_t kOnceRows = 4;         // mean rows of a segment that is about one block

// Everything that the host decides about a call, from its configuration alone.
struct ProductPlan {
  int64_t rows;
  int tile, blocks, strips, steps, splits;
  bool once;      // the experts' weights are too many to be kept, and are read by one block each
};

static ProductPlan product_plan(const moe_cfg* c, bool dense, int64_t nranks) {
  ProductPlan best{};
  best.rows = nranks * c->S * c->K;
  // segments that may have rows: each costs a block that is not full
  const int64_t live = dense ? 0 : std::min(nranks * (c->E + c->B), best.rows);
  const float out = float(best.rows) * c->Hp / (1 << 20);
  const float weights = float(live) * c->H * c->Hp / (1 << 20);
  float least = INFINITY;
  for (int k = 0; k < 4; ++k) {
    const Tile& t = kTiles[k];
    const int64_t blocks = (best.rows + t.height - 1) / t.height + live;
    const int64_t strips = (c->Hp + t.cols - 1) / t.cols, steps = (c->H + t.step_k - 1) / t.step_k;
    if (blocks * strips >= kMostItems) continue;
    for (int p = 1; p <= kMostSplits; p += p < 4 ? 1 : p < 8 ? 2 : p < 16 ? 4 : 8) {
      if (p > 1 && (p > steps || blocks * strips * p > kSplitItems * t.waves)) break;
      const int64_t items = blocks * strips * p, n = ((steps + p - 1) / p + t.waves - 1) / t.waves;
      const int64_t rest = items % t.at_once;
      const bool half = t.waves == 1 && rest > 0 && rest <= t.at_once / 2;
      const int64_t rounds = items / t.at_once + (rest > 0 && !half);
      float time = t.start + rounds * (n * t.step + t.round) + (half ? n * t.half + t.round : 0.f);
      time += t.filled * n * items / t.at_once + t.store * out;
      if (p > 1) time += t.join + p * (t.part + t.sums * out);
      if (!dense) time += t.list + t.weight * weights;
      if (time < least) {
        least = time;
        best.tile = k; best.blocks = int(blocks); best.strips = int(strips);
        best.steps = int(steps); best.splits = p;
      }
    }
  }
  best.once = best.tile < 2 && !dense && int64_t(c->E) * c->H * c->Hp * 2 > kCached &&
              best.rows <= kOnceRows * live;
  return best;
}

// Workspace of any ranks of a configuration: the number of blocks, their list,
// the rows' experts and the sums, each the most that a plan can want.
static int64_t most_blocks(const moe_cfg* c) {
  const int64_t rows = int64_t(c->R) * c->S * c->K;
  return (rows + 15) / 16 + std::min(int64_t(c->R) * (c->E + c->B), rows);
}
static size_t expert_at(const moe_cfg* c) {
  return 256 + align256(size_t(most_blocks(c)) * sizeof(RowItem));
}
static size_t sums_at(const moe_cfg* c) {
  return expert_at(c) + align256(size_t(c->R) * c->S * c->K * 4);
}
size_t product_ws_bytes(const moe_cfg* c) {
  const int64_t each = int64_t(c->R) * c->S * c->K * c->Hp * kMostSplits;
  return sums_at(c) + size_t(std::min(each, kSplitItems * kMidTile * kWideCols)) * 4;
}

// One workspace for the product with an epilogue and for the epilogue's backward.
static size_t epilogue_ws_bytes(const moe_cfg* c) {
  return std::max(product_ws_bytes(c), epilogue_bwd_ws_bytes(c));
}

template <bool SPLIT>
static void run_product(const ProductArgs& a, int tile, bool once, hipStream_t stream) {
  const int64_t items = int64_t(a.blocks) * a.strips * a.splits;
  const dim3 grid((unsigned)((items + 7) / 8 * 8)), block(256);
  if (tile == 0 && once) hipLaunchKernelGGL((k_few<1, SPLIT, true>), grid, block, 0, stream, a);
  else if (tile == 0) hipLaunchKernelGGL((k_few<1, SPLIT, false>), grid, block, 0, stream, a);
  else if (tile == 1 && once) hipLaunchKernelGGL((k_few<2, SPLIT, true>), grid, block, 0, stream, a);
  else if (tile == 1) hipLaunchKernelGGL((k_few<2, SPLIT, false>), grid, block, 0, stream, a);
  else if (tile == 2 && items <= kUnits)
    hipLaunchKernelGGL((k_mid<SPLIT, 2>), grid, dim3(512), 0, stream, a);
  else if (tile == 2) hipLaunchKernelGGL((k_mid<SPLIT, 1>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_wide<SPLIT>), grid, block, 0, stream, a);
}

}  // namespace moonep

using namespace moonep;

extern "C" int moe_epilogue_workspace_size(const moe_cfg* cfg, const moe_epilogue_cfg* ec,
                                           size_t* bytes_out) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  if (!valid_epilogue(ec) || !bytes_out) return MOE_EINVAL;
  *bytes_out = epilogue_ws_bytes(cfg);
  return MOE_OK;
}

extern "C" int moe_grouped_gemm_epilogue(const moe_cfg* cfg, const moe_epilogue_cfg* ec,
                                         const moe_plan* plan, const moe_bf16* xperm,
                                         const moe_bf16* w_home, const moe_bf16* w_pref,
                                         const float* bias, const void* residual,
                                         const int64_t* rng, void* y, moe_bf16* pre,
                                         int32_t rank_begin, int32_t rank_end, void* workspace,
                                         hipStream_t stream) {
  const int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  if (!valid_epilogue(ec)) return MOE_EINVAL;
  if (rank_begin < 0 || rank_end > cfg->R || rank_begin > rank_end) return MOE_EINVAL;
  if (!plan && !one_matrix(cfg)) return MOE_EINVAL;
  if (rank_begin == rank_end || cfg->S == 0) return MOE_OK;
  ProductArgs a{};
  Epilogue& ep = a.ep;
  drop_params(ec->p, &ep.cut, &ep.scale);
  const bool slots = plan && cfg->B > 0;
  if (!xperm || !w_home || !y || !workspace || !rng_ok(rng, ep.cut)) return MOE_EINVAL;
  if (plan && !plan->cu_seqlens) return MOE_EINVAL;
  if (slots && (!w_pref || !plan->slot_expert)) return MOE_EINVAL;
  if (!aligned16(xperm, w_home, slots ? w_pref : nullptr, bias, residual, y, pre, workspace))
    return MOE_EINVAL;
  // the listed ranks' parts of every tensor
  const int64_t SK = int64_t(cfg->S) * cfg->K, first = rank_begin * SK;
  const int64_t nr = rank_end - rank_begin, rows = nr * SK, segs = cfg->E + cfg->B;
  const int64_t out = cfg->Hp * (ec->f32 ? 4 : 2), w = int64_t(cfg->H) * cfg->Hp * 2;
  const int64_t ws = (int64_t)epilogue_ws_bytes(cfg);
  const char* yb = static_cast<const char*>(y) + first * out;
  const char* rb = residual ? static_cast<const char*>(residual) + first * out : nullptr;
  const moe_bf16* pb = pre ? pre + first * cfg->Hp : nullptr;
  if (clash({{yb, rows * out}, {pb, rows * cfg->Hp * 2}, {workspace, ws}},
            {{xperm + first * cfg->H, rows * cfg->H * 2},
             {w_home, cfg->E * w},
             {slots ? w_pref + int64_t(rank_begin) * cfg->B * (w / 2) : nullptr, nr * cfg->B * w},
             {plan ? plan->cu_seqlens + rank_begin * (segs + 1) : nullptr, nr * (segs + 1) * 4},
             {slots ? plan->slot_expert : nullptr, int64_t(cfg->R) * cfg->B * 4},
             {bias, int64_t(cfg->E) * cfg->Hp * 4},
             {rb == yb ? nullptr : rb, rows * out},
             {ep.cut ? rng : nullptr, 16}}) ||
      clash({{pb, rows * cfg->Hp * 2}, {workspace, ws}}, {{rb, rows * out}}))
    return MOE_EINVAL;
  const ProductPlan p = product_plan(cfg, !plan, nr);
  if (p.splits == 0) return MOE_ELIMIT;
  ep.bias = bias; ep.residual = residual; ep.rng = ep.cut ? rng : nullptr; ep.y = y; ep.pre = pre;
  ep.slot_expert = slots ? plan->slot_expert : nullptr;
  ep.act = ec->act; ep.f32 = ec->f32; ep.N = cfg->Hp;
  a.x = xperm; a.w_home = w_home; a.w_pref = w_pref; a.cu = plan ? plan->cu_seqlens : nullptr;
  a.H = cfg->H; a.E = cfg->E; a.B = cfg->B; a.SK = (int32_t)SK;
  a.first_rank = rank_begin; a.nranks = (int32_t)nr; a.rows = (int32_t)p.rows;
  a.height = kTiles[p.tile].height; a.cols = kTiles[p.tile].cols;
  a.once = p.once; a.blocks = p.blocks; a.strips = p.strips; a.steps = p.steps; a.splits = p.splits;
  char* at = static_cast<char*>(workspace);
  a.nblocks = reinterpret_cast<int32_t*>(at);
  const bool list = plan && nr * segs > kWave * kScan;
  a.list = list ? reinterpret_cast<RowItem*>(at + 256) : nullptr;
  a.row_expert = reinterpret_cast<int32_t*>(at + expert_at(cfg));
  a.partial = reinterpret_cast<float*>(at + sums_at(cfg));
  if (list) hipLaunchKernelGGL(k_row_blocks, dim3(1), dim3(1024), 0, stream, a);
  if (p.splits == 1) {
    run_product<false>(a, p.tile, p.once, stream);
  } else {
    run_product<true>(a, p.tile, p.once, stream);
    const int64_t groups = p.rows * (cfg->Hp / 8);
    hipLaunchKernelGGL(k_join, dim3((unsigned)((groups + 63) / 64)), dim3(64), 0, stream, a);
  }
  return hip_status();
}
