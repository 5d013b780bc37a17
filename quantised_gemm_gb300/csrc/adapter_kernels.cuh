// adapter_kernels.cuh -- low-rank adapters of many requests beside a shared
// projection: row i has adapter a(i) of a bank (A_a [r, K], B_a [N, r], s_a) or none.
//   forward    h_i = A_a x_i,  y_i = base_i + B_a (s_a h_i)
//   backward   dh_i = s_a B_a^T dy_i,  dx_i = base_i + A_a^T dh_i
//              dA_a = sum over a's rows of dh_i x_i^T,  dB_a = sum of s_a dy_i h_i^T
//
// With a rank of at most 128 every one of these is bound by reading or writing
// the long side (x, dy, base, y) once, so there is no tile of it in shared
// memory: the tensor cores take their fragments from registers as they were
// loaded, 16 bytes a lane.  The order of a contraction is free, so a lane's
// eight consecutive values are the k index of two products, and the order of
// the columns of a product is free, so a lane's results are eight consecutive
// columns.  Where a product contracts over the axis that is not contiguous in
// memory, movmatrix turns the 8 x 8 tiles in registers.  mma.sync instead of
// tcgen05: the operands need no trip through shared memory and the accumulators
// none through tensor memory, and with K = 16 to 128 a product is finished
// before a tcgen05 pipeline would have started.
// h and dh are fp32; where they are an operand they go in as two bf16 numbers,
// hi + lo, which keeps 16 bits of them (the lost part, 2^-17, is below the
// rounding of y, 2^-8); x, dy, A and B are bf16 as they are.  Sums are fp32.
#pragma once

#include <cstdint>

#include "internal.h"
#include "rows.cuh"

namespace fp8lin {

// Fragments: lane = 4 * g + t.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Lane (g, t) gives row g, columns 2t and 2t + 1 of an 8 x 8 tile and gets rows
// 2t and 2t + 1 of column g.
__device__ __forceinline__ uint32_t turn_tile(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// x and y as bf16 pairs hi + lo.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = cvt_bf16x2(x, y);
  float rx = x - bf16lo_to_f32(hi), ry = y - bf16hi_to_f32(hi);
  if (!(fabsf(rx) <= fabsf(x))) rx = 0.0f;  // an infinity is all in hi
  if (!(fabsf(ry) <= fabsf(y))) ry = 0.0f;
  lo = cvt_bf16x2(rx, ry);
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// ---------------------------------------------------------------- rows by adapter

// A route: first[count + 2], then rows[]: the row numbers of adapter 0 in
// order, of adapter 1, ..., and those without one; adapter g's begin at
// first[g], and first[count + 1] is the number of rows.
struct Route {
  const int32_t* first;
  const int32_t* rows;
  int groups;  // count + 1: the last one is the rows without an adapter
};

struct RowTile {
  int group;  // -1: no such tile
  int begin;  // in rows[]
  int count;
  int slot;   // index among the tiles of groups with several
  int block;  // index of its first 16 rows among the blocks of 16 of all groups
  bool only;  // the group's only tile
};

// Tile `want` of tiles of `size` rows of one group each (a group without rows
// has none).  All lanes of a warp call it and get the same.
__device__ __forceinline__ RowTile find_tile(const Route& r, int groups, int size, int want) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int before = 0, several_before = 0, blocks_before = 0;
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    int begin = 0, count = 0;
    if (g < groups) {
      begin = __ldg(r.first + g);
      count = __ldg(r.first + g + 1) - begin;
    }
    const int tiles = (count + size - 1) / size, several = tiles > 1 ? tiles : 0;
    const int blocks = (count + 15) / 16;
    int up = tiles, several_up = several, blocks_up = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, up, o);
      const int b = __shfl_up_sync(0xFFFFFFFFu, several_up, o);
      const int c = __shfl_up_sync(0xFFFFFFFFu, blocks_up, o);
      if (lane >= o) {
        up += a;
        several_up += b;
        blocks_up += c;
      }
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, before + up > want);
    if (hit != 0) {
      const int at = __ffs(static_cast<int>(hit)) - 1;
      const int inside = want - before - __shfl_sync(0xFFFFFFFFu, up - tiles, at);
      RowTile t;
      t.group = base + at;
      t.only = __shfl_sync(0xFFFFFFFFu, tiles, at) == 1;
      t.slot = several_before + __shfl_sync(0xFFFFFFFFu, several_up - several, at) + inside;
      t.block = blocks_before + __shfl_sync(0xFFFFFFFFu, blocks_up - blocks, at) + inside * (size / 16);
      t.begin = __shfl_sync(0xFFFFFFFFu, begin, at) + inside * size;
      t.count = min(size, __shfl_sync(0xFFFFFFFFu, count, at) - inside * size);
      return t;
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
    several_before += __shfl_sync(0xFFFFFFFFu, several_up, 31);
    blocks_before += __shfl_sync(0xFFFFFFFFu, blocks_up, 31);
  }
  return RowTile{-1, 0, 0, 0, 0, false};
}

// ---------------------------------------------------------------- low = x W^T

// low[i][j] = scale_a * sum_c x[i][c] w_a[j][c] for the rows i of one tile, 16 *
// kTiles of them for each of kRowWarps warps.  kAlong: w_a is [r, cols] (A:
// contiguous along the contraction); else [cols, r] (B).  The other warps, and the
// CTAs of a cluster, take other columns, 32 each in turn; their sums meet in
// shared memory.  Warps of the same columns read w_a from L1 after the first.
struct LowArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;
  const float* scale;  // null: 1
  float* low;          // [rows, rank] dense
  int cols, rank;
  int parts;  // CTAs of a cluster
  Route route;
};

constexpr int kLowWarps = 8;

// Ranks a lane holds side by side of a [cols, r] weight.
constexpr int ranks_a_lane(int rank_tiles) { return rank_tiles >= 4 ? 8 : 2 * rank_tiles; }

template <int kTiles, int kRankTiles, int kRowWarps, bool kAlong, bool kAligned>
__global__ void __launch_bounds__(32 * kLowWarps, kRankTiles <= 8 ? 2 : 1)
    adapter_low_kernel(const __grid_constant__ LowArgs p) {
  constexpr int kColWarps = kLowWarps / kRowWarps, kSums = kTiles * kRankTiles * 4;
  constexpr int kRoom = kColWarps > 1 ? kLowWarps / 2 : kLowWarps;
  __shared__ float sums[kRoom][kSums][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int row_warp = warp % kRowWarps, col_warp = warp / kRowWarps;
  const int g = lane >> 2, t = lane & 3;
  const int parts = p.parts, part = static_cast<int>(blockIdx.x) % parts;
  const RowTile tile = find_tile(p.route, p.route.groups, 16 * kTiles * kRowWarps,
                                 static_cast<int>(blockIdx.x) / parts);
  if (tile.group < 0) return;  // all CTAs of the cluster
  if (tile.group == p.route.groups - 1) {  // rows without an adapter
    if (part == 0)
      for (int at = warp; at < tile.count; at += kLowWarps)
        for (int j = lane; j < p.rank; j += 32)
          p.low[int64_t(__ldg(p.route.rows + tile.begin + at)) * p.rank + j] = 0.0f;
    return;
  }
  int64_t row[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (row_warp * kTiles + m) * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
    }
  const bool idle = row_warp * kTiles * 16 >= tile.count;
  const uint16_t* const w = p.w + int64_t(tile.group) * p.rank * p.cols;
  float acc[kTiles][kRankTiles][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  constexpr int kWide = ranks_a_lane(kRankTiles);
  const int step = 32 * kColWarps * parts;
  // A lane's x and w of 32 columns.  w along the contraction: rank 8 j + g, the
  // lane's eight columns; across it: row k of a product's tile is column
  // 8 (k / 2) + 4 s + k % 2 of the 32, and two more in its second half (the order
  // in which a lane holds x), and a lane has kWide ranks of it.
  constexpr int kBlocks = (kRankTiles + 3) / 4;
  constexpr int kLoads = kAlong ? kRankTiles : 4 * kBlocks;
  auto load_x = [&](int c, uint4 (&x)[kTiles][2]) {
    const int col = c + 8 * t;
    const int n = kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[m][i] = load_values<kAligned>(p.x + row[m][i] * p.ldx + col, row[m][i] >= 0 ? n : 0);
  };
  auto load_w = [&](int c, uint4 (&b)[kLoads]) {
    if constexpr (kAlong) {
      const int col = c + 8 * t;
      const int n = kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) {
        const int rank = 8 * j + g;
        b[j] = load_values<kAligned>(w + int64_t(rank) * p.cols + col, rank < p.rank ? n : 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {  // block, step, half
        const int col = c + 8 * (g >> 1) + 2 * (i & 3) + (g & 1);
        const int rank = 32 * (i >> 2) + kWide * t;
        const bool on = col < p.cols && rank < p.rank;
        const uint16_t* from = w + int64_t(col) * p.rank + rank;
        if constexpr (!kAligned) {
          b[i] = load_values<false>(from, on ? min(kWide, p.rank - rank) : 0);
        } else if constexpr (kWide == 8) {
          b[i] = load_if(from, on);
        } else if constexpr (kWide == 4) {
          const uint2 v = load2_if(from, on);
          b[i] = make_uint4(v.x, v.y, 0, 0);
        } else {
          b[i] = make_uint4(load1_if(from, on), 0, 0, 0);
        }
      }
    }
  };
  auto add = [&](const uint4 (&x)[kTiles][2], const uint4 (&b)[kLoads]) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) {
        uint32_t b0, b1;
        if constexpr (kAlong) {
          b0 = word(b[j], 2 * s);
          b1 = word(b[j], 2 * s + 1);
        } else {
          b0 = turn_tile(word(b[4 * (j >> 2) + 2 * s], j & 3));
          b1 = turn_tile(word(b[4 * (j >> 2) + 2 * s + 1], j & 3));
        }
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
          mma_bf16(acc[m][j], word(x[m][0], 2 * s), word(x[m][1], 2 * s), word(x[m][0], 2 * s + 1),
                   word(x[m][1], 2 * s + 1), b0, b1);
      }
  };
  // kAhead turns of x (and of w, where it is small) are on their way: 2 KB a turn
  // of a warp, 16 warps an SM, and HBM takes a microsecond.
  constexpr bool kRingW = kRankTiles <= 4;
  constexpr int kAhead = kRankTiles <= 2 ? 3 : 2;
  int c = idle ? p.cols : 32 * (part * kColWarps + col_warp);
  uint4 x[kAhead][kTiles][2], b[kRingW ? kAhead : 1][kLoads];
#pragma unroll
  for (int d = 0; d < kAhead; ++d) {
    load_x(c + d * step, x[d]);
    if constexpr (kRingW) load_w(c + d * step, b[d]);
  }
  while (c < p.cols) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      if (c < p.cols) {
        if constexpr (!kRingW) load_w(c, b[0]);
        add(x[d], b[kRingW ? d : 0]);
        load_x(c + kAhead * step, x[d]);
        if constexpr (kRingW) load_w(c + kAhead * step, b[d]);
        c += step;
      }
    }
  }
  float* const mine = &acc[0][0][0];
  // Sums of the warps of the same rows: the upper half's to shared memory, added
  // by the lower.
#pragma unroll
  for (int half = kLowWarps / 2; half >= kRowWarps; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) sums[warp - half][i][lane] = mine[i];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) mine[i] += sums[warp][i][lane];
    }
    __syncthreads();
  }
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
  auto rank_of = [&](int j, int i, int t) {
    return kAlong ? 8 * j + 2 * t + (i & 1) : 32 * (j >> 2) + kWide * t + 2 * (j & 3) + (i & 1);
  };
  if (parts == 1) {
    if (warp >= kRowWarps) return;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t to = row[m][i >> 1];
          const int rank = rank_of(j, i, t);
          if (to >= 0 && rank < p.rank) p.low[to * p.rank + rank] = scale * acc[m][j][i];
        }
    return;
  }
  // The cluster's sums: every CTA adds a part of the numbers, in the CTAs' order.
  if (warp < kRowWarps) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) sums[warp][i][lane] = mine[i];
  }
  cluster_sync_all();
  const int each = kRowWarps * kSums / parts;  // numbers of a lane; parts divides kRowWarps * kSums
  for (int k = part * each + warp; k < (part + 1) * each; k += kLowWarps) {
    const int of = k / kSums, m = k % kSums / (4 * kRankTiles), j = k / 4 % kRankTiles, i = k % 4;
    const uint32_t at = smem_addr(&sums[of][k % kSums][lane]);
    float sum = 0.0f;
#pragma unroll 8
    for (int from = 0; from < parts; ++from) sum += __uint_as_float(ld_shared_cluster_u32(map_to_cta(at, from)));
    const int which = (of * kTiles + m) * 16 + 8 * (i >> 1) + g, rank = rank_of(j, i, t);
    if (which < tile.count && rank < p.rank)
      p.low[int64_t(__ldg(p.route.rows + tile.begin + which)) * p.rank + rank] = scale * sum;
  }
  cluster_sync_all();
}

// ---------------------------------------------------------------- y = base + low W

// The ranks of a lane in step s of a product over ranks: four side by side.
template <int kSteps>
__device__ __forceinline__ int rank_at(int s, int t) {
  return kSteps == 1 ? 4 * t : 32 * (s >> 1) + 8 * t + 4 * (s & 1);
}

// y[i][c] = base[i][c] + sum_j scale_a low[i][j] w_a(j, c) for one tile of rows
// and `slab` columns.  kAlong: w_a is [cols, r] (B), else [r, cols] (A).
struct HighArgs {
  const float* low;
  const uint16_t* w;
  const float* scale;    // null: 1
  const uint16_t* base;  // null: 0
  uint16_t* y;
  int64_t ldbase, ldy;
  int cols, rank, slab;
  Route route;
  bool low_aligned;
};

constexpr int kHighWarps = 8;

// The operand of low: 16 * kTiles rows, hi and lo.
template <int kTiles, int kSteps>
struct LowFragments {
  uint32_t hi[kTiles][kSteps][4], lo[kTiles][kSteps][4];
};

__device__ __forceinline__ float4 load_ranks(const float* from, int n, bool aligned) {
  if (aligned && n >= 4) return *reinterpret_cast<const float4*>(from);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (n > 0) v.x = from[0];
  if (n > 1) v.y = from[1];
  if (n > 2) v.z = from[2];
  if (n > 3) v.w = from[3];
  return v;
}

template <int kTiles, int kSteps, int kRowWarps, bool kAlong, bool kAligned, bool kWAligned>
__global__ void __launch_bounds__(32 * kHighWarps, kSteps <= 4 ? 2 : 1)
    adapter_high_kernel(const __grid_constant__ HighArgs p) {
  constexpr int kColWarps = kHighWarps / kRowWarps;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int row_warp = warp % kRowWarps, col_warp = warp / kRowWarps;
  const int g = lane >> 2, t = lane & 3;
  const RowTile tile =
      find_tile(p.route, p.route.groups, 16 * kTiles * kRowWarps, static_cast<int>(blockIdx.x));
  if (tile.group < 0 || row_warp * kTiles * 16 >= tile.count) return;
  const bool none = tile.group == p.route.groups - 1;
  if (none && p.y == p.base) return;
  const int begin = static_cast<int>(blockIdx.y) * p.slab;
  const int end = min(begin + p.slab, p.cols);
  int64_t row[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (row_warp * kTiles + m) * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
    }
  // The base of a warp's next turns is on its way while it computes.
  auto values = [&](int c) {
    const int col = c + 8 * t;
    return c >= end ? 0 : kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
  };
  constexpr int kAhead = 2, kTurn = 32 * kColWarps;
  uint4 base[kAhead][kTiles][2];
  auto fetch = [&](int c, uint4 (&into)[kTiles][2]) {
    const int n = values(c);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        into[m][i] = load_values<kAligned>(p.base + row[m][i] * p.ldbase + c + 8 * t,
                                           p.base != nullptr && row[m][i] >= 0 ? n : 0);
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(begin + 32 * col_warp + d * kTurn, base[d]);
  LowFragments<kTiles, kSteps> f;
  const float scale = none || p.scale == nullptr ? 1.0f : __ldg(p.scale + tile.group);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int rank = rank_at<kSteps>(s, t);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row[m][i] >= 0 && !none)
          v = load_ranks(p.low + row[m][i] * p.rank + rank, p.rank - rank, p.low_aligned);
        split_pair(v.x * scale, v.y * scale, f.hi[m][s][i], f.lo[m][s][i]);
        split_pair(v.z * scale, v.w * scale, f.hi[m][s][i + 2], f.lo[m][s][i + 2]);
      }
  const uint16_t* const w = none ? nullptr : p.w + int64_t(tile.group) * p.rank * p.cols;
  auto turn = [&](int c, uint4 (&next)[kTiles][2]) {
    const int col = c + 8 * t;
    const int n = values(c);
    uint4 out[kTiles][2];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) out[m][i] = next[m][i];
    fetch(c + kAhead * kTurn, next);
    if (!none) {
      float acc[kTiles][4][4];
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.0f;
      // Column k of product q is column 8 (k / 2) + 2 q + k % 2 of the 32.
#pragma unroll
      for (int block = 0; block < (kSteps + 1) / 2; ++block) {
        uint32_t b[4][4];  // of product q: the two halves of one step or of two
        if constexpr (kAlong) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int from_col = c + 8 * (g >> 1) + 2 * q + (g & 1);
            const int rank = rank_at<kSteps>(2 * block, t);
            constexpr int kWide = kSteps == 1 ? 4 : 8;
            const bool on = from_col < p.cols && rank < p.rank;
            const uint16_t* from = w + int64_t(from_col) * p.rank + rank;
            uint4 v;
            if constexpr (!kWAligned) {
              v = load_values<false>(from, on ? min(kWide, p.rank - rank) : 0);
            } else if constexpr (kWide == 8) {
              v = load_if(from, on);
            } else {
              const uint2 u = load2_if(from, on);
              v = make_uint4(u.x, u.y, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) b[q][i] = word(v, i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < (kSteps == 1 ? 2 : 4); ++i) {
            const int rank = rank_at<kSteps>(2 * block + (i >> 1), g >> 1) + 2 * (i & 1) + (g & 1);
            const uint4 v = load_values<kWAligned>(w + int64_t(rank) * p.cols + col, rank < p.rank ? n : 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q][i] = turn_tile(word(v, q));
          }
        }
#pragma unroll
        for (int s = 2 * block; s < 2 * block + (kSteps == 1 ? 1 : 2); ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t b0 = b[q][2 * (s - 2 * block)], b1 = b[q][2 * (s - 2 * block) + 1];
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
              mma_bf16(acc[m][q], f.lo[m][s][0], f.lo[m][s][1], f.lo[m][s][2], f.lo[m][s][3], b0, b1);
              mma_bf16(acc[m][q], f.hi[m][s][0], f.hi[m][s][1], f.hi[m][s][2], f.hi[m][s][3], b0, b1);
            }
          }
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[8];
          bf16x8_to_f32(out[m][i], v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[2 * q] += acc[m][q][2 * i];
            v[2 * q + 1] += acc[m][q][2 * i + 1];
          }
          out[m][i] = f32_to_bf16x8(v);
        }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        store_values<kAligned, 4>(p.y + (row[m][i] < 0 ? 0 : row[m][i]) * p.ldy + col, out[m][i],
                                  row[m][i] < 0 ? 0 : n);
  };
  for (int c = begin + 32 * col_warp; c < end; c += kAhead * kTurn) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
      if (c + d * kTurn < end) turn(c + d * kTurn, base[d]);
  }
}

// ---------------------------------------------------------------- dW = x^T low

// dw[c][j] = sum over the rows i of one adapter of x[i][c] scale_a low[i][j], for
// a slab of columns c.  The CTA's warps take blocks of 16 rows in turn (kRowWarps
// of them) and columns side by side (the others); a tile of rows that is its
// adapter's only one is written as bf16 into dw, else its sums go to the
// partials, one slot a tile, which adapter_sum_kernel adds up.
struct WeightArgs {
  const uint16_t* x;
  int64_t ldx;
  const float* low;
  const float* scale;  // null: 1
  uint16_t* dw;
  float* partials;  // [slot][cols * rank]
  int cols, rank, tile_rows, tiles, slabs;
  const uint4* packed;  // low as adapter_pack_kernel left it, or null
  bool along;    // dw is [cols, r] (dB), else [r, cols] (dA)
  bool aligned;  // x's rows
  bool dw_aligned;
};

constexpr int kWeightWarps = 8;

// With a small rank the rows' numbers are few beside x, and splitting the rows
// leaves fewer partial sums; with a large one warps of the same rows share them.
template <int kRankTiles>
struct WeightShape {
  static constexpr int kRowWarps = kRankTiles <= 2 ? 4 : kRankTiles == 4 ? 2 : 1;
  static constexpr int kColWarps = kWeightWarps / kRowWarps;
  static constexpr int kChunks = kRankTiles <= 4 ? 2 : 1;  // of 32 columns a warp
  static constexpr int kSlab = 32 * kChunks * kColWarps;
  static constexpr int kSums = 2 * kChunks * kRankTiles * 4;  // a lane's
};

// What a lane needs of rank tile j of 16 rows of low: rows 2 t, 2 t + 1 and 2 t + 8,
// 2 t + 9 of rank 8 j + g, as pairs hi (x, y) and lo (z, w).
__device__ __forceinline__ uint4 low_operand(float a, float b, float c, float d) {
  uint4 v;
  split_pair(a, b, v.x, v.z);
  split_pair(c, d, v.y, v.w);
  return v;
}

// low of one or two calls to adapter_weight_kernel in that form, block by block of
// 16 rows of an adapter: a warp a block.
struct PackArgs {
  const float* low;
  const float* scale;
  uint4* packed;
};
constexpr int kPackWarps = 4;

template <int kRankTiles>
__global__ void __launch_bounds__(32 * kPackWarps)
    adapter_pack_kernel(const PackArgs a, const PackArgs b, const Route route, int rank, int blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int at = static_cast<int>(blockIdx.x) * kPackWarps + static_cast<int>(threadIdx.x >> 5);
  const int g = lane >> 2, t = lane & 3;
  const PackArgs& p = at < blocks ? a : b;
  const RowTile tile = find_tile(route, route.groups - 1, 16, at < blocks ? at : at - blocks);
  if (p.packed == nullptr || tile.group < 0) return;
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
  float v[kRankTiles][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int of = 2 * t + (e & 1) + 8 * (e >> 1);
    const float* from =
        of < tile.count ? p.low + int64_t(__ldg(route.rows + tile.begin + of)) * rank : nullptr;
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
      v[j][e] = from != nullptr && 8 * j + g < rank ? scale * from[8 * j + g] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kRankTiles; ++j)
    p.packed[(int64_t(tile.block) * kRankTiles + j) * 32 + lane] = low_operand(v[j][0], v[j][1], v[j][2], v[j][3]);
}

template <int kRankTiles, bool kAligned>
__device__ __forceinline__ void weight_tile(const WeightArgs& p, const Route& route, int block,
                                            float (*sums)[WeightShape<kRankTiles>::kSums][32]) {
  using S = WeightShape<kRankTiles>;
  constexpr int kChunks = S::kChunks, kSums = S::kSums;
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int col_warp = warp % S::kColWarps, row_warp = warp / S::kColWarps;
  const int g = lane >> 2, t = lane & 3;
  // The last rows first: they are what is left in L2 of the pass before.
  const RowTile tile = find_tile(route, route.groups - 1, p.tile_rows, p.tiles - 1 - block / p.slabs);
  if (tile.group < 0) return;
  const int col0 = ((block % p.slabs) * S::kColWarps + col_warp) * 32 * kChunks;
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
  float acc[2 * kChunks][kRankTiles][4];
#pragma unroll
  for (int m = 0; m < 2 * kChunks; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  const int32_t* const rows = route.rows + tile.begin;
  // x of the next blocks and the row numbers of one more are on their way.
  constexpr int kStep = 16 * S::kRowWarps, kAhead = kRankTiles <= 8 ? 3 : 2;
  int at[2];
  uint4 ring[kAhead][kChunks][2];
  auto find = [&](int r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int of = r + 8 * i + g;
      at[i] = of < tile.count ? __ldg(rows + of) : -1;
    }
  };
  auto fetch = [&](uint4 (&into)[kChunks][2]) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = col0 + 32 * c + 8 * t;
        const int n = at[i] < 0 ? 0 : values_at(col, p.cols);
        into[c][i] = load_values<kAligned>(p.x + at[i] * p.ldx + col, n);
      }
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) {
    find(16 * row_warp + d * kStep);
    fetch(ring[d]);
  }
  find(16 * row_warp + kAhead * kStep);
  auto turn = [&](int r, uint4 (&x)[kChunks][2]) {
    uint4 low[kRankTiles];
    if (p.packed != nullptr) {
      const uint4* from = p.packed + (int64_t(tile.block + r / 16) * kRankTiles) * 32 + lane;
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) low[j] = __ldg(from + 32 * j);
    } else {
      float v[kRankTiles][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int of = r + 2 * t + (e & 1) + 8 * (e >> 1);
        const float* from = of < tile.count ? p.low + int64_t(__ldg(rows + of)) * p.rank : nullptr;
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j)
          v[j][e] = from != nullptr && 8 * j + g < p.rank ? scale * __ldg(from + 8 * j + g) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) low[j] = low_operand(v[j][0], v[j][1], v[j][2], v[j][3]);
    }
    uint32_t a[kChunks][4][2];  // of columns 8 (k / 2) + 2 q + k % 2, rows 0-7 and 8-15
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) a[c][q][i] = turn_tile(word(x[c][i], q));
    fetch(x);
    find(r + (kAhead + 1) * kStep);
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          mma_bf16(acc[2 * c + m][j], a[c][2 * m][0], a[c][2 * m + 1][0], a[c][2 * m][1],
                   a[c][2 * m + 1][1], low[j].z, low[j].w);
          mma_bf16(acc[2 * c + m][j], a[c][2 * m][0], a[c][2 * m + 1][0], a[c][2 * m][1],
                   a[c][2 * m + 1][1], low[j].x, low[j].y);
        }
    }
  };
  for (int r = 16 * row_warp; r < tile.count; r += kAhead * kStep) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
      if (r + d * kStep < tile.count) turn(r + d * kStep, ring[d]);
  }
  if constexpr (S::kRowWarps > 1) {
    float* const mine = &acc[0][0][0];
#pragma unroll
    for (int half = kWeightWarps / 2; half >= S::kColWarps; half >>= 1) {
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) sums[warp - half][i][lane] = mine[i];
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) mine[i] += sums[warp][i][lane];
      }
      __syncthreads();
    }
  }
  if (row_warp != 0 || col0 >= p.cols) return;
  const int64_t size = int64_t(p.cols) * p.rank;
  uint16_t* const dw = p.dw + tile.group * size;
  float* const part = tile.only ? nullptr : p.partials + tile.slot * size;
  // A lane has of product (c, j) columns 8 (g / 2) + 2 q + g % 2, q = 0 .. 3, of
  // ranks 8 j + 2 t and the next.
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j) {
      if (p.along) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = col0 + 32 * c + 8 * (g >> 1) + 2 * q + (g & 1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rank = 8 * j + 2 * t + e;
            if (col >= p.cols || rank >= p.rank) continue;
            const float v = acc[2 * c + (q >> 1)][j][2 * (q & 1) + e];
            const int64_t to = int64_t(col) * p.rank + rank;
            if (part != nullptr)
              part[to] = v;
            else
              dw[to] = static_cast<uint16_t>(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
          }
        }
        continue;
      }
      // Lanes of neighbouring g swap, so that one has eight columns side by side
      // of the first rank and the other of the second.
      float v[8];
      const int e = g & 1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* a = acc[2 * c + (q >> 1)][j] + 2 * (q & 1);
        const float got = __shfl_xor_sync(0xFFFFFFFFu, e ? a[0] : a[1], 4);
        v[2 * q] = e ? got : a[0];
        v[2 * q + 1] = e ? a[1] : got;
      }
      const int col = col0 + 32 * c + 8 * (g >> 1), rank = 8 * j + 2 * t + e;
      const int64_t to = int64_t(rank) * p.cols + col;
      if (rank < p.rank && p.dw_aligned && col < p.cols) {
        if (part != nullptr) {
          float4* put = reinterpret_cast<float4*>(part + to);
          put[0] = make_float4(v[0], v[1], v[2], v[3]);
          put[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          *reinterpret_cast<uint4*>(dw + to) = f32_to_bf16x8(v);
        }
      } else if (rank < p.rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col + i >= p.cols) continue;
          if (part != nullptr)
            part[to + i] = v[i];
          else
            dw[to + i] = static_cast<uint16_t>(cvt_bf16x2(v[i], 0.0f) & 0xFFFFu);
        }
      }
    }
}

// dB (blocks from 0 on) and dA (the others) in one launch; either may have none.
template <int kRankTiles>
__global__ void __launch_bounds__(32 * kWeightWarps, kRankTiles <= 2 ? 2 : 1)
    adapter_weight_kernel(const __grid_constant__ WeightArgs db, const __grid_constant__ WeightArgs da,
                          const Route route) {
  griddep_wait();
  griddep_launch_dependents();
  const int block = static_cast<int>(blockIdx.x), first = db.tiles * db.slabs;
  const bool is_db = block < first;
  using S = WeightShape<kRankTiles>;
  __shared__ float sums[S::kRowWarps > 1 ? kWeightWarps / 2 : 1][S::kSums][32];
  const WeightArgs& p = is_db ? db : da;
  if (p.aligned)
    weight_tile<kRankTiles, true>(p, route, is_db ? block : block - first, sums);
  else
    weight_tile<kRankTiles, false>(p, route, is_db ? block : block - first, sums);
}

// The partials of adapters with several tiles, added in order, and zeros for
// those without rows.  One CTA row an adapter.
struct SumArgs {
  const float* partials;
  uint16_t* dw;
  int64_t size;  // cols * rank
  int tile_rows;
  Route route;
};
constexpr int kSumThreads = 256;

__device__ __forceinline__ void sum_partials(const SumArgs& p, int group, int block, int blocks) {
  // Slots before this adapter's: a sum over the groups before it.
  int mine = 0, before = 0;
  const int lane = static_cast<int>(threadIdx.x & 31u);
  for (int g = lane; g <= group; g += 32) {
    const int count = __ldg(p.route.first + g + 1) - __ldg(p.route.first + g);
    const int tiles = (count + p.tile_rows - 1) / p.tile_rows;
    if (g == group)
      mine = tiles;
    else if (tiles > 1)
      before += tiles;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if (mine == 1) return;  // written already
  uint16_t* const dw = p.dw + group * p.size;
  const float* const from = p.partials + before * p.size;
  for (int64_t i = int64_t(block) * kSumThreads + threadIdx.x; i < p.size; i += int64_t(blocks) * kSumThreads) {
    float v = 0.0f;
#pragma unroll 8
    for (int s = 0; s < mine; ++s) v += __ldcg(from + s * p.size + i);
    dw[i] = static_cast<uint16_t>(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
  }
}

}  // namespace fp8lin
