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
  bool only;  // the group's only tile
};

// Tile `want` of tiles of `size` rows of one group each (a group without rows
// has none).  All lanes of a warp call it and get the same.
__device__ __forceinline__ RowTile find_tile(const Route& r, int groups, int size, int want) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int before = 0, several_before = 0;
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    int begin = 0, count = 0;
    if (g < groups) {
      begin = __ldg(r.first + g);
      count = __ldg(r.first + g + 1) - begin;
    }
    const int tiles = (count + size - 1) / size, several = tiles > 1 ? tiles : 0;
    int up = tiles, several_up = several;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, up, o);
      const int b = __shfl_up_sync(0xFFFFFFFFu, several_up, o);
      if (lane >= o) {
        up += a;
        several_up += b;
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
      t.begin = __shfl_sync(0xFFFFFFFFu, begin, at) + inside * size;
      t.count = min(size, __shfl_sync(0xFFFFFFFFu, count, at) - inside * size);
      return t;
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
    several_before += __shfl_sync(0xFFFFFFFFu, several_up, 31);
  }
  return RowTile{-1, 0, 0, 0, false};
}

// ---------------------------------------------------------------- low = x W^T

// low[i][j] = scale_a * sum_c x[i][c] w_a[j][c] for the rows i of one tile, 16 *
// kTiles of them.  kAlong: w_a is [r, cols] (A: contiguous along the contraction);
// else [cols, r] (B).  The CTA's warps take 32 columns each in turn, and so do
// the CTAs of a cluster; their sums meet in shared memory.
struct LowArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;
  const float* scale;  // null: 1
  float* low;          // [rows, rank] dense
  int cols, rank;
  int parts;  // CTAs of a cluster
  Route route;
  bool w_aligned;
};

constexpr int kLowWarps = 8;

// Ranks a lane holds side by side of a [cols, r] weight.
constexpr int ranks_a_lane(int rank_tiles) { return rank_tiles >= 4 ? 8 : 2 * rank_tiles; }

template <int kTiles, int kRankTiles, bool kAlong, bool kAligned>
__global__ void __launch_bounds__(32 * kLowWarps)
    adapter_low_kernel(const __grid_constant__ LowArgs p) {
  __shared__ float sums[kLowWarps / 2][kTiles * kRankTiles * 4][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int g = lane >> 2, t = lane & 3;
  const int parts = p.parts, part = static_cast<int>(blockIdx.x) % parts;
  const RowTile tile =
      find_tile(p.route, p.route.groups, 16 * kTiles, static_cast<int>(blockIdx.x) / parts);
  if (tile.group < 0) return;  // all CTAs of the cluster
  int64_t row[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = m * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
    }
  const bool none = tile.group == p.route.groups - 1;
  if (none) {
    if (part == 0)
      for (int at = warp; at < tile.count; at += kLowWarps)
        for (int j = lane; j < p.rank; j += 32)
          p.low[int64_t(__ldg(p.route.rows + tile.begin + at)) * p.rank + j] = 0.0f;
    return;
  }
  const uint16_t* const w = p.w + int64_t(tile.group) * p.rank * p.cols;
  float acc[kTiles][kRankTiles][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  constexpr int kWide = ranks_a_lane(kRankTiles);
  const int step = 32 * kLowWarps * parts;
#pragma unroll 2
  for (int c = 32 * (part * kLowWarps + warp); c < p.cols; c += step) {
    const int col = c + 8 * t;
    const int n = kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
    uint4 x[kTiles][2];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[m][i] = row[m][i] >= 0 ? load_values<kAligned>(p.x + row[m][i] * p.ldx + col, n)
                                 : make_uint4(0, 0, 0, 0);
    if constexpr (kAlong) {
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) {
        const int rank = 8 * j + g;
        uint4 b = make_uint4(0, 0, 0, 0);
        if (rank < p.rank) {
          const uint16_t* from = w + int64_t(rank) * p.cols + col;
          b = p.w_aligned ? load_values<true>(from, n) : load_values<false>(from, n);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
            mma_bf16(acc[m][j], word(x[m][0], 2 * s), word(x[m][1], 2 * s), word(x[m][0], 2 * s + 1),
                     word(x[m][1], 2 * s + 1), word(b, 2 * s), word(b, 2 * s + 1));
      }
    } else {
      // Row k of a product's tile is column 8 (k / 2) + 4 s + k % 2 of the 32,
      // and two more in its second half: the order in which a lane holds x.
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int block = 0; block < (kRankTiles + 3) / 4; ++block) {
          uint4 b[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int from_col = c + 8 * (g >> 1) + 4 * s + 2 * half + (g & 1);
            const int rank = 32 * block + kWide * t;
            b[half] = make_uint4(0, 0, 0, 0);
            if (from_col < p.cols && rank < p.rank) {
              const uint16_t* from = w + int64_t(from_col) * p.rank + rank;
              if (!p.w_aligned) {
                b[half] = load_values<false>(from, min(kWide, p.rank - rank));
              } else if constexpr (kWide == 8) {
                b[half] = *reinterpret_cast<const uint4*>(from);
              } else if constexpr (kWide == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                b[half] = make_uint4(v.x, v.y, 0, 0);
              } else {
                b[half].x = *reinterpret_cast<const uint32_t*>(from);
              }
            }
          }
#pragma unroll
          for (int q = 0; q < kWide / 2; ++q) {
            const uint32_t b0 = turn_tile(word(b[0], q)), b1 = turn_tile(word(b[1], q));
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
              mma_bf16(acc[m][4 * block + q], word(x[m][0], 2 * s), word(x[m][1], 2 * s),
                       word(x[m][0], 2 * s + 1), word(x[m][1], 2 * s + 1), b0, b1);
          }
        }
      }
    }
  }
  // The warps' sums: the upper half's to shared memory, added by the lower.
#pragma unroll
  for (int half = kLowWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[warp - half][(m * kRankTiles + j) * 4 + i][lane] = acc[m][j][i];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][j][i] += sums[warp][(m * kRankTiles + j) * 4 + i][lane];
    }
    __syncthreads();
  }
  if (parts > 1) {  // the cluster's: every other CTA's from its shared memory, in order
    if (warp == 0 && part != 0) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[0][(m * kRankTiles + j) * 4 + i][lane] = acc[m][j][i];
    }
    cluster_sync_all();
    if (warp == 0 && part == 0) {
      for (int from = 1; from < parts; ++from) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[m][j][i] += __uint_as_float(ld_shared_cluster_u32(
                  map_to_cta(smem_addr(&sums[0][(m * kRankTiles + j) * 4 + i][lane]), from)));
      }
    }
    cluster_sync_all();
  }
  if (warp != 0 || part != 0) return;
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t to = row[m][i >> 1];
        const int rank = kAlong ? 8 * j + 2 * t + (i & 1)
                                : 32 * (j >> 2) + kWide * t + 2 * (j & 3) + (i & 1);
        if (to >= 0 && rank < p.rank) p.low[to * p.rank + rank] = scale * acc[m][j][i];
      }
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
  bool w_aligned, low_aligned;
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

template <int kTiles, int kSteps, bool kAlong, bool kAligned>
__global__ void __launch_bounds__(32 * kHighWarps)
    adapter_high_kernel(const __grid_constant__ HighArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int g = lane >> 2, t = lane & 3;
  const RowTile tile = find_tile(p.route, p.route.groups, 16 * kTiles, static_cast<int>(blockIdx.x));
  if (tile.group < 0) return;
  const bool none = tile.group == p.route.groups - 1;
  if (none && p.y == p.base) return;
  const int begin = static_cast<int>(blockIdx.y) * p.slab;
  const int end = min(begin + p.slab, p.cols);
  int64_t row[kTiles][2];
  LowFragments<kTiles, kSteps> f;
  const float scale = none || p.scale == nullptr ? 1.0f : __ldg(p.scale + tile.group);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = m * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int rank = rank_at<kSteps>(s, t);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row[m][i] >= 0 && !none)
          v = load_ranks(p.low + row[m][i] * p.rank + rank, p.rank - rank, p.low_aligned);
        split_pair(v.x * scale, v.y * scale, f.hi[m][s][i], f.lo[m][s][i]);
        split_pair(v.z * scale, v.w * scale, f.hi[m][s][i + 2], f.lo[m][s][i + 2]);
      }
    }
  const uint16_t* const w = none ? nullptr : p.w + int64_t(tile.group) * p.rank * p.cols;
  for (int c = begin + 32 * warp; c < end; c += 32 * kHighWarps) {
    const int col = c + 8 * t;
    const int n = kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
    uint4 base[kTiles][2];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        base[m][i] = p.base != nullptr && row[m][i] >= 0
                         ? load_values<kAligned>(p.base + row[m][i] * p.ldbase + col, n)
                         : make_uint4(0, 0, 0, 0);
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
            uint4 v = make_uint4(0, 0, 0, 0);
            if (from_col < p.cols && rank < p.rank) {
              const uint16_t* from = w + int64_t(from_col) * p.rank + rank;
              if (!p.w_aligned) {
                v = load_values<false>(from, min(kWide, p.rank - rank));
              } else if constexpr (kWide == 8) {
                v = *reinterpret_cast<const uint4*>(from);
              } else {
                const uint2 u = *reinterpret_cast<const uint2*>(from);
                v = make_uint4(u.x, u.y, 0, 0);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) b[q][i] = word(v, i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < (kSteps == 1 ? 2 : 4); ++i) {
            const int rank = rank_at<kSteps>(2 * block + (i >> 1), g >> 1) + 2 * (i & 1) + (g & 1);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (rank < p.rank) {
              const uint16_t* from = w + int64_t(rank) * p.cols + col;
              v = p.w_aligned ? load_values<true>(from, n) : load_values<false>(from, n);
            }
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
          bf16x8_to_f32(base[m][i], v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[2 * q] += acc[m][q][2 * i];
            v[2 * q + 1] += acc[m][q][2 * i + 1];
          }
          base[m][i] = f32_to_bf16x8(v);
        }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        store_values<kAligned, 4>(p.y + (row[m][i] < 0 ? 0 : row[m][i]) * p.ldy + col, base[m][i],
                                  row[m][i] < 0 ? 0 : n);
  }
}

// ---------------------------------------------------------------- dW = x^T low

// dw[c][j] = sum over the rows i of one adapter of x[i][c] scale_a low[i][j], for
// `slab` columns c.  A tile of rows that is its adapter's only one is written as
// bf16 into dw; else its sums go to the partials, one slot a tile, which
// adapter_sum_kernel adds up.  kAlong: dw is [cols, r] (dB), else [r, cols] (dA).
struct WeightArgs {
  const uint16_t* x;
  int64_t ldx;
  const float* low;
  const float* scale;  // null: 1
  uint16_t* dw;
  float* partials;  // [slot][cols * rank]
  int cols, rank, tile_rows;
  Route route;
};

constexpr int kWeightWarps = 8;
constexpr int kWeightRows = 64;  // rows of low in shared memory at a time

// 16-column tiles of x that a warp holds sums for.
constexpr int weight_tiles(int rank_tiles) { return rank_tiles >= 8 ? 2 : 4; }
constexpr int weight_slab(int rank_tiles) { return kWeightWarps * 16 * weight_tiles(rank_tiles); }

template <int kRankTiles, bool kAlong, bool kAligned>
__global__ void __launch_bounds__(32 * kWeightWarps)
    adapter_weight_kernel(const __grid_constant__ WeightArgs p) {
  constexpr int kTiles = weight_tiles(kRankTiles), kChunks = kTiles / 2;
  constexpr int kRanks = 8 * kRankTiles;
  // Rows 2 k and 2 k + 1 of low side by side: [hi, lo][k][rank]; the padding
  // spreads the four k of a quarter-warp over the banks.
  constexpr int kPitch = kRanks % 32 == 8 ? kRanks : (kRanks + 31) / 32 * 32 + 8;
  __shared__ uint32_t low[2][kWeightRows / 2][kPitch];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int g = lane >> 2, t = lane & 3;
  const RowTile tile = find_tile(p.route, p.route.groups - 1, p.tile_rows, static_cast<int>(blockIdx.x));
  if (tile.group < 0) return;
  const int col0 = (static_cast<int>(blockIdx.y) * kWeightWarps + warp) * 16 * kTiles;
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
  float acc[kTiles][kRankTiles][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  for (int r0 = 0; r0 < tile.count; r0 += kWeightRows) {
    const int rows = min(kWeightRows, tile.count - r0);
    __syncthreads();
    for (int i = static_cast<int>(threadIdx.x); i < kWeightRows / 2 * kRanks; i += 32 * kWeightWarps) {
      const int k = i / kRanks, j = i % kRanks;
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] = 0.0f;
        if (2 * k + e < rows && j < p.rank)
          v[e] = scale * p.low[int64_t(__ldg(p.route.rows + tile.begin + r0 + 2 * k + e)) * p.rank + j];
      }
      split_pair(v[0], v[1], low[0][k][j], low[1][k][j]);
    }
    __syncthreads();
    if (col0 >= p.cols) continue;
    for (int r = 0; r < rows; r += 16) {
      int64_t row[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = r + i * 8 + g;
        row[i] = at < rows ? __ldg(p.route.rows + tile.begin + r0 + at) : -1;
      }
      uint4 x[kChunks][2];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = col0 + 32 * c + 8 * t;
          const int n = kAligned ? (col < p.cols ? 8 : 0) : values_at(col, p.cols);
          x[c][i] = row[i] >= 0 ? load_values<kAligned>(p.x + row[i] * p.ldx + col, n)
                                : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t a[4][2];  // of columns 8 (k / 2) + 2 q + k % 2, rows 0-7 and 8-15
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) a[q][i] = turn_tile(word(x[c][i], q));
#pragma unroll
        for (int j = 0; j < kRankTiles; ++j) {
#pragma unroll
          for (int part = 1; part >= 0; --part) {
            const uint32_t b0 = low[part][r / 2 + t][8 * j + g], b1 = low[part][r / 2 + 4 + t][8 * j + g];
#pragma unroll
            for (int m = 0; m < 2; ++m)
              mma_bf16(acc[2 * c + m][j], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], b0, b1);
          }
        }
      }
    }
  }
  if (col0 >= p.cols) return;
  const int64_t size = int64_t(p.cols) * p.rank;
  uint16_t* const dw = p.dw + tile.group * size;
  float* const part = tile.only ? nullptr : p.partials + tile.slot * size;
  // A lane has of product (c, j) columns 8 (g / 2) + 2 q + g % 2, q = 0 .. 3, of
  // ranks 8 j + 2 t and the next.
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j) {
      if constexpr (kAlong) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = col0 + 32 * c + 8 * (g >> 1) + 2 * q + (g & 1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rank = 8 * j + 2 * t + e;
            if (col >= p.cols || rank >= p.rank) continue;
            const float v = acc[2 * c + (q >> 1)][j][2 * (q & 1) + e];
            const int64_t at = int64_t(col) * p.rank + rank;
            if (part != nullptr)
              part[at] = v;
            else
              dw[at] = static_cast<uint16_t>(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
          }
        }
      } else {
        // Lanes of neighbouring g swap, so that one has eight columns side by
        // side of the first rank and the other of the second.
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
        if (rank >= p.rank) continue;
        const int64_t at = int64_t(rank) * p.cols + col;
        if (kAligned && col < p.cols) {
          if (part != nullptr) {
            float4* to = reinterpret_cast<float4*>(part + at);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            *reinterpret_cast<uint4*>(dw + at) = f32_to_bf16x8(v);
          }
          continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col + i >= p.cols) continue;
          if (part != nullptr)
            part[at + i] = v[i];
          else
            dw[at + i] = static_cast<uint16_t>(cvt_bf16x2(v[i], 0.0f) & 0xFFFFu);
        }
      }
    }
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
