// adapter_kernels.cuh -- what the kernels of the low-rank adapters share.  Row i
// has adapter a(i) of a bank (A_a [r, K], B_a [N, r], s_a) or none:
//   forward    h_i = A_a x_i,  y_i = base_i + B_a (s_a h_i)
//   backward   dh_i = s_a B_a^T dy_i,  dx_i = base_i + A_a^T dh_i
//              dA_a = sum over a's rows of dh_i x_i^T,  dB_a = sum of s_a dy_i h_i^T
//
// With a rank of at most 128 every one of these is bound by reading or writing
// the long side (x, dy, base, y) once.  So no tile of it is shared: a lane has
// eight consecutive values of a row, through slots in shared memory of its own
// that cp.async fills some turns ahead, and they are its part of a fragment as
// they are.  The order of a contraction is free, so those eight are the k index
// of two products, and the order of a product's columns is free, so a lane's
// results are eight consecutive columns.  Where a product contracts over the axis
// that is not contiguous in memory, movmatrix or ldmatrix turns 8 x 8 tiles.  What
// the warps of a CTA have in common (A, B, the rows' low numbers) goes through a
// shared part of the same stages.  mma.sync instead of tcgen05: the operand from
// the long side needs no layout in shared memory and the accumulators no trip
// through tensor memory, and a product over 16 to 128 ranks is done before such a
// pipeline would have started.
// h and dh are fp32; where they are an operand they go in as two bf16 numbers,
// hi + lo, which keeps 16 bits of them (the lost part, 2^-17, is below the
// rounding of y, 2^-8); x, dy, A and B are bf16 as they are.  Sums are fp32.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

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

// Two bf16 values, 0 for one that is infinite or NaN.
__device__ __forceinline__ uint32_t finite_values(uint32_t v) {
  const uint32_t e = v & 0x7F807F80u;
  return ((e & 0x7F80u) == 0x7F80u ? 0u : v & 0xFFFFu) | (e >= 0x7F800000u ? 0u : v & 0xFFFF0000u);
}

// Whether one of the vectors' values is infinite or NaN: such a value times 0 is NaN, any other is 0.
template <int kVecs>
__device__ __forceinline__ bool any_not_finite(const uint4 (&v)[kVecs]) {
  uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[j]) : "r"(word(v[i], j)), "r"(0u));
  return (sum[0] | sum[1] | sum[2] | sum[3]) != 0;
}

// Four 8 x 8 tiles from shared memory, lane l giving the row l % 8 of tile l / 8;
// a lane (g, t) gets of each columns 2t and 2t + 1 of row g, or, turned, rows 2t and
// 2t + 1 of column g.
template <bool kTurn>
__device__ __forceinline__ void load_tiles(uint32_t (&v)[4], const void* row) {
  if constexpr (kTurn)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(smem_addr(row)) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(smem_addr(row)) : "memory");
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
  int block;  // index of its first 16 rows among the blocks of 16 of all groups
};

// Tile `want` of tiles of `size` rows (a multiple of 16) of one group each; a group
// without rows has none.  All lanes of a warp call it and get the same.
__device__ __forceinline__ RowTile find_tile(const Route& r, int groups, int size, int want) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int before = 0, blocks_before = 0;
  for (int base = 0; base < groups; base += 32) {
    const int g = base + lane;
    int begin = 0, count = 0;
    if (g < groups) {
      begin = __ldg(r.first + g);
      count = __ldg(r.first + g + 1) - begin;
    }
    const int tiles = (count + size - 1) / size, blocks = (count + 15) / 16;
    int up = tiles, blocks_up = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, up, o);
      const int b = __shfl_up_sync(0xFFFFFFFFu, blocks_up, o);
      if (lane >= o) {
        up += a;
        blocks_up += b;
      }
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, before + up > want);
    if (hit != 0) {
      const int at = __ffs(static_cast<int>(hit)) - 1;
      const int inside = want - before - __shfl_sync(0xFFFFFFFFu, up - tiles, at);
      RowTile t;
      t.group = base + at;
      t.block = blocks_before + __shfl_sync(0xFFFFFFFFu, blocks_up - blocks, at) + inside * (size / 16);
      t.begin = __shfl_sync(0xFFFFFFFFu, begin, at) + inside * size;
      t.count = min(size, __shfl_sync(0xFFFFFFFFu, count, at) - inside * size);
      return t;
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
    blocks_before += __shfl_sync(0xFFFFFFFFu, blocks_up, 31);
  }
  return RowTile{-1, 0, 0, 0};
}

// Part `part` of `parts` of a group's rows, as many blocks of 16 each but for the last.
__device__ __forceinline__ RowTile group_part(const Route& r, int group, int part, int parts) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int blocks = 0;
  for (int g = lane; g < group; g += 32) blocks += (__ldg(r.first + g + 1) - __ldg(r.first + g) + 15) / 16;
  const int begin = __ldg(r.first + group), count = __ldg(r.first + group + 1) - begin;
  const int each = ((count + 15) / 16 + parts - 1) / parts * 16;
  RowTile t;
  t.group = group;
  t.block = __reduce_add_sync(0xFFFFFFFFu, blocks) + part * (each / 16);
  t.begin = begin + part * each;
  t.count = max(min(each, count - part * each), 0);
  return t;
}

// ---------------------------------------------------------------- stages

constexpr int kAdapterThreads = 256, kAdapterWarps = 8;

// Stages of a turn each: kVecs vectors a thread, its own, and kShared for all
// threads, or (kAlone) that many for each warp.  A turn's copies begin kStages - 1
// turns before it is due:
//   fill the stages 0 to kStages - 2;  each turn: wait(), take(), fill the stage that
//   the turn before left, next()
// wait() ends with a barrier (of the warp where it is alone), after which that stage
// may be filled.  Where rows are not 16-byte aligned a vector is two, those that its
// values lie in.
// kTurned: lanes (g, t) of a warp have the t-th vector of row g, and the vectors lie
// so that the eight of one t are in different banks, for load_tiles() over them.
template <int kStages, int kVecs, int kShared, bool kAlone, bool kAligned, bool kTurned = false>
struct Stages {
  static constexpr int kEach = kAligned ? 1 : 2;
  static constexpr int kOwn = kEach * kVecs * kAdapterThreads;
  static constexpr int kSize = kOwn + (kAlone ? kAdapterWarps : 1) * kShared;
  static constexpr size_t kBytes = sizeof(uint4) * kStages * kSize;
  static constexpr int kCount = kStages;
  uint4* const base;
  int due = 0, filling = 0;  // offsets of stages

  __device__ __forceinline__ explicit Stages(uint4* shared) : base(shared) {}
  __device__ __forceinline__ static int slot() {
    const int i = static_cast<int>(threadIdx.x);
    return kTurned ? i ^ (i >> 3 & 3) : i;
  }
  // The 16 x 16 tile of vectors v (rows 0 to 7) and v + 1 (8 to 15) and the t-th eight
  // columns and the next, turned: the operand whose rows are the columns.
  __device__ __forceinline__ void turned(uint32_t (&a)[4], int v, int t) const {
    const int lane = static_cast<int>(threadIdx.x & 31u), of = lane >> 3, row = lane & 7;
    load_tiles<true>(a, base + due + kEach * (v + (of >> 1)) * kAdapterThreads + (threadIdx.x & ~31u) +
                            4 * row + ((t + (of & 1)) ^ (row >> 1)));
  }
  // Puts vectors that take() has shifted into place, for turned().
  __device__ __forceinline__ void put_back(const uint4 (&x)[kVecs]) const {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) base[due + kEach * v * kAdapterThreads + slot()] = x[v];
    __syncwarp();
  }
  __device__ __forceinline__ static void step(int& stage) {
    stage = stage == (kStages - 1) * kSize ? 0 : stage + kSize;
  }
  __device__ __forceinline__ uint4* shared_at(int stage) const {
    return base + stage + kOwn + (kAlone ? (threadIdx.x >> 5) * kShared : 0);
  }
  __device__ __forceinline__ uint4* shared_filling() const { return shared_at(filling); }
  __device__ __forceinline__ const uint4* shared_due() const { return shared_at(due); }
  // The thread's own vectors of the turn that is filled: from(vector, n) gives a
  // pointer and how many values it has.
  template <typename From>
  __device__ __forceinline__ void copy(From from) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      int n;
      const uint16_t* p = from(v, n);
      uint4* const to = base + filling + kEach * v * kAdapterThreads + slot();
      if constexpr (kAligned) {
        copy16(to, p, n > 0);
      } else {
        const int off = offset(p);
        copy16(to, p - off, n > 0);
        copy16(to + kAdapterThreads, p - off + 8, n > 0 && off + n > 8);
      }
    }
  }
  __device__ __forceinline__ void filled() {
    copies_end();
    step(filling);
  }
  // The vectors of the turn that is due, with the same from().
  template <typename From>
  __device__ __forceinline__ void take(uint4 (&out)[kVecs], From from) const {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const uint4* const at = base + due + kEach * v * kAdapterThreads + slot();
      if constexpr (kAligned) {
        out[v] = at[0];
      } else {
        int n;
        const uint16_t* p = from(v, n);
        out[v] = shift_values(at[0], at[kAdapterThreads], static_cast<uint32_t>(offset(p)));
        if (n < 8) out[v] = first_values(out[v], n);
      }
    }
  }
  __device__ __forceinline__ void wait() const {
    copies_wait<kStages - 2>();
    if constexpr (kAlone)
      __syncwarp();
    else
      __syncthreads();
  }
  __device__ __forceinline__ void next() { step(due); }

 private:
  // Values between a pointer and the 16-byte boundary before it.
  __device__ __forceinline__ static int offset(const uint16_t* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
  }
};

// As many stages as `bytes` hold, 2 to 8.
constexpr int stages_in(size_t bytes, size_t stage) {
  const size_t n = bytes / stage;
  return n < 2 ? 2 : n > 8 ? 8 : static_cast<int>(n);
}
// Two CTAs an SM.
constexpr size_t kStageRoom = 96 * 1024;

// 8 bytes to shared memory, as copy16.
__device__ __forceinline__ void copy8(void* to, const void* from, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_addr(to)), "l"(from),
               "r"(on ? 8 : 0)
               : "memory");
}

// A stage of a weight, kSpans times 32 columns that lie `apart` apart and all ranks,
// filled by the CTA or (kAlone) by each warp for itself.
//   kColumns = false: A, [r, cols].  Rank j of span s is at (s * 8 * kRankTiles + j) * 4,
//     four vectors of eight columns.
//   kColumns = true: B, [cols, r], vectors of eight ranks.  The products take the
//     eight columns 8 (k / 2) + 2 q + k % 2 of 32 together, so these lie side by side,
//     as place 8 q + k, and a column's vectors are in an order turned by its place, so
//     that the eight lie in different banks.
__device__ __forceinline__ int column_place(int col) {
  return (col & ~31) + ((col >> 1 & 3) << 3) + (col >> 3 & 3) * 2 + (col & 1);
}
template <int kRankTiles>
__device__ __forceinline__ int place_vector(int place, int piece) {
  constexpr int kTurns = kRankTiles < 8 ? kRankTiles : 8;
  return place * kRankTiles + (piece ^ ((place & 7) * kTurns / 8));
}

template <int kRankTiles, int kSpans, bool kColumns, bool kAlone, bool kAligned>
struct WeightStage {
  static constexpr int kVecs = kSpans * kRankTiles * 32, kThreads = kAlone ? 32 : kAdapterThreads;
  static constexpr int kPieces = (kVecs + kThreads - 1) / kThreads;
  static constexpr bool kKept = kPieces <= 2;  // few enough to keep what does not change
  struct Piece {
    int from, col, n, to;  // offset in w, column (both from c on), values a vector has, place
  };
  const uint16_t* const w;
  const int apart, cols, rank;
  Piece kept[kKept ? kPieces : 1];

  __device__ __forceinline__ WeightStage(const uint16_t* weight, int between, int columns, int ranks)
      : w(weight), apart(between), cols(columns), rank(ranks) {
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) kept[i] = piece(i);
    }
  }
  __device__ __forceinline__ Piece piece(int of) const {
    const int i = of * kThreads + static_cast<int>(threadIdx.x) % kThreads;
    Piece p;
    if constexpr (kColumns) {
      const int k = i / kRankTiles, part = i % kRankTiles;
      p.col = (k >> 5) * apart + (k & 31);
      p.n = values_at(8 * part, rank);
      p.from = p.col * rank + (p.n > 0 ? 8 * part : 0);
      p.to = place_vector<kRankTiles>(column_place(k), part);
    } else {
      const int j = i / 4 % (8 * kRankTiles);
      p.col = apart * (i / (kRankTiles * 32)) + 8 * (i & 3);
      p.n = j < rank ? 8 : 0;
      p.from = (j < rank ? j : 0) * cols + p.col;
      p.to = i;
    }
    if (kVecs % kThreads != 0 && i >= kVecs) p.n = -1;  // no such vector
    return p;
  }
  // Columns c on into a stage.
  __device__ __forceinline__ void copy(uint4* to, int c) const {
    const uint16_t* const at = w + (kColumns ? int64_t(c) * rank : int64_t(c));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const Piece p = kKept ? kept[kKept ? i : 0] : piece(i);
      if (kVecs % kThreads != 0 && p.n < 0) continue;
      const bool on = p.n > 0 && c + p.col < cols;
      const uint16_t* const from = at + p.from;
      if constexpr (!kAligned) {
        to[p.to] = load_values<false>(from, !on ? 0 : kColumns ? p.n : values_at(c + p.col, cols));
      } else if (!kColumns || rank % 8 == 0) {
        copy16(to + p.to, from, on);
      } else {  // a multiple of 4
        copy8(to + p.to, from, on);
        copy8(reinterpret_cast<uint2*>(to + p.to) + 1, p.n > 4 ? from + 4 : from, on && p.n > 4);
      }
    }
  }
};

// ---------------------------------------------------------------- launching

// Launches a kernel that may need more dynamic shared memory than the default.
template <auto* kKernel, typename... Args>
cudaError_t launch_staged(dim3 grid, size_t bytes, const DeviceInfo& dev, cudaStream_t stream, int cluster,
                          const Args&... args) {
  if (bytes > 0) {
    static std::mutex mu;
    static bool done[64];  // devices on which the kernel may have that much
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev.device]) {
      const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(bytes));
      if (e != cudaSuccess) return e;
      done[dev.device] = true;
    }
  }
  return launch_kernel(kKernel, grid, dim3(kAdapterThreads), bytes, stream, cluster, false, args...);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool rows_aligned(const void* p, int64_t ld, int64_t cols) {
  return p == nullptr || (aligned16(p) && ld % 8 == 0 && cols % 8 == 0);
}

// 1, 2, 4, 8 or 16 tiles of eight ranks.
inline int rank_tiles(int rank) {
  int t = 1;
  while (8 * t < rank) t *= 2;
  return t;
}

template <int kValue>
using Int = std::integral_constant<int, kValue>;
using Yes = std::true_type;
using No = std::false_type;

template <typename Run>
cudaError_t with_rank_tiles(int rank, Run run) {
  switch (rank_tiles(rank)) {
    case 1: return run(Int<1>());
    case 2: return run(Int<2>());
    case 4: return run(Int<4>());
    case 8: return run(Int<8>());
    default: return run(Int<16>());
  }
}

// Tiles of `size` rows, at most: each adapter with rows may end inside one.
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t size) {
  const int64_t t = rows / size + groups;
  return t < rows ? t : rows;
}

inline Route route_of(const AdapterArgs& a) {
  return Route{a.route, a.route + a.count + 2, static_cast<int>(a.count) + 1};
}

// Whether a stage of A or B can be filled by copies.
inline bool a_aligned(const AdapterArgs& a) { return aligned16(a.a) && a.k % 8 == 0; }
inline bool b_aligned(const AdapterArgs& a) { return aligned16(a.b) && a.rank % 4 == 0; }

}  // namespace fp8lin
