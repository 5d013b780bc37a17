// adapter_high.cu -- the adapters' product over the ranks, added to a base:
//   y[i][c] = base[i][c] + sum_j s_a low[i][j] w_a(j, c)
// y = base + s h B^T in the forward, dx = base + dh A in the backward.
//
// Bound by reading base and writing y: 16384 x 4096 with rank 16 takes 49 us (5.5 TB/s);
// 8192 x 4096 with rank 64 47 us, of which the products of hi and lo are 14 of tensor
// pipe and their operands' loads as much again.  A and B go through shared stages
// (loaded from L2 for each product, rank 64 took 51 us with the operands' latency bare).
// Rows of y that are not 16-byte aligned: 777 x 4801 with rank 8 takes 15 us; each lane
// shifts its vectors, and a row's piece of a CTA begins and ends inside one.
#include "adapter_kernels.cuh"

namespace fp8lin {
namespace {

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

// A tile of 16 * kTiles rows for each of kRowWarps warps, and `slab` columns, of
// which every other warp takes 32 a turn.  kSteps products of 16 ranks, each for
// hi and lo.  kAlong: w_a is [cols, r] (B), else [r, cols] (A).
template <int kTiles, int kSteps, int kRowWarps, bool kAligned>
struct HighShape {
  static constexpr int kColWarps = kAdapterWarps / kRowWarps;
  // Where the weight is small beside y each warp has its own, and there are no barriers.
  static constexpr bool kAlone = kSteps == 1 || kRowWarps == 1;
  static constexpr int kSpans = kAlone ? 1 : kColWarps;
  static constexpr int kShared = kSpans * 2 * kSteps * 32;
  static constexpr size_t kStage =
      sizeof(uint4) * ((kAligned ? 2 : 4) * kTiles * kAdapterThreads + (kAlone ? kAdapterWarps : 1) * kShared);
  using S = Stages<stages_in(kStageRoom, kStage), 2 * kTiles, kShared, kAlone, kAligned>;
};

__device__ __forceinline__ float2 load_ranks(const float* from, int n, bool aligned) {
  if (aligned && n >= 2) return *reinterpret_cast<const float2*>(from);
  float2 v = make_float2(0.0f, 0.0f);
  if (n > 0) v.x = from[0];
  if (n > 1) v.y = from[1];
  return v;
}

template <int kTiles, int kSteps, int kRowWarps, bool kAlong, bool kAligned, bool kWAligned>
__global__ void __launch_bounds__(kAdapterThreads, kSteps <= 4 ? 2 : 1)
    adapter_high_kernel(const __grid_constant__ HighArgs p) {
  using Shape = HighShape<kTiles, kSteps, kRowWarps, kAligned>;
  using S = typename Shape::S;
  constexpr int kColWarps = Shape::kColWarps, kRankTiles = 2 * kSteps, kTurn = 32 * kColWarps;
  extern __shared__ uint4 shared[];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int row_warp = warp % kRowWarps, col_warp = warp / kRowWarps;
  const int g = lane >> 2, t = lane & 3;
  const RowTile tile =
      find_tile(p.route, p.route.groups, 16 * kTiles * kRowWarps, static_cast<int>(blockIdx.x));
  const bool none = tile.group == p.route.groups - 1;
  if (tile.group < 0 || (none && p.y == p.base)) return;
  const int begin = static_cast<int>(blockIdx.y) * p.slab;
  const int end = min(begin + p.slab, p.cols);
  // A warp's turns: every kColWarps-th 32 columns, or, where rows of y are not
  // aligned, 32 after 32, so that what a turn leaves of a vector the next one writes.
  const int span = kAligned ? 32 : p.slab / kColWarps, apart = kAligned ? kTurn : 32;
  const int turns = kAligned ? (end - begin + kTurn - 1) / kTurn : min(span, end - begin + 31) / 32;
  int64_t row[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (row_warp * kTiles + m) * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
    }
  const bool idle = row_warp * kTiles * 16 >= tile.count;
  const uint16_t* const w = none ? nullptr : p.w + int64_t(tile.group) * p.rank * p.cols;
  S stages(shared);
  const int begin_warp = begin + span * col_warp, end_warp = kAligned ? end : min(begin_warp + span, end);
  auto base_of = [&](int turn) {
    return [&, c = begin_warp + turn * apart + 8 * t](int v, int& n) {
      const int64_t of = row[v >> 1][v & 1];
      n = p.base == nullptr || of < 0 || turn >= turns ? 0 : values_at(c, end_warp);
      return p.base + (of < 0 ? 0 : of) * p.ldbase + c;
    };
  };
  const WeightStage<kRankTiles, Shape::kSpans, kAlong, Shape::kAlone, kWAligned> weight(w, span, p.cols, p.rank);
  auto copy_w = [&](int turn) {
    if (turn < turns && !none && !(Shape::kAlone && idle))
      weight.copy(stages.shared_filling(), (Shape::kAlone ? begin_warp : begin) + turn * apart);
  };
#pragma unroll
  for (int i = 0; i < S::kCount - 1; ++i) {
    copy_w(i);
    stages.copy(base_of(i));
    stages.filled();
  }
  uint32_t hi[kTiles][kSteps][4], lo[kTiles][kSteps][4];  // low of the rows, as an operand
  const float scale = none || p.scale == nullptr ? 1.0f : __ldg(p.scale + tile.group);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int rank = 16 * s + 8 * (i >> 1) + 2 * t;
        float2 v = make_float2(0.0f, 0.0f);
        if (row[m][i & 1] >= 0 && !none)
          v = load_ranks(p.low + row[m][i & 1] * p.rank + rank, p.rank - rank, p.low_aligned);
        split_pair(v.x * scale, v.y * scale, hi[m][s][i], lo[m][s][i]);
      }
  StoreRun<4> runs[kAligned ? 1 : 2 * kTiles];
  for (int turn = 0; turn < turns; ++turn, stages.next()) {
    stages.wait();
    uint4 out[2 * kTiles];
    stages.take(out, base_of(turn));
    copy_w(turn + S::kCount - 1);
    stages.copy(base_of(turn + S::kCount - 1));
    stages.filled();
    const int col = begin_warp + turn * apart + 8 * t;
    if (idle) continue;
    // Adds the products to out.  kGuarded: lo only where the weight is finite.
    auto add_products = [&](auto guarded) {
      const uint4* const ws = stages.shared_due() + (Shape::kAlone ? 0 : col_warp * kRankTiles * 32);
      float acc[kTiles][4][4];
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.0f;
      // Column k of product q is column 8 (k / 2) + 2 q + k % 2 of the 32.
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t b[2][4];  // ranks 16 s to 16 s + 7 and the next eight, of the four products
        if constexpr (kAlong) {
#pragma unroll
          for (int i = 0; i < 2; ++i) load_tiles<false>(b[i], ws + place_vector<kRankTiles>(lane, 2 * s + i));
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = ws[(16 * s + 8 * i + g) * 4 + t];
#pragma unroll
            for (int q = 0; q < 4; ++q) b[i][q] = turn_tile(word(v, q));
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            if constexpr (decltype(guarded)::value)
              mma_bf16(acc[m][q], lo[m][s][0], lo[m][s][1], lo[m][s][2], lo[m][s][3], finite_values(b[0][q]),
                       finite_values(b[1][q]));
            else
              mma_bf16(acc[m][q], lo[m][s][0], lo[m][s][1], lo[m][s][2], lo[m][s][3], b[0][q], b[1][q]);
            mma_bf16(acc[m][q], hi[m][s][0], hi[m][s][1], hi[m][s][2], hi[m][s][3], b[0][q], b[1][q]);
          }
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[8];
          bf16x8_to_f32(out[2 * m + i], v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[2 * q] += acc[m][q][2 * i];
            v[2 * q + 1] += acc[m][q][2 * i + 1];
          }
          out[2 * m + i] = f32_to_bf16x8(v);
        }
    };
    const int n = values_at(col, end_warp);
    auto store = [&]() {
#pragma unroll
      for (int v = 0; v < 2 * kTiles; ++v) {
        const int64_t of = row[v >> 1][v & 1];
        uint16_t* const to = p.y + (of < 0 ? 0 : of) * p.ldy + col;
        if constexpr (kAligned) {
          if (of >= 0 && n > 0) *reinterpret_cast<uint4*>(to) = out[v];
        } else {
          runs[v].store(to, out[v], of < 0 ? 0 : n);
        }
      }
    };
    if (!none) add_products(No());
    // hi w + lo w is NaN for an infinite w unless hi and lo have the same sign.  Aligned rows are
    // looked at while they are on their way out, and then written again.
    if constexpr (kAligned) store();
    if (!none && __any_sync(0xFFFFFFFFu, any_not_finite(out))) {
      stages.take(out, base_of(turn));
      add_products(Yes());
      if constexpr (kAligned) store();
    }
    if constexpr (!kAligned) store();
  }
  if constexpr (!kAligned) {
#pragma unroll
    for (int v = 0; v < 2 * kTiles; ++v) runs[v].end();
  }
  copies_wait<0>();
}

}  // namespace

cudaError_t launch_adapter_high(const AdapterArgs& a, bool backward, const float* low,
                                const uint16_t* base, int64_t ldbase, uint16_t* y, int64_t ldy,
                                const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("adapter_high_kernel");
  HighArgs p = {};
  p.low = low;
  p.w = backward ? a.a : a.b;
  p.scale = backward ? nullptr : a.scale;
  p.base = base;
  p.y = y;
  p.ldbase = base != nullptr ? ldbase : 0;
  p.ldy = ldy;
  p.cols = static_cast<int>(backward ? a.k : a.n);
  p.rank = a.rank;
  p.route = route_of(a);
  p.low_aligned = aligned16(low) && a.rank % 2 == 0;
  const bool aligned = rows_aligned(base, ldbase, p.cols) && rows_aligned(y, ldy, p.cols);
  const bool w_aligned = backward ? a_aligned(a) : b_aligned(a);
  return with_rank_tiles(a.rank, [&](auto ranks) {
    constexpr int kSteps = decltype(ranks)::value <= 2 ? 1 : decltype(ranks)::value / 2;
    auto run = [&](auto tiles, auto row_warps) {
      constexpr int kTiles = decltype(tiles)::value, kRowWarps = decltype(row_warps)::value;
      const int64_t most = most_tiles(a.rows, a.count + 1, 16 * kTiles * kRowWarps);
      // Slabs of whole turns; one wave of two CTAs an SM, as far as the rows have tiles.
      constexpr int kTurn = 32 * kAdapterWarps / kRowWarps;
      const int turns = (p.cols + kTurn - 1) / kTurn;
      int64_t slabs = 2 * int64_t(dev.num_sms) / most;
      slabs = slabs < 1 ? 1 : slabs > turns ? turns : slabs;
      const int per = static_cast<int>((turns + slabs - 1) / slabs);
      p.slab = per * kTurn;
      const dim3 grid(static_cast<unsigned>(most), static_cast<unsigned>((turns + per - 1) / per));
      auto go = [&](auto along, auto whole, auto w_whole) {
        constexpr bool kAligned = decltype(whole)::value;
        return launch_staged<adapter_high_kernel<kTiles, kSteps, kRowWarps, decltype(along)::value, kAligned,
                                                 decltype(w_whole)::value>>(
            grid, HighShape<kTiles, kSteps, kRowWarps, kAligned>::S::kBytes, dev, stream, 1, p);
      };
      if (!w_aligned) return backward ? go(No(), No(), No()) : go(Yes(), No(), No());
      if (backward) return aligned ? go(No(), Yes(), Yes()) : go(No(), No(), Yes());
      return aligned ? go(Yes(), Yes(), Yes()) : go(Yes(), No(), Yes());
    };
    // Wide tiles share w, narrow ones waste fewer rows.  Rank 64: 8192 x 4096 x 4096
    // with 4 adapters takes 78 us in all wide and 105 narrow, with 64 adapters 112 and
    // 108.  Rank 16, where w is little: 51 and 54, but 66 and 55 with 64 adapters, 21
    // and 20 for 2048 rows of 4.
    if (a.rows < (kSteps == 1 ? 1024 : 256) * a.count) return run(Int<1>(), Int<1>());
    return run(Int<kSteps <= 2 ? 2 : 1>(), Int<4>());
  });
}

}  // namespace fp8lin
