// adapter_low.cu -- the adapters' product over the long side:
//   low[i][j] = s_a sum_c x[i][c] w_a(j, c)
// h = x A^T in the forward, dh = s dy B in the backward.
//
// Bound by reading x: 16384 x 14336 with rank 16 takes 83 us (5.7 TB/s), 8192 x 4096
// with rank 64 27 us, where 64 KB of x on the way in an SM and 8 us at a CTA's start
// and end are what is left.  One wave of CTAs: with three of half the size it took 98.
#include "adapter_kernels.cuh"

namespace fp8lin {
namespace {

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

// A tile of 16 * kTiles rows for each of kRowWarps warps.  The other warps, and the
// CTAs of a cluster, take other columns, 32 each a turn; their sums meet in shared
// memory.  kAlong: w_a is [r, cols] (A), else [cols, r] (B).
template <int kTiles, int kRankTiles, int kRowWarps, bool kAligned>
struct LowShape {
  static constexpr int kColWarps = kAdapterWarps / kRowWarps;
  // Where the weight is small beside x each warp has its own, and there are no barriers.
  static constexpr bool kAlone = kRankTiles <= 2 || kRowWarps == 1;
  static constexpr int kSpans = kAlone ? 1 : kColWarps;
  static constexpr int kShared = kSpans * kRankTiles * 32;
  static constexpr size_t kStage =
      sizeof(uint4) * ((kAligned ? 2 : 4) * kTiles * kAdapterThreads + (kAlone ? kAdapterWarps : 1) * kShared);
  using S = Stages<stages_in(kStageRoom, kStage), 2 * kTiles, kShared, kAlone, kAligned>;
};

template <int kTiles, int kRankTiles, int kRowWarps, bool kAlong, bool kAligned, bool kWAligned>
__global__ void __launch_bounds__(kAdapterThreads, kRankTiles <= 8 ? 2 : 1)
    adapter_low_kernel(const __grid_constant__ LowArgs p) {
  using Shape = LowShape<kTiles, kRankTiles, kRowWarps, kAligned>;
  using S = typename Shape::S;
  constexpr int kColWarps = Shape::kColWarps, kSums = kTiles * kRankTiles * 4;
  extern __shared__ uint4 shared[];
  __shared__ float sums[kAdapterWarps / 2][kSums][32];
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
      for (int at = warp; at < tile.count; at += kAdapterWarps)
        for (int j = lane; j < p.rank; j += 32)
          p.low[int64_t(__ldg(p.route.rows + tile.begin + at)) * p.rank + j] = 0.0f;
    return;
  }
  int64_t row[kTiles][2];
  const uint16_t* from[kTiles][2];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (row_warp * kTiles + m) * 16 + i * 8 + g;
      row[m][i] = at < tile.count ? __ldg(p.route.rows + tile.begin + at) : -1;
      from[m][i] = p.x + (row[m][i] < 0 ? 0 : row[m][i]) * p.ldx + 8 * t;
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
  const int first = 32 * kColWarps * part, step = 32 * kColWarps * parts;
  const int turns = first < p.cols ? (p.cols - first + step - 1) / step : 0;
  S stages(shared);
  auto x_of = [&](int turn) {
    return [&, c = first + turn * step + 32 * col_warp](int v, int& n) {
      n = row[v >> 1][v & 1] < 0 ? 0 : values_at(c + 8 * t, p.cols);
      return from[v >> 1][v & 1] + c;
    };
  };
  const WeightStage<kRankTiles, Shape::kSpans, !kAlong, Shape::kAlone, kWAligned> weight(w, 32, p.cols, p.rank);
  auto copy_w = [&](int turn) {
    if (turn < turns && !(Shape::kAlone && idle))
      weight.copy(stages.shared_filling(), first + turn * step + (Shape::kAlone ? 32 * col_warp : 0));
  };
#pragma unroll
  for (int i = 0; i < S::kCount - 1; ++i) {
    copy_w(i);
    stages.copy(x_of(i));
    stages.filled();
  }
  for (int turn = 0; turn < turns; ++turn, stages.next()) {
    stages.wait();
    uint4 x[2 * kTiles];
    stages.take(x, x_of(turn));
    copy_w(turn + S::kCount - 1);
    stages.copy(x_of(turn + S::kCount - 1));
    stages.filled();
    if (idle) continue;
    const uint4* const ws = stages.shared_due() + (Shape::kAlone ? 0 : col_warp * kRankTiles * 32);
    if constexpr (kAlong) {
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j) {
        const uint4 b = ws[(8 * j + g) * 4 + t];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
            mma_bf16(acc[m][j], word(x[2 * m], 2 * s), word(x[2 * m + 1], 2 * s),
                     word(x[2 * m], 2 * s + 1), word(x[2 * m + 1], 2 * s + 1), word(b, 2 * s),
                     word(b, 2 * s + 1));
      }
    } else {
      // Row k of a product's tile is column 8 (k / 2) + 4 s + k % 2 of the 32, and two
      // more in its second half: the order in which a lane holds x.
      const int of = lane >> 3, place = 8 * (of & 1) + (lane & 7);
      if constexpr (kRankTiles == 1) {  // both steps of the one rank tile
        uint32_t b[4];
        load_tiles<true>(b, ws + place_vector<1>(place + 16 * (of >> 1), 0));
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
            mma_bf16(acc[m][0], word(x[2 * m], 2 * s), word(x[2 * m + 1], 2 * s),
                     word(x[2 * m], 2 * s + 1), word(x[2 * m + 1], 2 * s + 1), b[2 * s], b[2 * s + 1]);
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < kRankTiles; j += 2) {
            uint32_t b[4];
            load_tiles<true>(b, ws + place_vector<kRankTiles>(place + 16 * s, j + (of >> 1)));
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int m = 0; m < kTiles; ++m)
                mma_bf16(acc[m][j + e], word(x[2 * m], 2 * s), word(x[2 * m + 1], 2 * s),
                         word(x[2 * m], 2 * s + 1), word(x[2 * m + 1], 2 * s + 1), b[2 * e], b[2 * e + 1]);
          }
      }
    }
  }
  copies_wait<0>();
  float* const mine = &acc[0][0][0];
  // Sums of the warps of the same rows: the upper half's to shared memory, added
  // by the lower.
#pragma unroll
  for (int half = kAdapterWarps / 2; half >= kRowWarps; half >>= 1) {
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
  if (parts == 1) {
    if (warp >= kRowWarps) return;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t to = row[m][i >> 1];
          const int rank = 8 * j + 2 * t + (i & 1);
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
  const int each = (kRowWarps * kSums + parts - 1) / parts;  // numbers of a lane
  const int last = min((part + 1) * each, kRowWarps * kSums);
  for (int k = part * each + warp; k < last; k += kAdapterWarps) {
    const int of = k / kSums, m = k % kSums / (4 * kRankTiles), j = k / 4 % kRankTiles, i = k % 4;
    const uint32_t at = smem_addr(&sums[of][k % kSums][lane]);
    float sum = 0.0f;
#pragma unroll 8
    for (int cta = 0; cta < parts; ++cta) sum += __uint_as_float(ld_shared_cluster_u32(map_to_cta(at, cta)));
    const int which = (of * kTiles + m) * 16 + 8 * (i >> 1) + g, rank = 8 * j + 2 * t + (i & 1);
    if (which < tile.count && rank < p.rank)
      p.low[int64_t(__ldg(p.route.rows + tile.begin + which)) * p.rank + rank] = scale * sum;
  }
  cluster_sync_all();
}

}  // namespace

cudaError_t launch_adapter_low(const AdapterArgs& a, bool backward, const uint16_t* x, int64_t ldx,
                               float* low, const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("adapter_low_kernel");
  LowArgs p = {};
  p.x = x;
  p.ldx = ldx;
  p.w = backward ? a.b : a.a;
  p.scale = backward ? a.scale : nullptr;
  p.low = low;
  p.cols = static_cast<int>(backward ? a.n : a.k);
  p.rank = a.rank;
  p.route = route_of(a);
  const bool aligned = rows_aligned(x, ldx, p.cols), w_aligned = backward ? b_aligned(a) : a_aligned(a);
  return with_rank_tiles(a.rank, [&](auto ranks) {
    constexpr int kRankTiles = decltype(ranks)::value;
    auto run = [&](auto tiles, auto row_warps) {
      constexpr int kTiles = decltype(tiles)::value, kRowWarps = decltype(row_warps)::value;
      const int64_t most = most_tiles(a.rows, a.count + 1, 16 * kTiles * kRowWarps);
      // One wave of two CTAs an SM, as far as the rows have tiles (a CTA spends 8 us
      // on finding its rows and on the sums), and a turn of all its warps at least.
      constexpr int kTurn = 32 * kAdapterWarps / kRowWarps;
      p.parts = 1;
      while (p.parts < 8 && most * p.parts * 2 <= 2 * dev.num_sms && kTurn * 2 * p.parts <= p.cols) p.parts *= 2;
      const dim3 grid(static_cast<unsigned>(most * p.parts));
      auto go = [&](auto along, auto whole, auto w_whole) {
        constexpr bool kAligned = decltype(whole)::value;
        return launch_staged<adapter_low_kernel<kTiles, kRankTiles, kRowWarps, decltype(along)::value, kAligned,
                                                decltype(w_whole)::value>>(
            grid, LowShape<kTiles, kRankTiles, kRowWarps, kAligned>::S::kBytes, dev, stream, p.parts, p);
      };
      if (!w_aligned) return backward ? go(No(), No(), No()) : go(Yes(), No(), No());
      if (backward) return aligned ? go(No(), Yes(), Yes()) : go(No(), No(), Yes());
      return aligned ? go(Yes(), Yes(), Yes()) : go(Yes(), No(), Yes());
    };
    // Tiles of 64 rows read w once for all, tiles of 16 waste fewer rows: 8192 x 4096 x
    // 4096 with rank 64 and 4 adapters takes 78 us in all with the former and 88 with
    // the latter, 2048 rows of 32 adapters 47 and 46 (rank 16: 30 and 27).
    if (a.rows < 128 * a.count) return run(Int<1>(), Int<1>());
    return run(Int<kRankTiles <= 4 ? 2 : 1>(), Int<kRankTiles <= 4 ? 2 : 4>());
  });
}

}  // namespace fp8lin
