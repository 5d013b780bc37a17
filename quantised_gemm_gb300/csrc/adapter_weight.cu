// adapter_weight.cu -- the gradients of the adapters' weights:
//   dw[c][j] = sum over the rows i of one adapter of x[i][c] s_a low[i][j]
// dB (x = dy, low = h) and dA (x the input, low = dh) in one launch.
//
// Bound by reading x again: 16384 rows of 14336 and 4096 columns with rank 16 take
// 118 us (5.2 TB/s).  A cluster shares the rows of a large adapter; partial sums in
// the workspace and a launch that adds them took 11 us more, and 153 more for 8192 x 4096
// x 4096 with rank 128.
#include "adapter_kernels.cuh"

namespace fp8lin {
namespace {

// A slab of columns of one adapter's gradient, by a CTA or by a cluster of them that
// share the adapter's rows.  The CTA's warps take blocks of 16 rows side by side
// (kRowWarps of them) and columns side by side (the others); their sums meet in
// shared memory, and those of a cluster's CTAs in distributed shared memory.
struct WeightArgs {
  const uint16_t* x;
  int64_t ldx;
  const float* low;
  const float* scale;  // null: 1
  uint16_t* dw;
  int cols, rank, slabs;
  const uint4* packed;  // low as adapter_pack_kernel left it, or null
  bool along;    // dw is [cols, r] (dB), else [r, cols] (dA)
  bool aligned;  // x's rows
};

// With a small rank the rows' numbers are few beside x, and splitting the rows leaves
// fewer CTAs to a cluster; with a large one warps of the same rows share them.  Rank 64
// with all warps on the same rows took 14 us more for the backward of 608 x 793 x 777 (45
// us), where a turn's latency counts, and 3 more for 4096 x 4096 x 4096 (125).
template <int kRankTiles>
struct WeightShape {
  static constexpr int kRowWarps = kRankTiles <= 2 ? 4 : kRankTiles <= 8 ? 2 : 1;
  static constexpr int kColWarps = kAdapterWarps / kRowWarps;
  static constexpr int kChunks = kRankTiles <= 4 ? 2 : 1;  // of 32 columns a warp
  static constexpr int kSlab = 32 * kChunks * kColWarps;
  static constexpr int kSums = 2 * kChunks * kRankTiles * 4;  // a lane's
  static constexpr int kCtaSums = kRowWarps > 1 ? kSums : 1;  // that warps of a CTA add up
  static constexpr bool kAlone = kRankTiles <= 2;  // each warp has its own low operands
  static constexpr int kShared = (kAlone ? 1 : kRowWarps) * kRankTiles * 32;  // of a turn
  template <bool kAligned>
  // More stages than 80 KB hold cost a short sum more than they give a long one.
  using T = Stages<stages_in(kAlone || kRankTiles == 8 ? kStageRoom - 16 * 1024 : kRankTiles == 4 ? kStageRoom - 32 * 1024 : kStageRoom,
                             sizeof(uint4) * ((kAligned ? 2 : 4) * kChunks * kAdapterThreads +
                                              (kAlone ? kAdapterWarps : 1) * kShared)),
                   2 * kChunks, kShared, kAlone, kAligned, true>;
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
                                            int part, int parts,
                                            float (*sums)[WeightShape<kRankTiles>::kCtaSums][32],
                                            uint4* shared) {
  using S = WeightShape<kRankTiles>;
  constexpr int kChunks = S::kChunks, kSums = S::kSums;
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int col_warp = warp % S::kColWarps, row_warp = warp / S::kColWarps;
  const int g = lane >> 2, t = lane & 3;
  const RowTile tile = group_part(route, block / p.slabs, part, parts);
  const int slab0 = block % p.slabs * S::kSlab, col0 = slab0 + col_warp * 32 * kChunks;
  const float scale = p.scale != nullptr ? __ldg(p.scale + tile.group) : 1.0f;
  float acc[2 * kChunks][kRankTiles][4];
#pragma unroll
  for (int m = 0; m < 2 * kChunks; ++m)
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
  const int32_t* const rows = route.rows + tile.begin;
  // x and the low operands are on their way, and for two turns more the row numbers.
  constexpr int kStep = 16 * S::kRowWarps;
  const int turns = (tile.count + kStep - 1) / kStep;
  using T = typename S::template T<kAligned>;
  T stages(shared);
  constexpr int kBefore = T::kCount - 1;
  int n_of[kChunks];  // values of the lane's columns
#pragma unroll
  for (int c = 0; c < kChunks; ++c) n_of[c] = values_at(col0 + 32 * c + 8 * t, p.cols);
  const uint16_t* const column = p.x + (n_of[0] > 0 ? col0 + 8 * t : 0);
  auto find = [&](int (&to)[2], int turn) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int of = turn * kStep + 16 * row_warp + 8 * i + g;
      to[i] = of < tile.count ? __ldg(rows + of) : -1;
    }
  };
  auto x_of = [&](const int (&of)[2]) {
    const uint16_t* const at[2] = {column + max(of[0], 0) * p.ldx, column + max(of[1], 0) * p.ldx};
    const bool on[2] = {of[0] >= 0, of[1] >= 0};
    return [=, &n_of](int v, int& n) {
      n = on[v & 1] ? n_of[v >> 1] : 0;
      return at[v & 1] + 32 * (v >> 1);
    };
  };
  constexpr int kThreads = S::kAlone ? 32 : kAdapterThreads, kBlock = kRankTiles * 32;
  const int me = static_cast<int>(threadIdx.x) % kThreads;
  const uint4* packed = p.packed == nullptr
                            ? nullptr
                            : p.packed + int64_t(tile.block + (S::kAlone ? row_warp : 0)) * kBlock + me;
  int next_low = 0;  // the first row of the turn that copy_low() is for
  auto copy_low = [&]() {
    uint4* const to = stages.shared_filling() + me;
#pragma unroll
    for (int i0 = 0; i0 < S::kShared; i0 += kThreads) {
      if (S::kShared % kThreads != 0 && i0 + me >= S::kShared) break;
      const int i = i0 + me;
      const int r = next_low + 16 * (S::kAlone ? row_warp : i / kBlock);  // the block's first row
      if (packed != nullptr) {
        copy16(to + i0, packed + i0, r < tile.count);
        continue;
      }
      const int j = i / 32 % kRankTiles;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int of = r + 2 * (i & 3) + (e & 1) + 8 * (e >> 1), rank = 8 * j + (i >> 2 & 7);
        v[e] = of < tile.count && rank < p.rank
                   ? scale * __ldg(p.low + int64_t(__ldg(rows + of)) * p.rank + rank)
                   : 0.0f;
      }
      to[i0] = low_operand(v[0], v[1], v[2], v[3]);
    }
    next_low += kStep;
    if (packed != nullptr) packed += S::kRowWarps * kBlock;
  };
  int numbers[kBefore + 2][2];
#pragma unroll
  for (int i = 0; i < kBefore + 2; ++i) find(numbers[i], i);
#pragma unroll
  for (int i = 0; i < kBefore; ++i) {
    stages.copy(x_of(numbers[i]));
    copy_low();
    stages.filled();
  }
  int number[2] = {numbers[kBefore][0], numbers[kBefore][1]};
  int later[2] = {numbers[kBefore + 1][0], numbers[kBefore + 1][1]};
  for (int turn = 0; turn < turns; ++turn, stages.next()) {
    stages.wait();
    if constexpr (!kAligned) {
      uint4 x[2 * kChunks];
      int due[2];
      find(due, turn);
      stages.take(x, x_of(due));
      stages.put_back(x);
    }
    uint32_t a[2 * kChunks][4];  // 16 columns and 16 rows each
#pragma unroll
    for (int m = 0; m < 2 * kChunks; ++m) stages.turned(a[m], m & ~1, 2 * (m & 1));
    copy_low();
    stages.copy(x_of(number));
    stages.filled();
#pragma unroll
    for (int i = 0; i < 2; ++i) number[i] = later[i];
    find(later, turn + kBefore + 2);
    const uint4* const operand = stages.shared_due() + (S::kAlone ? 0 : row_warp * kRankTiles * 32) + lane;
#pragma unroll
    for (int j = 0; j < kRankTiles; ++j) {
      const uint4 low = operand[32 * j];
#pragma unroll
      for (int m = 0; m < 2 * kChunks; ++m) {
        mma_bf16(acc[m][j], a[m][0], a[m][1], a[m][2], a[m][3], low.z, low.w);
        mma_bf16(acc[m][j], a[m][0], a[m][1], a[m][2], a[m][3], low.x, low.y);
      }
    }
  }
  copies_wait<0>();
  if constexpr (S::kRowWarps > 1) {
    float* const mine = &acc[0][0][0];
#pragma unroll
    for (int half = kAdapterWarps / 2; half >= S::kColWarps; half >>= 1) {
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
  uint16_t* const dw = p.dw + tile.group * (int64_t(p.cols) * p.rank);
  // Number i of a lane of col_warp: product (m, j) has columns 16 m + g and 16 m + g + 8
  // of ranks 8 j + 2 t and the next.
  auto put = [&](int of_warp, int i, float v) {
    const int m = i / (4 * kRankTiles), j = i / 4 % kRankTiles, e = i % 4;
    const int col = slab0 + of_warp * 32 * kChunks + 16 * m + 8 * (e >> 1) + g, rank = 8 * j + 2 * t + (e & 1);
    if (col >= p.cols || rank >= p.rank) return;
    dw[p.along ? int64_t(col) * p.rank + rank : int64_t(rank) * p.cols + col] =
        static_cast<uint16_t>(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
  };
  if (parts == 1) {
    if (row_warp != 0) return;
#pragma unroll
    for (int m = 0; m < 2 * kChunks; ++m)
#pragma unroll
      for (int j = 0; j < kRankTiles; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) put(col_warp, (m * kRankTiles + j) * 4 + i, acc[m][j][i]);
    return;
  }
  // The cluster's sums: every CTA adds a part of the numbers, in the CTAs' order.
  __syncthreads();  // the stages are read
  float* const of_cta = reinterpret_cast<float*>(shared);
  if (row_warp == 0) {
    const float* const mine = &acc[0][0][0];
#pragma unroll
    for (int i = 0; i < kSums; ++i) of_cta[(col_warp * kSums + i) * 32 + lane] = mine[i];
  }
  cluster_sync_all();
  constexpr int kAll = S::kColWarps * kSums;
  const int each = (kAll + parts - 1) / parts, last = min((part + 1) * each, kAll);
  for (int k = part * each + warp; k < last; k += kAdapterWarps) {
    const uint32_t at = smem_addr(of_cta + k * 32 + lane);
    float sum = 0.0f;
#pragma unroll 8
    for (int cta = 0; cta < parts; ++cta) sum += __uint_as_float(ld_shared_cluster_u32(map_to_cta(at, cta)));
    put(k / kSums, k % kSums, sum);
  }
  cluster_sync_all();
}

// dB (blocks from 0 on) and dA (the others) in one launch; either may have none.
template <int kRankTiles>
__global__ void __launch_bounds__(kAdapterThreads, kRankTiles <= 8 ? 2 : 1)
    adapter_weight_kernel(const __grid_constant__ WeightArgs db, const __grid_constant__ WeightArgs da,
                          const Route route, int parts) {
  griddep_wait();
  griddep_launch_dependents();
  const int block = static_cast<int>(blockIdx.x) / parts, part = static_cast<int>(blockIdx.x) % parts;
  const int first = db.slabs * (route.groups - 1);
  const bool is_db = block < first;
  using S = WeightShape<kRankTiles>;
  extern __shared__ uint4 shared[];
  __shared__ float sums[S::kRowWarps > 1 ? kAdapterWarps / 2 : 1][S::kCtaSums][32];
  const WeightArgs& p = is_db ? db : da;
  if (p.aligned)
    weight_tile<kRankTiles, true>(p, route, is_db ? block : block - first, part, parts, sums, shared);
  else
    weight_tile<kRankTiles, false>(p, route, is_db ? block : block - first, part, parts, sums, shared);
}

}  // namespace

size_t adapter_packed_bytes(const AdapterArgs& a) {
  return static_cast<size_t>(most_tiles(a.rows, a.count, 16)) * rank_tiles(a.rank) * 32 * sizeof(uint4);
}

cudaError_t launch_adapter_pack(const AdapterArgs& a, const AdapterWeight& db, const AdapterWeight& da,
                                cudaStream_t stream) {
  set_error_site("adapter_pack_kernel");
  const int blocks = static_cast<int>(most_tiles(a.rows, a.count, 16));
  const PackArgs pa = {da.low, nullptr, static_cast<uint4*>(da.packed)};
  const PackArgs pb = {db.low, a.scale, static_cast<uint4*>(db.packed)};
  const int both = da.packed != nullptr ? 2 : 1;
  const dim3 grid(static_cast<unsigned>((both * int64_t(blocks) + kPackWarps - 1) / kPackWarps));
  return with_rank_tiles(a.rank, [&](auto ranks) {
    return launch_kernel(adapter_pack_kernel<decltype(ranks)::value>, grid, dim3(32 * kPackWarps), 0, stream,
                         1, false, pb, pa, route_of(a), a.rank, blocks);
  });
}

cudaError_t launch_adapter_weight(const AdapterArgs& a, const AdapterWeight& db, const AdapterWeight& da,
                                  const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("adapter_weight_kernel");
  return with_rank_tiles(a.rank, [&](auto ranks) {
    constexpr int kRankTiles = decltype(ranks)::value;
    using S = WeightShape<kRankTiles>;
    auto job = [&](const AdapterWeight& j, bool is_da) {
      WeightArgs p = {};
      if (j.dw == nullptr) return p;
      p.x = j.x;
      p.ldx = j.ldx;
      p.low = j.low;
      p.scale = is_da ? nullptr : a.scale;
      p.dw = j.dw;
      p.cols = static_cast<int>(is_da ? a.k : a.n);
      p.rank = a.rank;
      p.packed = static_cast<const uint4*>(j.packed);
      p.slabs = (p.cols + S::kSlab - 1) / S::kSlab;
      p.along = !is_da;
      p.aligned = rows_aligned(j.x, j.ldx, p.cols);
      return p;
    };
    const WeightArgs b = job(db, false), c = job(da, true);
    const int64_t slabs = (int64_t(b.slabs) + c.slabs) * a.count;
    // More CTAs than are resident, so that an adapter with many rows does not keep the
    // others waiting, but with enough rows each for their start and their sums.  The
    // whole backward with four CTAs an SM and with eight: 16384 x 4096 x 14336, rank
    // 16, 264 and 262 us; 4096 x 4096 x 4096, rank 64, 129 and 125.  With 128 rows and
    // with 256: 1267 x 1600 x 2501, rank 12 and four adapters, 33 and 36; 1024 x 4096 x
    // 4096 of one adapter, rank 64, 48 and 45 (rank 16: 31 and 27).
    const int64_t most = (a.rank <= 32 ? 4 : 8) * int64_t(dev.num_sms), least = a.rank <= 16 ? 128 : 256;
    int parts = 1;
    while (parts < 8 && slabs * parts * 2 <= most && a.rows >= least * 2 * parts * a.count) parts *= 2;
    const dim3 grid(static_cast<unsigned>(slabs * parts));
    constexpr size_t kA = S::template T<true>::kBytes, kB = S::template T<false>::kBytes;
    constexpr size_t kSum = sizeof(float) * 32 * S::kColWarps * S::kSums;
    constexpr size_t kStages = kA > kB ? kA : kB;
    return launch_staged<adapter_weight_kernel<kRankTiles>>(grid, kStages > kSum ? kStages : kSum, dev, stream, parts,
                                                            b, c, route_of(a), parts);
  });
}

}  // namespace fp8lin
