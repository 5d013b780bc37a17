// adapter.cu -- the low-rank adapters' rows sorted by adapter, and the one-launch
// forward of a few rows.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "adapter_kernels.cuh"
#include "internal.h"

namespace fp8lin {
namespace {

// ---------------------------------------------------------------- route

constexpr int kRouteWarps = 32, kRouteCluster = 8;

// The rows sorted by adapter, each adapter's in order: a counting sort by one CTA or
// by one cluster of them, of whose warps the w-th takes the w-th run of rows.
// Latency: two trips to L2, a few barriers and some 100 cycles for 32 rows of a warp.
template <bool kClustered>
__global__ void __launch_bounds__(32 * kRouteWarps)
    adapter_route_kernel(const int32_t* index, int rows, int count, int32_t* first, int32_t* sorted) {
  extern __shared__ int table[];  // [warp][group]: how many, then where the next one goes
  __shared__ int warp_total[kRouteWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int groups = count + 1, threads = static_cast<int>(blockDim.x), warps = threads / 32;
  constexpr int ctas = kClustered ? kRouteCluster : 1;
  const int cta = kClustered ? static_cast<int>(blockIdx.x) : 0;
  int* const totals = table + warps * groups;  // [cta][group] of a cluster
  for (int i = static_cast<int>(threadIdx.x); i < groups * warps; i += threads) table[i] = 0;
  __syncthreads();
  const int run = ((rows + warps * ctas - 1) / (warps * ctas) + 31) / 32 * 32;
  const int64_t begin = int64_t(cta * warps + warp) * run;
  int* const mine = table + warp * groups;
  // Eight loads of a lane are in flight together.
  constexpr int kLoads = 8;
  auto each = [&](auto fn) {
    for (int64_t i0 = begin; i0 < begin + run && i0 < rows; i0 += 32 * kLoads) {
      int a[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        a[j] = i < begin + run && i < rows ? __ldg(index + i) : 0;
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        const int g = i < begin + run && i < rows ? (a[j] >= 0 && a[j] < count ? a[j] : count) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, g);
        if (i0 + 32 * j < begin + run && i0 + 32 * j < rows) fn(i, g, same);
      }
    }
  };
  each([&](int64_t, int g, uint32_t same) {
    if (g >= 0 && __ffs(static_cast<int>(same)) - 1 == lane) mine[g] += __popc(same);
    __syncwarp();
  });
  __syncthreads();
  auto of_warps = [&](int g, int (&n)[kRouteWarps]) {
    int total = 0;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) {
      n[w] = w < warps && g < groups ? table[w * groups + g] : 0;
      total += n[w];
    }
    return total;
  };
  if constexpr (kClustered) {  // every CTA's numbers to all
    cluster_sync_all();
    for (int g = static_cast<int>(threadIdx.x); g < groups; g += threads) {
      int n[kRouteWarps];
      const int total = of_warps(g, n);
      const uint32_t at = smem_addr(totals + cta * groups + g);
      for (int to = 0; to < ctas; ++to) st_shared_cluster_u32(map_to_cta(at, to), static_cast<uint32_t>(total));
    }
    cluster_sync_all();
  }
  // Group by group, CTA by CTA, warp by warp: exclusive sums.
  int before = 0;
  for (int base = 0; base < groups; base += threads) {
    const int g = base + static_cast<int>(threadIdx.x);
    int n[kRouteWarps], ctas_before = 0;
    int total = of_warps(g, n);
    if constexpr (kClustered) {
      total = 0;
      for (int c = 0; c < ctas && g < groups; ++c) {
        if (c < cta) ctas_before += totals[c * groups + g];
        total += totals[c * groups + g];
      }
    }
    int up = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, up, o);
      if (lane >= o) up += a;
    }
    if (lane == 31) warp_total[warp] = up;
    __syncthreads();
    const int of_warp = lane < warps ? warp_total[lane] : 0;
    const int warps_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of_warp : 0);
    const int all = __reduce_add_sync(0xFFFFFFFFu, of_warp);
    int at = before + warps_before + up - total;
    if (g < groups) {
      if (cta == 0) {
        first[g] = at;
        if (g == groups - 1) first[groups] = rows;
      }
      at += ctas_before;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) {
        if (w < warps) table[w * groups + g] = at;
        at += n[w];
      }
    }
    before += all;
    __syncthreads();
  }
  each([&](int64_t i, int g, uint32_t same) {
    if (g >= 0) sorted[mine[g] + __popc(same & ((1u << lane) - 1u))] = static_cast<int32_t>(i);
    __syncwarp();
    if (g >= 0 && __ffs(static_cast<int>(same)) - 1 == lane) mine[g] += __popc(same);
    __syncwarp();
  });
}

// ---------------------------------------------------------------- a few rows

// One row a cluster: each CTA takes a part of K for the low product, the parts'
// sums go to every CTA of the cluster through distributed shared memory, and
// each CTA takes a part of N for the high product.  Bound by reading A and B
// once, and by latency: one launch.  32 x 4096 x 14336 with rank 16 and an adapter a
// row: 6.6 us (9.7 with B loaded after the low product), one row 5.0.
struct FewArgs {
  const uint16_t *x, *a, *b, *base;
  uint16_t* y;
  const float* scale;
  const int32_t* index;
  float* low;
  int64_t ldx, ldbase, ldy;
  int k, n, rank, count;
};
constexpr int kFewWarps = 16, kFewCluster = 8;
// Steps of B that a warp loads before it waits for the low product.
constexpr int few_ahead(int lanes) { return lanes <= 2 ? 8 : 4; }

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float sum) {
  float x[8], y[8];
  bf16x8_to_f32(a, x);
  bf16x8_to_f32(b, y);
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(x[j], y[j], sum);
  return sum;
}

// kLanes: lanes a column of B, eight ranks each.
template <int kLanes, bool kAligned>
__global__ void __launch_bounds__(32 * kFewWarps, 2)  // 32 rows are 256 CTAs, all resident
    adapter_few_kernel(const __grid_constant__ FewArgs p) {
  constexpr int kRanks = 8 * kLanes;
  __shared__ float sums[kFewCluster][kRanks];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int64_t row = blockIdx.x / kFewCluster;
  const int part = static_cast<int>(blockIdx.x) % kFewCluster;
  const int adapter = __ldg(p.index + row);
  const bool none = adapter < 0 || adapter >= p.count;
  // The columns of y that this CTA writes, and of x that it reads: multiples of 8.
  const int n_part = ((p.n + kFewCluster - 1) / kFewCluster + 7) / 8 * 8;
  const int n0 = part * n_part, n1 = min(n0 + n_part, p.n);
  const uint16_t* const base = p.base == nullptr ? nullptr : p.base + row * p.ldbase;
  uint16_t* const y = p.y + row * p.ldy;
  if (none) {
    if (part == 0)
      for (int j = static_cast<int>(threadIdx.x); j < p.rank; j += 32 * kFewWarps) p.low[row * p.rank + j] = 0.0f;
    if (y != base)
      for (int c = n0 + static_cast<int>(threadIdx.x); c < n1; c += 32 * kFewWarps)
        y[c] = base == nullptr ? uint16_t(0) : base[c];
    return;  // all CTAs of the cluster
  }
  cluster_arrive();  // this CTA has begun: its shared memory may be written
  const uint16_t* const a = p.a + int64_t(adapter) * p.rank * p.k;
  const uint16_t* const b = p.b + int64_t(adapter) * p.rank * p.n;
  const uint16_t* const x = p.x + row * p.ldx;
  const int k_part = ((p.k + kFewCluster - 1) / kFewCluster + 7) / 8 * 8;
  const int k0 = part * k_part, k1 = min(k0 + k_part, p.k);
  // B's first steps are on their way during the low product.
  constexpr int kCols = 32 / kLanes;  // columns a warp takes a step
  constexpr int kStep = kFewWarps * kCols;
  const int sub = lane % kLanes, at = lane / kLanes;
  const int ranks = min(max(p.rank - 8 * sub, 0), 8);
  auto load_b = [&](int c) {
    return load_values<kAligned>(b + int64_t(c) * p.rank + 8 * sub, c < n1 ? ranks : 0);
  };
  const int c0 = n0 + warp * kCols + at;
  constexpr int kAhead = few_ahead(kLanes);
  uint4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = load_b(c0 + i * kStep);
  // A warp's ranks together: x is read once, and all loads of a turn are in flight.
  constexpr int kPer = kRanks > kFewWarps ? kRanks / kFewWarps : 1;
  float part_sum[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) part_sum[i] = 0.0f;
  if (warp < p.rank) {
    for (int c = k0 + 8 * lane; c - 8 * lane < k1; c += 256) {
      const int n = values_at(c, k1);
      const uint4 v = load_values<kAligned>(x + c, n);
      uint4 w[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = warp + i * kFewWarps;
        w[i] = load_values<kAligned>(a + int64_t(j) * p.k + c, j < p.rank ? n : 0);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) part_sum[i] = dot8(v, w[i], part_sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part_sum[i] += __shfl_xor_sync(0xFFFFFFFFu, part_sum[i], o);
  }
  cluster_wait();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = warp + i * kFewWarps;
    if (j >= p.rank) part_sum[i] = 0.0f;  // an infinity in x times the 0 past the ranks is not
    if (lane < kFewCluster && j < kRanks)
      st_shared_cluster_u32(map_to_cta(smem_addr(&sums[part][j]), lane), __float_as_uint(part_sum[i]));
  }
  cluster_sync_all();
  float low[8];
  const float scale = __ldg(p.scale + adapter);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    low[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kFewCluster; ++i) low[j] += sums[i][8 * sub + j];
  }
  if (part == 0 && warp == 0 && at == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * sub + j < p.rank) p.low[row * p.rank + 8 * sub + j] = low[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) low[j] *= scale;
  auto column = [&](int c, const uint4& v) {
    float w[8], sum = 0.0f;
    bf16x8_to_f32(v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(low[j], w[j], sum);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (c < n1 && sub == 0) {
      if (base != nullptr) sum += bf16lo_to_f32(base[c]);
      y[c] = static_cast<uint16_t>(cvt_bf16x2(sum, 0.0f) & 0xFFFFu);
    }
  };
  for (int c = c0; c - at < n1; c += kAhead * kStep) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) column(c + i * kStep, ahead[i]);
    if (c - at + kAhead * kStep < n1) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ahead[i] = load_b(c + (i + kAhead) * kStep);
    }
  }
}

}  // namespace

cudaError_t launch_adapter_route(const int32_t* index, int64_t rows, int64_t count, int32_t* route,
                                 const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("adapter_route_kernel");
  // 32 rows a warp where there are few, a cluster where there are many (65536 rows of
  // 4 adapters: 8 us, by one CTA 29; 8192 rows 6 us either way).
  int64_t warps = (rows + 31) / 32;
  warps = warps < 4 ? 4 : warps > kRouteWarps ? kRouteWarps : warps;
  const bool clustered = rows > 8192;
  const int ctas = clustered ? kRouteCluster : 1;
  const size_t bytes = sizeof(int) * static_cast<size_t>((warps + ctas) * (count + 1));
  if (bytes > 40 * 1024) {
    static std::mutex mu;
    static bool done[64];
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev.device]) {
      const int most = static_cast<int>(sizeof(int) * (kRouteWarps + kRouteCluster) * (kAdapterMaxCount + 1));
      cudaError_t e = cudaFuncSetAttribute(adapter_route_kernel<false>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(adapter_route_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      done[dev.device] = true;
    }
  }
  return launch_kernel(clustered ? adapter_route_kernel<true> : adapter_route_kernel<false>,
                       dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(32 * warps)), bytes, stream,
                       ctas, false, index, static_cast<int>(rows), static_cast<int>(count), route,
                       route + count + 2);
}

bool adapter_few_fits(const AdapterArgs& a) {
  // Rows do not share what they read, and 32 of them fill the GPU once: 64 x 4096 x 4096
  // with 32 adapters takes 11 us so and 16 sorted at rank 16, 22 and 17 at rank 64.
  return a.rows <= 64 && a.rows * 8 * rank_tiles(a.rank) <= 2048;
}

cudaError_t launch_adapter_few(const AdapterArgs& a, const int32_t* index, const uint16_t* x, int64_t ldx,
                               const uint16_t* base, int64_t ldbase, uint16_t* y, int64_t ldy,
                               float* low, cudaStream_t stream) {
  set_error_site("adapter_few_kernel");
  FewArgs p = {};
  p.x = x;
  p.a = a.a;
  p.b = a.b;
  p.base = base;
  p.y = y;
  p.scale = a.scale;
  p.index = index;
  p.low = low;
  p.ldx = ldx;
  p.ldbase = ldbase;
  p.ldy = ldy;
  p.k = static_cast<int>(a.k);
  p.n = static_cast<int>(a.n);
  p.rank = a.rank;
  p.count = static_cast<int>(a.count);
  const bool aligned = rows_aligned(x, ldx, a.k) && a_aligned(a) && aligned16(a.b) && a.rank % 8 == 0;
  const dim3 grid(static_cast<unsigned>(a.rows) * kFewCluster), block(32 * kFewWarps);
  return with_rank_tiles(a.rank, [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value;
    return aligned ? launch_kernel(adapter_few_kernel<kLanes, true>, grid, block, 0, stream, kFewCluster, false, p)
                   : launch_kernel(adapter_few_kernel<kLanes, false>, grid, block, 0, stream, kFewCluster, false, p);
  });
}

}  // namespace fp8lin
