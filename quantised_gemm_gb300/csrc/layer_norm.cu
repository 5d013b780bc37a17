// layer_norm.cu -- layer norm of bf16 rows, with an optional residual before
// it, and its backward pass:
//   h = bf16(x + r) (r given) or x;  mu = mean(h), rstd = 1 / sqrt(mean((h - mu)^2) + eps)
//   y = bf16((h - mu) rstd w + b)
//   xhat = (h - mu) rstd, g = dy w
//   dx = bf16(rstd (g - mean(g) - xhat mean(g xhat)) + dres)
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Bound by memory: each tensor is read or written once.  A group of threads
// holds a row in registers, eight consecutive values a vector, so the second
// look at the values (the deviations; the backward's dx) costs no second read,
// and the variance is the mean of squared deviations, not a difference of
// large sums.  Statistics and column sums are fp32; y, h and dx are rounded
// once.  In the backward a thread owns the same columns of every row that its
// CTA takes and keeps their sums in registers; a CTA writes one row of partial
// sums, and a second launch adds those in a fixed order.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "rows.cuh"

namespace fp8lin {
namespace {

constexpr int kGroupWarps = 4;  // rows a CTA takes at a time where a warp has one

// kThreads threads a row; a CTA of one such group, or of kGroupWarps warps
// with a row each.
template <int kThreads>
struct Group {
  static constexpr int kRows = kThreads == 32 ? kGroupWarps : 1;
  static constexpr int kBlock = kThreads * kRows;
};

// The sums of v and u over the group's threads, in every thread.  turn: a
// number that differs from the last call's (two sets of words take turns, so
// one barrier is enough).
template <int kThreads, bool kTwo>
__device__ __forceinline__ void group_sum(float& v, float& u, int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (kTwo) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  }
  if constexpr (kThreads > 32) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float words[2][2][kWarps];
    if ((threadIdx.x & 31) == 0) {
      words[turn & 1][0][threadIdx.x >> 5] = v;
      if (kTwo) words[turn & 1][1][threadIdx.x >> 5] = u;
    }
    __syncthreads();
    v = u = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      v += words[turn & 1][0][i];
      if (kTwo) u += words[turn & 1][1][i];
    }
  }
}

// The CTA's largest magnitude (fp32 bits) to *out, through the self-cleaning
// words acc and ticket.
__device__ __forceinline__ void record_max(uint32_t bits, uint32_t* acc, uint32_t* ticket,
                                           uint32_t* out) {
  __shared__ uint32_t most;
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if ((threadIdx.x & 31) == 0) atomicMax(&most, bits);
  __syncthreads();
  if (threadIdx.x == 0) {
    atomicMax(acc, most);
    __threadfence();
    if (atomicAdd(ticket, 1u) == gridDim.x - 1u) {
      __threadfence();
      *out = atomicExch(acc, 0u);
      atomicExch(ticket, 0u);
    }
  }
}

// The largest magnitude of eight bf16 values, as bf16 bits.
__device__ __forceinline__ uint32_t max_bits(const uint4& u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                              __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu);
}

struct NormParams {
  const uint16_t *x, *r;
  uint16_t *h, *y;
  const void *w, *b;  // b may be null
  float* stats;       // null, or means and then inverse deviations
  int64_t ldx, ldr, ldh, ldy, rows;
  int cols;
  float eps, inv_cols;
  uint32_t *amax, *acc, *ticket;  // amax null: not wanted
};

template <int kThreads, int kVecs, bool kAligned, bool kResidual, typename P>
__global__ void __launch_bounds__(Group<kThreads>::kBlock)
    layer_norm_kernel(const __grid_constant__ NormParams p) {
  using G = Group<kThreads>;
  griddep_wait();
  griddep_launch_dependents();
  const int t = G::kRows > 1 ? static_cast<int>(threadIdx.x & 31u) : static_cast<int>(threadIdx.x);
  const int group = G::kRows > 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  uint32_t most = 0;
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * G::kRows + group; row < p.rows;
       row += int64_t(gridDim.x) * G::kRows) {
    uint4 v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kThreads + t) * 8;
      v[k] = load_values<kAligned>(p.x + row * p.ldx + c, values_at(c, p.cols));
    }
    if constexpr (kResidual) {
      uint4 u[kVecs];
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        u[k] = load_values<kAligned>(p.r + row * p.ldr + c, values_at(c, p.cols));
      }
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        float a[8], b[8];
        bf16x8_to_f32(v[k], a);
        bf16x8_to_f32(u[k], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        v[k] = f32_to_bf16x8(a);
        store_values<kAligned>(p.h + row * p.ldh + c, v[k], values_at(c, p.cols));
      }
    }
    float sum = 0.0f, none = 0.0f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float a[8];
      bf16x8_to_f32(v[k], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += a[j];
    }
    group_sum<kThreads, false>(sum, none, turn++);
    const float mean = sum * p.inv_cols;
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int n = values_at((k * kThreads + t) * 8, p.cols);
      float a[8];
      bf16x8_to_f32(v[k], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = a[j] - mean;
        if (j < n) sq = fmaf(d, d, sq);
      }
    }
    group_sum<kThreads, false>(sq, none, turn++);
    const float rstd = __frsqrt_rn(sq * p.inv_cols + p.eps);
    if (p.stats != nullptr && t == 0) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kThreads + t) * 8;
      const int n = values_at(c, p.cols);
      float a[8], w[8], b[8];
      bf16x8_to_f32(v[k], a);
      load_params(static_cast<const P*>(p.w) + c, n, w);
      if (p.b != nullptr) {
        load_params(static_cast<const P*>(p.b) + c, n, b);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = fmaf((a[j] - mean) * rstd, w[j], b[j]);
      const uint4 y = f32_to_bf16x8(a);
      store_values<kAligned>(p.y + row * p.ldy + c, y, n);
      if (p.amax != nullptr) most = max(most, max_bits(first_values(y, n)));
    }
  }
  if (p.amax != nullptr) record_max(most << 16, p.acc, p.ticket, p.amax);
}

struct NormBackwardParams {
  const uint16_t *dy, *x, *dres;
  uint16_t* dx;  // null: not wanted
  const void* w;
  const float* stats;
  float* partials;  // a group's sums: cols of dw, then cols of db
  int64_t lddy, ldx, lddres, lddx, rows;
  int cols;
  float inv_cols;
  uint32_t *amax, *acc, *ticket;
};

template <int kThreads, int kVecs, bool kAligned, bool kResidual, typename P>
__global__ void __launch_bounds__(Group<kThreads>::kBlock)
    layer_norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  using G = Group<kThreads>;
  griddep_wait();
  griddep_launch_dependents();
  const int t = G::kRows > 1 ? static_cast<int>(threadIdx.x & 31u) : static_cast<int>(threadIdx.x);
  const int64_t group = int64_t(blockIdx.x) * G::kRows + (G::kRows > 1 ? threadIdx.x >> 5 : 0);
  const int64_t step = int64_t(gridDim.x) * G::kRows;
  float dw[kVecs][8], db[kVecs][8];
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.0f;
  uint32_t most = 0;
  int turn = 0;
  uint4 x[kVecs], dy[kVecs], dr[kVecs];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kThreads + t) * 8;
      const int n = values_at(c, p.cols);
      x[k] = load_values<kAligned>(p.x + row * p.ldx + c, n);
      dy[k] = load_values<kAligned>(p.dy + row * p.lddy + c, n);
      if (kResidual) dr[k] = load_values<kAligned>(p.dres + row * p.lddres + c, n);
    }
    mean = p.stats[row];
    rstd = p.stats[p.rows + row];
  };
  if (group < p.rows) load(group);
  for (int64_t row = group; row < p.rows; row += step) {
    float s1 = 0.0f, s2 = 0.0f;
    float g[kVecs][8], xhat[kVecs][8];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kThreads + t) * 8;
      const int n = values_at(c, p.cols);
      float w[8], a[8];
      load_params(static_cast<const P*>(p.w) + c, n, w);
      bf16x8_to_f32(x[k], xhat[k]);
      bf16x8_to_f32(dy[k], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xhat[k][j] = (xhat[k][j] - mean) * rstd;
        g[k][j] = a[j] * w[j];
        if (j < n) {
          dw[k][j] = fmaf(a[j], xhat[k][j], dw[k][j]);
          db[k][j] += a[j];
          s1 += g[k][j];
          s2 = fmaf(g[k][j], xhat[k][j], s2);
        }
      }
    }
    const float scale = rstd;
    uint4 res[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (kResidual) res[k] = dr[k];
    if (row + step < p.rows) load(row + step);
    group_sum<kThreads, true>(s1, s2, turn++);
    s1 *= p.inv_cols;
    s2 *= p.inv_cols;
    if (p.dx != nullptr) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        const int n = values_at(c, p.cols);
        float a[8], b[8];
        if constexpr (kResidual) bf16x8_to_f32(res[k], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = g[k][j] - s1 - xhat[k][j] * s2;
          a[j] = kResidual ? fmaf(a[j], scale, b[j]) : a[j] * scale;
        }
        const uint4 out = f32_to_bf16x8(a);
        store_values<kAligned>(p.dx + row * p.lddx + c, out, n);
        if (p.amax != nullptr) most = max(most, max_bits(first_values(out, n)));
      }
    }
  }
  if (p.partials != nullptr) {
    float* to = p.partials + group * 2 * p.cols;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = (k * kThreads + t) * 8 + j;
        if (c < p.cols) {
          to[c] = dw[k][j];
          to[p.cols + c] = db[k][j];
        }
      }
    }
  }
  if (p.amax != nullptr) record_max(most << 16, p.acc, p.ticket, p.amax);
}

// Column sums of `groups` rows of partial sums: 32 columns a CTA, its warps
// each every kSumWarps-th row.
constexpr int kSumWarps = 16;

template <typename P>
__global__ void __launch_bounds__(32 * kSumWarps)
    layer_norm_sum_kernel(const float* partials, int groups, int cols, P* dw, P* db) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;  // of dw and db together
  float sum = 0.0f;
  if (c < 2 * cols) {
#pragma unroll 4
    for (int g = warp; g < groups; g += kSumWarps) sum += partials[int64_t(g) * 2 * cols + c];
  }
  __shared__ float part[kSumWarps][33];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= 2 * cols) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) sum += part[i][lane];
  P* to = c < cols ? dw : db;
  if (to == nullptr) return;
  if constexpr (sizeof(P) == 2)
    to[c < cols ? c : c - cols] = static_cast<uint16_t>(cvt_bf16x2(sum, 0.0f) & 0xFFFFu);
  else
    to[c < cols ? c : c - cols] = sum;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether all of a tensor's vectors are aligned; a null tensor's are.
bool rows_aligned(const void* p, int64_t ld) { return p == nullptr || (aligned16(p) && ld % 8 == 0); }

// Threads a row and vectors a thread.
template <int kThreads, int kVecs>
struct Shape {
  static constexpr int threads = kThreads, vecs = kVecs;
};

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("layer_norm_kernel");
  NormParams p = {};
  p.x = a.x;
  p.r = a.r;
  p.h = a.h;
  p.y = a.y;
  p.w = a.w;
  p.b = a.b;
  p.stats = a.stats;
  p.ldx = a.ldx;
  p.ldr = a.ldr;
  p.ldh = a.ldh;
  p.ldy = a.ldy;
  p.rows = a.rows;
  p.cols = static_cast<int>(a.cols);
  p.eps = a.eps;
  p.inv_cols = 1.0f / static_cast<float>(a.cols);
  p.amax = a.amax;
  p.acc = a.acc;
  p.ticket = a.ticket;
  const bool aligned = a.cols % 8 == 0 && rows_aligned(a.x, a.ldx) && rows_aligned(a.r, a.ldr) &&
                       rows_aligned(a.h, a.ldh) && rows_aligned(a.y, a.ldy);
  auto run = [&](auto shape) {
    using S = decltype(shape);
    using G = Group<S::threads>;
    const int64_t want = (a.rows + G::kRows - 1) / G::kRows;
    const int64_t most = int64_t(dev.num_sms) * (2048 / G::kBlock);
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    auto go = [&](auto* kernel) {
      return launch_kernel(kernel, grid, dim3(G::kBlock), 0, stream, 1, false, p);
    };
    auto pick = [&](auto flag) {
      constexpr bool kAligned = decltype(flag)::value;
      if (a.param_f32)
        return a.r != nullptr ? go(layer_norm_kernel<S::threads, S::vecs, kAligned, true, float>)
                              : go(layer_norm_kernel<S::threads, S::vecs, kAligned, false, float>);
      return a.r != nullptr ? go(layer_norm_kernel<S::threads, S::vecs, kAligned, true, uint16_t>)
                            : go(layer_norm_kernel<S::threads, S::vecs, kAligned, false, uint16_t>);
    };
    return aligned ? pick(std::true_type()) : pick(std::false_type());
  };
  if (a.cols <= 256) return run(Shape<32, 1>());
  if (a.cols <= 512) return run(Shape<32, 2>());
  if (a.cols <= 1024) return run(Shape<128, 1>());
  if (a.cols <= 2048) return run(Shape<128, 2>());
  if (a.cols <= 4096) return run(Shape<256, 2>());
  if (a.cols <= 8192) return run(Shape<512, 2>());
  return run(Shape<1024, 2>());
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, const DeviceInfo& dev,
                                       cudaStream_t stream, int* launches) {
  set_error_site("layer_norm_backward_kernel");
  NormBackwardParams p = {};
  p.dy = a.dy;
  p.x = a.x;
  p.dres = a.dres;
  p.dx = a.dx;
  p.w = a.w;
  p.stats = a.stats;
  p.lddy = a.lddy;
  p.ldx = a.ldx;
  p.lddres = a.lddres;
  p.lddx = a.lddx;
  p.rows = a.rows;
  p.cols = static_cast<int>(a.cols);
  p.inv_cols = 1.0f / static_cast<float>(a.cols);
  p.amax = a.amax;
  p.acc = a.acc;
  p.ticket = a.ticket;
  const bool sums = a.dw != nullptr || a.db != nullptr;
  const bool aligned = a.cols % 8 == 0 && rows_aligned(a.x, a.ldx) && rows_aligned(a.dy, a.lddy) &&
                       rows_aligned(a.dres, a.lddres) && rows_aligned(a.dx, a.lddx);
  int groups = 0;
  auto run = [&](auto shape) {
    using S = decltype(shape);
    using G = Group<S::threads>;
    const int64_t want = (a.rows + G::kRows - 1) / G::kRows;
    int64_t most = int64_t(dev.num_sms) * (1024 / G::kBlock);
    if (sums) {
      const int64_t room = static_cast<int64_t>(a.ws_bytes / (sizeof(float) * 2 * a.cols)) / G::kRows;
      if (room < most) most = room;
    }
    if (most < 1) return cudaErrorInvalidValue;  // the caller has checked that one fits
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    groups = static_cast<int>(grid.x) * G::kRows;
    p.partials = sums ? a.ws : nullptr;
    auto go = [&](auto* kernel) {
      return launch_kernel(kernel, grid, dim3(G::kBlock), 0, stream, 1, false, p);
    };
    auto pick = [&](auto flag) {
      constexpr bool kAligned = decltype(flag)::value;
      if (a.param_f32)
        return a.dres != nullptr
                   ? go(layer_norm_backward_kernel<S::threads, S::vecs, kAligned, true, float>)
                   : go(layer_norm_backward_kernel<S::threads, S::vecs, kAligned, false, float>);
      return a.dres != nullptr
                 ? go(layer_norm_backward_kernel<S::threads, S::vecs, kAligned, true, uint16_t>)
                 : go(layer_norm_backward_kernel<S::threads, S::vecs, kAligned, false, uint16_t>);
    };
    return aligned ? pick(std::true_type()) : pick(std::false_type());
  };
  cudaError_t e;
  if (a.cols <= 256) e = run(Shape<32, 1>());
  else if (a.cols <= 512) e = run(Shape<32, 2>());
  else if (a.cols <= 1024) e = run(Shape<128, 1>());
  else if (a.cols <= 2048) e = run(Shape<256, 1>());
  else if (a.cols <= 4096) e = run(Shape<512, 1>());
  else if (a.cols <= 8192) e = run(Shape<512, 2>());
  else e = run(Shape<1024, 2>());
  *launches = 1;
  if (e != cudaSuccess || !sums) return e;
  *launches = 2;
  set_error_site("layer_norm_sum_kernel");
  const int cols = static_cast<int>(a.cols);
  const dim3 grid(static_cast<unsigned>((2 * cols + 31) / 32)), block(32 * kSumWarps);
  const float* partials = a.ws;
  if (a.param_f32)
    return launch_kernel(layer_norm_sum_kernel<float>, grid, block, 0, stream, 1, false, partials,
                         groups, cols, static_cast<float*>(a.dw), static_cast<float*>(a.db));
  return launch_kernel(layer_norm_sum_kernel<uint16_t>, grid, block, 0, stream, 1, false, partials,
                       groups, cols, static_cast<uint16_t*>(a.dw), static_cast<uint16_t*>(a.db));
}

}  // namespace fp8lin
