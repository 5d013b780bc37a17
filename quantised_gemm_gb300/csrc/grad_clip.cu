// grad_clip.cu -- the global 2-norm of a list of gradients and their scaling
// to a largest norm:
//   norm = sqrt(sum_t sum_i g_t[i]^2),  out_t[i] = g_t[i] * min(1, max_norm / (norm + eps)).
//
// Bound by memory: the norm reads every gradient once, the scaling reads and
// writes it once.  738 M fp32 values: 434 us and 899 us, 6.8 and 6.6 TB/s;
// 31 M bf16 values into fp32: 44 us together, of which 27 us is the traffic.
// The list travels in the kernel's parameters (no table on the device, so the
// calls can be captured and the tensors may move from call to call).  It is
// cut into chunks, and each CTA takes a run of them, so all CTAs read alike
// whatever the tensors' sizes.  The scaling walks its runs from their ends,
// where the norm stopped, and adds up the norm's partial sums itself where
// one launch made them all (a last CTA that does it costs 4 us more).
// Squares are added in fp32 over kUnroll vectors of a thread, in pairs of
// fp32 numbers within a CTA and in fp64 from there on, always in the same
// order: the norm has the same bits for the same list.  A CTA whose squares
// leave fp32's range goes over its share again with scaled values.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kClipThreads = 512;
constexpr int kChunk = 2048;    // values of a chunk
constexpr int kUnroll = 4;      // 16-byte loads a thread has in flight
constexpr int kSmallList = 32;  // tensors of the short parameter block

template <int kMax>
struct TensorList {
  const void* g[kMax];
  void* out[kMax];
  int64_t n[kMax];
  int64_t first[kMax];  // index of the tensor's first chunk
  int count;
  int64_t chunks;
};

template <int kMax>
__device__ __forceinline__ int find_tensor(const TensorList<kMax>& l, int64_t chunk) {
  int lo = 0, hi = l.count - 1;  // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Sixteen bytes of values as fp32.
template <bool kBf16>
struct Vec {
  static constexpr int kN = kBf16 ? 8 : 4;
  float v[kN];
  __device__ __forceinline__ explicit Vec(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kBf16) {
        v[2 * j] = bf16lo_to_f32(w[j]);
        v[2 * j + 1] = bf16hi_to_f32(w[j]);
      } else {
        v[j] = __uint_as_float(w[j]);
      }
    }
  }
};

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (kBf16)
    return bf16lo_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ bool aligned(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The sum of the CTAs' partial sums by the block's first four warps, in a
// fixed order; the result in thread 0.
__device__ __forceinline__ double sum_partials(const double* partials, int count) {
  constexpr int kPer = kClipMaxPartials / 128;
  __shared__ double red[4];
  if (threadIdx.x < 128) {
    double part[kPer], all = 0.0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {  // all loads in flight together
      const int i = threadIdx.x + 128 * k;
      part[k] = i < count ? __ldcg(partials + i) : 0.0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (128 * k < count) all += part[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_down_sync(0xFFFFFFFFu, all, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = all;
  }
  __syncthreads();
  return threadIdx.x == 0 ? (red[0] + red[1]) + (red[2] + red[3]) : 0.0;
}

// A CTA's run of chunks is a piece of one tensor or of several; walk() calls
// fn(tensor, first value, values) for each piece.
template <int kMax, typename Fn>
__device__ __forceinline__ void walk(const TensorList<kMax>& l, Fn fn) {
  int64_t c = l.chunks * blockIdx.x / gridDim.x;
  const int64_t end = l.chunks * (blockIdx.x + 1) / gridDim.x;
  if (c >= end) return;
  for (int t = find_tensor(l, c); c < end; ++t) {
    const int64_t begin = (c - l.first[t]) * kChunk;
    const int64_t stop = min(l.n[t], (end - l.first[t]) * kChunk);
    fn(t, begin, stop - begin);
    c = l.first[t] + (l.n[t] + kChunk - 1) / kChunk;
  }
}

// An unevaluated sum hi + lo of fp32 numbers >= 0: 48 bits at fp32 rates
// (this GPU adds two fp64 numbers a clock and SM).
struct Pair {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x) {  // Knuth's exact sum
    const float t = __fadd_rn(hi, x);
    const float z = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
    hi = t;
  }
};

// Adds the squares of this thread's share of n values, times scale first
// where kScaled, to acc: in fp32 over kUnroll vectors, then in the pair.  The
// values' bits are collected in `any`.
template <bool kBf16, bool kScaled>
__device__ __forceinline__ void square_sums(const uint8_t* base, int64_t n, float scale, Pair& acc,
                                            uint32_t& any) {
  constexpr int kN = Vec<kBf16>::kN;
  int64_t done = 0;
  if (aligned(base)) {
    const int64_t vecs = n / kN;
    const uint4* v = reinterpret_cast<const uint4*>(base);
    for (int64_t i = threadIdx.x; i < vecs; i += kUnroll * kClipThreads) {
      uint4 u[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        u[k] = i + k * kClipThreads < vecs ? __ldg(v + i + k * kClipThreads)
                                           : make_uint4(0, 0, 0, 0);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (!kScaled) any |= u[k].x | u[k].y | u[k].z | u[k].w;
        const Vec<kBf16> x(u[k]);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const float y = kScaled ? __fmul_rn(x.v[j], scale) : x.v[j];
          s = __fmaf_rn(y, y, s);
        }
      }
      acc.add(s);
    }
    done = vecs * kN;
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kClipThreads) {
    const float x = load_one<kBf16>(base, i);
    if (!kScaled) any |= __float_as_uint(x);
    const float y = kScaled ? __fmul_rn(x, scale) : x;
    acc.add(__fmul_rn(y, y));
  }
}

// What a norm launch does with the CTAs' partial sums.
enum NormEnd : int {
  kLeave = 0,   // leaves them for the scaling, which adds them up itself
  kCarry = 1,   // the last CTA adds them to *total
  kFinish = 2,  // the last CTA adds them up (and *total, unless first) and writes the norm
};

template <bool kBf16, int kMax>
__global__ void __launch_bounds__(kClipThreads, 2048 / kClipThreads)
    grad_norm_kernel(const __grid_constant__ TensorList<kMax> l, double* partials, double* total,
                     uint32_t* ticket, float* norm, bool first, int end) {
  griddep_wait();
  griddep_launch_dependents();
  Pair acc;
  uint32_t any = 0;
  walk(l, [&](int t, int64_t begin, int64_t n) {
    square_sums<kBf16, false>(static_cast<const uint8_t*>(l.g[t]) + begin * (kBf16 ? 2 : 4), n, 1.0f,
                              acc, any);
  });
  // Squares that may overflow (values from 1e15 on, infinities, NaN) or that
  // may lose bits to underflow (all below 1e-14, though not all zero): the
  // share again, its values times a power of two that keeps any sum of them
  // in range.
  float scale = 1.0f;
  if (__syncthreads_or(!(acc.hi < 1e30f))) {
    scale = 0x1p-80f;
  } else if (__syncthreads_and(acc.hi < 1e-28f) &&
             __syncthreads_or((any & (kBf16 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) != 0)) {
    scale = 0x1p100f;
  }
  if (scale != 1.0f) {
    acc = Pair();
    walk(l, [&](int t, int64_t begin, int64_t n) {
      square_sums<kBf16, true>(static_cast<const uint8_t*>(l.g[t]) + begin * (kBf16 ? 2 : 4), n,
                               scale, acc, any);
    });
  }
  __shared__ float2 warp_sum[kClipThreads / 32];
  auto warp_add = [&](int from) {
#pragma unroll
    for (int o = from; o > 0; o >>= 1) {
      const float hi = __shfl_down_sync(0xFFFFFFFFu, acc.hi, o);
      const float lo = __shfl_down_sync(0xFFFFFFFFu, acc.lo, o);
      acc.add(hi);
      acc.lo = __fadd_rn(acc.lo, lo);
    }
  };
  warp_add(16);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = make_float2(acc.hi, acc.lo);
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x < 32) {
    const float2 w = threadIdx.x < kClipThreads / 32 ? warp_sum[threadIdx.x] : make_float2(0, 0);
    acc.hi = w.x;
    acc.lo = w.y;
    warp_add(kClipThreads / 64);
    // An infinite sum has lost its error terms.
    sum = isinf(acc.hi) ? acc.hi : static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
    const double back = 1.0 / scale;  // a power of two
    sum *= back * back;
  }
  __shared__ bool is_last;
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = sum;
    if (end != kLeave) {
      __threadfence();
      is_last = atomicAdd(ticket, 1u) == gridDim.x - 1u;
    }
  }
  if (end == kLeave) return;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  double all = sum_partials(partials, gridDim.x);
  if (threadIdx.x == 0) {
    *ticket = 0u;
    if (!first) all += *total;
    if (end == kFinish)
      *norm = static_cast<float>(sqrt(all));
    else
      *total = all;
  }
}

template <bool kBf16, bool kOutBf16, int kMax>
__global__ void __launch_bounds__(kClipThreads, 2048 / kClipThreads)
    grad_scale_kernel(const __grid_constant__ TensorList<kMax> l, float* norm, float max_norm,
                      float eps, const double* partials, int count) {
  griddep_wait();
  griddep_launch_dependents();
  float length;
  if (count > 0) {  // the norm launch left its partial sums
    __shared__ float shared_length;
    const double all = sum_partials(partials, count);
    if (threadIdx.x == 0) {
      shared_length = static_cast<float>(sqrt(all));
      if (blockIdx.x == 0) *norm = shared_length;
    }
    __syncthreads();
    length = shared_length;
  } else {
    length = *norm;
  }
  // A comparison, not the smaller of 1 and the quotient: inf / inf (nothing is
  // to be clipped) and 0 / 0 would be NaN.  A NaN norm makes every gradient NaN.
  const float bound = __fadd_rn(length, eps);
  const float coef = bound <= max_norm ? 1.0f : __fdiv_rn(max_norm, bound);
  // A thread's vector: 16 bytes of the wider of the two types.
  constexpr int kN = kBf16 && kOutBf16 ? 8 : 4;
  using In = std::conditional_t<kBf16 && !kOutBf16, uint2, uint4>;
  walk(l, [&](int t, int64_t begin, int64_t n) {
    // In place, a factor of one leaves the values as they are.
    if (kBf16 == kOutBf16 && coef == 1.0f && l.g[t] == l.out[t]) return;
    const uint8_t* base = static_cast<const uint8_t*>(l.g[t]) + begin * (kBf16 ? 2 : 4);
    uint8_t* dst = static_cast<uint8_t*>(l.out[t]) + begin * (kOutBf16 ? 2 : 4);
    const int64_t vecs = aligned(base) && aligned(dst) ? n / kN : 0;
    const In* v = reinterpret_cast<const In*>(base);
    // From the end: what the norm read last is still in L2.
    for (int64_t top = vecs; top > 0; top -= kUnroll * kClipThreads) {
      In u[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t i = top - 1 - k * kClipThreads - threadIdx.x;
        if (i >= 0) u[k] = v[i];
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t i = top - 1 - k * kClipThreads - threadIdx.x;
        if (i < 0) break;
        float x[kN];
        if constexpr (kBf16) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&u[k]);
#pragma unroll
          for (int j = 0; j < kN / 2; ++j) mul2_rn(w[j] << 16, w[j] & 0xFFFF0000u, coef, x[2 * j], x[2 * j + 1]);
        } else {
          mul2_rn(u[k].x, u[k].y, coef, x[0], x[1]);
          mul2_rn(u[k].z, u[k].w, coef, x[2], x[3]);
        }
        if constexpr (!kOutBf16)
          __stcs(reinterpret_cast<float4*>(dst) + i, make_float4(x[0], x[1], x[2], x[3]));
        else if constexpr (kN == 8)
          __stcs(reinterpret_cast<uint4*>(dst) + i,
                 make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]),
                            cvt_bf16x2(x[6], x[7])));
        else
          __stcs(reinterpret_cast<uint2*>(dst) + i,
                 make_uint2(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3])));
      }
    }
    for (int64_t i = vecs * kN + threadIdx.x; i < n; i += kClipThreads) {
      const float x = __fmul_rn(load_one<kBf16>(base, i), coef);
      if constexpr (kOutBf16)
        reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(cvt_bf16x2(x, 0.0f) & 0xFFFFu);
      else
        reinterpret_cast<float*>(dst)[i] = x;
    }
  });
}

template <int kMax>
TensorList<kMax> make_list(const GradTensor* t, int n) {
  TensorList<kMax> l;
  l.count = 0;
  l.chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;  // every tensor of the list has a chunk
    l.g[l.count] = t[i].g;
    l.out[l.count] = t[i].out;
    l.n[l.count] = t[i].n;
    l.first[l.count] = l.chunks;
    l.chunks += (t[i].n + kChunk - 1) / kChunk;
    ++l.count;
  }
  return l;
}

unsigned clip_grid(int64_t chunks, const DeviceInfo& dev) {
  int64_t most = 2048 / kClipThreads * int64_t(dev.num_sms);  // all resident at once
  if (most > kClipMaxPartials) most = kClipMaxPartials;
  const int64_t g = chunks < most ? chunks : most;
  return static_cast<unsigned>(g > 0 ? g : 1);
}

template <int kMax>
cudaError_t norm_list(const GradTensor* t, int n, const GradNormArgs& a, const DeviceInfo& dev,
                      cudaStream_t stream, int* grid_out) {
  const TensorList<kMax> l = make_list<kMax>(t, n);
  const dim3 grid(clip_grid(l.chunks, dev)), block(kClipThreads);
  *grid_out = static_cast<int>(grid.x);
  const int end = a.leave ? kLeave : a.last ? kFinish : kCarry;
  return a.bf16 ? launch_kernel(grad_norm_kernel<true, kMax>, grid, block, 0, stream, 1, false, l,
                                a.partials, a.total, a.ticket, a.norm, a.first, end)
                : launch_kernel(grad_norm_kernel<false, kMax>, grid, block, 0, stream, 1, false, l,
                                a.partials, a.total, a.ticket, a.norm, a.first, end);
}

template <int kMax>
cudaError_t scale_list(const GradTensor* t, int n, const GradScaleArgs& a, const DeviceInfo& dev,
                       cudaStream_t stream) {
  const TensorList<kMax> l = make_list<kMax>(t, n);
  const dim3 grid(clip_grid(l.chunks, dev)), block(kClipThreads);
  auto run = [&](auto* kernel) {
    return launch_kernel(kernel, grid, block, 0, stream, 1, false, l, a.norm, a.max_norm, a.eps,
                         static_cast<const double*>(a.partials), a.count);
  };
  if (a.bf16)
    return a.out_bf16 ? run(grad_scale_kernel<true, true, kMax>)
                      : run(grad_scale_kernel<true, false, kMax>);
  return a.out_bf16 ? run(grad_scale_kernel<false, true, kMax>)
                    : run(grad_scale_kernel<false, false, kMax>);
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* t, int n, const GradNormArgs& a,
                             const DeviceInfo& dev, cudaStream_t stream, int* grid) {
  set_error_site("grad_norm_kernel");
  return n <= kSmallList ? norm_list<kSmallList>(t, n, a, dev, stream, grid)
                         : norm_list<kClipMaxTensors>(t, n, a, dev, stream, grid);
}

cudaError_t launch_grad_scale(const GradTensor* t, int n, const GradScaleArgs& a,
                              const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("grad_scale_kernel");
  return n <= kSmallList ? scale_list<kSmallList>(t, n, a, dev, stream)
                         : scale_list<kClipMaxTensors>(t, n, a, dev, stream);
}

}  // namespace fp8lin
