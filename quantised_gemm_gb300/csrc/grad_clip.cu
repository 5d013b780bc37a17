// grad_clip.cu -- the global 2-norm of a list of gradients and their scaling
// to a largest norm:
//   norm = sqrt(sum_t sum_i g_t[i]^2),  out_t[i] = g_t[i] * min(1, max_norm / (norm + eps)).
//
// Bound by memory: the norm reads every gradient once, the scaling reads and
// writes it once.  The list travels in the kernel's parameters (no table on
// the device, so the calls can be captured and the tensors may move from call
// to call).  The list is cut into chunks of kChunk values; a CTA takes chunks
// round-robin and finds a chunk's tensor by bisection.  Squares are added in
// fp32 within a thread's share of a chunk and in fp64 from there on, always
// in the same order: the norm has the same bits for the same list.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kClipThreads = 256;
constexpr int kChunk = 16384;   // values of a chunk: 8 rounds of 8 values a thread
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

// Sum over the block in a fixed order; the result in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kClipThreads / 32; ++w) s += red[w];
  return s;
}

// One thread's share of the squares of n values, added up in Acc.
template <bool kBf16, typename Acc>
__device__ __forceinline__ Acc square_sum(const uint8_t* base, int n) {
  constexpr int kN = Vec<kBf16>::kN;
  Acc s = 0;
  int done = 0;
  if (aligned(base)) {
    const int vecs = n / kN;
    const uint4* v = reinterpret_cast<const uint4*>(base);
    for (int i = threadIdx.x; i < vecs; i += 4 * kClipThreads) {
      uint4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[k] = i + k * kClipThreads < vecs ? __ldg(v + i + k * kClipThreads)
                                           : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Vec<kBf16> x(u[k]);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const Acc y = x.v[j];
          s = fma(y, y, s);
        }
      }
    }
    done = vecs * kN;
  }
  for (int i = done + threadIdx.x; i < n; i += kClipThreads) {
    const Acc y = load_one<kBf16>(base, i);
    s = fma(y, y, s);
  }
  return s;
}

template <bool kBf16, int kMax>
__global__ void __launch_bounds__(kClipThreads)
    grad_norm_kernel(const __grid_constant__ TensorList<kMax> l, double* partials, double* total,
                     uint32_t* ticket, float* norm, bool first, bool last) {
  griddep_wait();
  griddep_launch_dependents();
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const int t = find_tensor(l, c);
    const int64_t begin = (c - l.first[t]) * kChunk;
    const int64_t left = l.n[t] - begin;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    const uint8_t* base = static_cast<const uint8_t*>(l.g[t]) + begin * (kBf16 ? 2 : 4);
    const float s = square_sum<kBf16, float>(base, n);
    // Squares of values above 1.8e19 overflow fp32: those shares again in fp64.
    sum += isinf(s) ? square_sum<kBf16, double>(base, n) : static_cast<double>(s);
  }
  sum = block_sum(sum);
  __shared__ bool is_last;
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = sum;
    __threadfence();
    is_last = atomicAdd(ticket, 1u) == gridDim.x - 1u;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  double all = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kClipThreads) all += __ldcg(partials + i);
  all = block_sum(all);
  if (threadIdx.x == 0) {
    *ticket = 0u;
    if (!first) all += *total;
    if (last)
      *norm = static_cast<float>(sqrt(all));
    else
      *total = all;
  }
}

template <bool kBf16, bool kOutBf16, int kMax>
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(const __grid_constant__ TensorList<kMax> l, const float* norm, float max_norm,
                      float eps) {
  griddep_wait();
  griddep_launch_dependents();
  const float q = __fdiv_rn(max_norm, __fadd_rn(*norm, eps));
  const float coef = q > 1.0f ? 1.0f : q;  // a NaN norm makes every gradient NaN
  constexpr int kN = Vec<kBf16>::kN;
  for (int64_t c0 = blockIdx.x; c0 < l.chunks; c0 += gridDim.x) {
    // From the end of the list: what the norm read last may still be in L2.
    const int64_t c = l.chunks - 1 - c0;
    const int t = find_tensor(l, c);
    // In place, a factor of one leaves the values as they are.
    if (kBf16 == kOutBf16 && coef == 1.0f && l.g[t] == l.out[t]) continue;
    const int64_t begin = (c - l.first[t]) * kChunk;
    const int64_t left = l.n[t] - begin;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    const uint8_t* base = static_cast<const uint8_t*>(l.g[t]) + begin * (kBf16 ? 2 : 4);
    uint8_t* dst = static_cast<uint8_t*>(l.out[t]) + begin * (kOutBf16 ? 2 : 4);
    int done = 0;
    if (aligned(base) && aligned(dst)) {
      const int vecs = n / kN;
      const uint4* v = reinterpret_cast<const uint4*>(base);
      for (int i0 = threadIdx.x; i0 < vecs; i0 += 4 * kClipThreads) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + k * kClipThreads < vecs) u[k] = v[i0 + k * kClipThreads];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k * kClipThreads;
          if (i >= vecs) break;
          const Vec<kBf16> x(u[k]);
          if constexpr (kOutBf16 && kBf16) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = cvt_bf16x2(__fmul_rn(x.v[2 * j], coef), __fmul_rn(x.v[2 * j + 1], coef));
            reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
          } else if constexpr (kOutBf16) {
            reinterpret_cast<uint2*>(dst)[i] =
                make_uint2(cvt_bf16x2(__fmul_rn(x.v[0], coef), __fmul_rn(x.v[1], coef)),
                           cvt_bf16x2(__fmul_rn(x.v[2], coef), __fmul_rn(x.v[3], coef)));
          } else {
#pragma unroll
            for (int j = 0; j < kN / 4; ++j)
              reinterpret_cast<float4*>(dst)[i * (kN / 4) + j] =
                  make_float4(__fmul_rn(x.v[4 * j], coef), __fmul_rn(x.v[4 * j + 1], coef),
                              __fmul_rn(x.v[4 * j + 2], coef), __fmul_rn(x.v[4 * j + 3], coef));
          }
        }
      }
      done = vecs * kN;
    }
    for (int i = done + threadIdx.x; i < n; i += kClipThreads) {
      const float x = __fmul_rn(load_one<kBf16>(base, i), coef);
      if constexpr (kOutBf16)
        reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(cvt_bf16x2(x, 0.0f) & 0xFFFFu);
      else
        reinterpret_cast<float*>(dst)[i] = x;
    }
  }
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
  int64_t most = 8 * int64_t(dev.num_sms);
  if (most > kClipMaxPartials) most = kClipMaxPartials;
  const int64_t g = chunks < most ? chunks : most;
  return static_cast<unsigned>(g > 0 ? g : 1);
}

template <int kMax>
cudaError_t norm_list(const GradTensor* t, int n, bool bf16, bool first, bool last,
                      double* partials, double* total, uint32_t* ticket, float* norm,
                      const DeviceInfo& dev, cudaStream_t stream) {
  const TensorList<kMax> l = make_list<kMax>(t, n);
  const dim3 grid(clip_grid(l.chunks, dev)), block(kClipThreads);
  return bf16 ? launch_kernel(grad_norm_kernel<true, kMax>, grid, block, 0, stream, 1, false, l,
                              partials, total, ticket, norm, first, last)
              : launch_kernel(grad_norm_kernel<false, kMax>, grid, block, 0, stream, 1, false, l,
                              partials, total, ticket, norm, first, last);
}

template <int kMax>
cudaError_t scale_list(const GradTensor* t, int n, bool bf16, bool out_bf16, const float* norm,
                       float max_norm, float eps, const DeviceInfo& dev, cudaStream_t stream) {
  const TensorList<kMax> l = make_list<kMax>(t, n);
  if (l.chunks == 0) return cudaSuccess;
  const dim3 grid(clip_grid(l.chunks, dev)), block(kClipThreads);
  if (bf16)
    return out_bf16 ? launch_kernel(grad_scale_kernel<true, true, kMax>, grid, block, 0, stream, 1,
                                    false, l, norm, max_norm, eps)
                    : launch_kernel(grad_scale_kernel<true, false, kMax>, grid, block, 0, stream, 1,
                                    false, l, norm, max_norm, eps);
  return out_bf16 ? launch_kernel(grad_scale_kernel<false, true, kMax>, grid, block, 0, stream, 1,
                                  false, l, norm, max_norm, eps)
                  : launch_kernel(grad_scale_kernel<false, false, kMax>, grid, block, 0, stream, 1,
                                  false, l, norm, max_norm, eps);
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* t, int n, bool bf16, bool first, bool last,
                             double* partials, double* total, uint32_t* ticket, float* norm,
                             const DeviceInfo& dev, cudaStream_t stream) {
  set_error_site("grad_norm_kernel");
  return n <= kSmallList ? norm_list<kSmallList>(t, n, bf16, first, last, partials, total, ticket,
                                                 norm, dev, stream)
                         : norm_list<kClipMaxTensors>(t, n, bf16, first, last, partials, total,
                                                      ticket, norm, dev, stream);
}

cudaError_t launch_grad_scale(const GradTensor* t, int n, bool bf16, bool out_bf16,
                              const float* norm, float max_norm, float eps, const DeviceInfo& dev,
                              cudaStream_t stream) {
  set_error_site("grad_scale_kernel");
  return n <= kSmallList ? scale_list<kSmallList>(t, n, bf16, out_bf16, norm, max_norm, eps, dev, stream)
                         : scale_list<kClipMaxTensors>(t, n, bf16, out_bf16, norm, max_norm, eps,
                                                       dev, stream);
}

}  // namespace fp8lin
