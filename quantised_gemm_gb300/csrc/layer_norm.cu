// layer_norm.cu -- layer norm of bf16 rows, with an optional residual before
// it, and its backward pass:
//   h = bf16(x + r) (r given) or x;  mu = mean(h), rstd = 1 / sqrt(mean((h - mu)^2) + eps)
//   y = bf16((h - mu) rstd w + b)
//   xhat = (h - mu) rstd, g = dy w
//   dx = bf16(rstd (g - mean(g) - xhat mean(g xhat)) + dres)
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Bound by memory: each tensor is read or written once.  65536 x 4096 with a
// residual: forward 303 us (7.1 TB/s), backward 350 us (6.1 TB/s) and 5 for the sums
// over the CTAs; 12288 x 1600 from L2 14 us, of which the issue of instructions is 10.
// Few rows are latency: 16 x 4096 takes 3 us, the backward of 256 x 4096 8 us in two
// launches.  4096 x 16384 takes 102 us forward and 188 backward with a residual (5.3 and
// 2.9 TB/s): 1024 threads leave 64 registers each, and the row's values spill.
// A group of threads holds a row in registers, eight consecutive values a vector, so
// the second look at the values (the deviations; the backward's dx) costs no second
// read, and the variance is the mean of squared deviations, not a difference of
// large sums.  A finite row whose sums leave fp32's range is computed once more from 2^-72
// of its values.  Statistics and column sums are fp32, in packed pairs (half the
// instructions); y, h and dx are rounded once.  The forward takes two rows of a group
// at a time and one CTA a pair: 304 us where CTAs that loop over rows took 328.
// In the backward a thread owns the same columns of every row that its CTA takes and
// keeps their sums in registers, with the rows ahead on their way in shared memory
// (558 us without); a CTA writes one row of partial sums, and a second launch adds
// those in a fixed order.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
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
template <int kThreads>
__device__ __forceinline__ void group_sum(float& v, float& u, int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  }
  if constexpr (kThreads > 32) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float2 words[2][kWarps];
    if ((threadIdx.x & 31) == 0) words[turn & 1][threadIdx.x >> 5] = make_float2(v, u);
    __syncthreads();
    v = u = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float2 w = words[turn & 1][i];
      v += w.x;
      u += w.y;
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

// Pairs of fp32 numbers, each rounded as the scalar operation rounds it.
union F2 {
  float2 f;
  uint64_t u;
};
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 r;
  r.f = make_float2(x, y);
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
}
__device__ __forceinline__ void unpack(const uint4& u, F2 (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j]));
}

template <typename P>
__device__ __forceinline__ void load_pairs(const P* p, int n, F2 (&v)[4]) {
  float w[8];
  load_params(p, n, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair(w[2 * j], w[2 * j + 1]);
}

// n values of a row that are real, of the eight from column c on.
template <bool kAligned>
__device__ __forceinline__ int values_of(int c, int cols) {
  return kAligned ? (c < cols ? 8 : 0) : values_at(c, cols);
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

constexpr float kInf = __builtin_huge_valf(), kDown = 0x1p-72f;

// sum / cols: the product with 1 / cols and what the remainder adds to it (a division took
// 15.0 us for 12288 x 1600 instead of 14.9).  The sum of equal values is exact (8 bits and 14
// for their number), and so is their mean then.
__device__ __forceinline__ float mean_of(float sum, const NormParams& p) {
  const float q = sum * p.inv_cols;
  return fmaf(fmaf(-q, static_cast<float>(p.cols), sum), p.inv_cols, q);
}

// Two rows of a group at a time: their loads are in flight together, they share
// the barriers, and w and b are read once for both.
template <int kThreads, int kVecs, bool kAligned, bool kResidual, typename P>
__global__ void __launch_bounds__(Group<kThreads>::kBlock)
    layer_norm_kernel(const __grid_constant__ NormParams p) {
  using G = Group<kThreads>;
  griddep_wait();
  griddep_launch_dependents();
  const int t = G::kRows > 1 ? static_cast<int>(threadIdx.x & 31u) : static_cast<int>(threadIdx.x);
  const int64_t group = int64_t(blockIdx.x) * G::kRows + (G::kRows > 1 ? threadIdx.x >> 5 : 0);
  const int64_t step = int64_t(gridDim.x) * G::kRows;
  uint32_t most = 0;
  int turn = 0;
  for (int64_t row = group; row < p.rows; row += 2 * step) {
    const int64_t at[2] = {row, row + step};
    const bool second = at[1] < p.rows;
    uint4 v[2][kVecs];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        v[i][k] = load_values<kAligned>(p.x + at[i] * p.ldx + c, i == 0 || second ? values_of<kAligned>(c, p.cols) : 0);
      }
    }
    if constexpr (kResidual) {
      uint4 u[2][kVecs];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = (k * kThreads + t) * 8;
          u[i][k] = load_values<kAligned>(p.r + at[i] * p.ldr + c, i == 0 || second ? values_of<kAligned>(c, p.cols) : 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = (k * kThreads + t) * 8;
          float a[8], b[8];
          bf16x8_to_f32(v[i][k], a);
          bf16x8_to_f32(u[i][k], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] += b[j];
          v[i][k] = f32_to_bf16x8(a);
          store_values<kAligned>(p.h + at[i] * p.ldh + c, v[i][k],
                                 i == 0 || second ? values_of<kAligned>(c, p.cols) : 0);
        }
      }
    }
    F2 d[2][kVecs][4];  // the values, then their deviations from the mean
    float mean[2], sq[2];
    float down[2] = {1.0f, 1.0f};
    auto deviations = [&](auto scaled) {
      float sum[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        F2 s = pair(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          unpack(v[i][k], d[i][k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (decltype(scaled)::value) d[i][k][j] = d[i][k][j] * pair(down[i], down[i]);
            s = s + d[i][k][j];
          }
        }
        sum[i] = s.f.x + s.f.y;
      }
      group_sum<kThreads>(sum[0], sum[1], turn++);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mean[i] = mean_of(sum[i], p);
        F2 s = pair(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int n = values_of<kAligned>((k * kThreads + t) * 8, p.cols);
          const float less = n > 0 ? -mean[i] : 0.0f;  // 0 stays 0 past the row's end
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[i][k][j] = d[i][k][j] + pair(less, !kAligned && 2 * j + 1 >= n ? 0.0f : less);
            if (!kAligned && 2 * j >= n) d[i][k][j].f.x = 0.0f;
            s = fma2(d[i][k][j], d[i][k][j], s);
          }
        }
        sq[i] = s.f.x + s.f.y;
      }
      group_sum<kThreads>(sq[0], sq[1], turn++);
    };
    deviations(std::false_type());
    float rstd[2] = {__frsqrt_rn(sq[0] * p.inv_cols + p.eps), __frsqrt_rn(sq[1] * p.inv_cols + p.eps)};
    float rstd_out[2] = {rstd[0], rstd[1]};
    if (!(sq[0] < kInf) || !(sq[1] < kInf)) {
      // A row whose sums leave fp32's range (or that has a NaN or an infinity): the same with
      // 2^-72 of its values, whose squares' sum is at most 2^(2 (128 - 72) + 14).  The values are
      // read again, as they are not kept.
      __syncwarp();  // the neighbour may have written some of the lane's part of h
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!(sq[i] < kInf)) down[i] = kDown;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = (k * kThreads + t) * 8;
          v[i][k] = load_values<kAligned>((kResidual ? p.h + at[i] * p.ldh : p.x + at[i] * p.ldx) + c,
                                          i == 0 || second ? values_of<kAligned>(c, p.cols) : 0);
        }
      }
      deviations(std::true_type());
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float var = fmaf(sq[i], p.inv_cols, p.eps * down[i] * down[i]);
        // Without deviations eps decides, too small to be scaled, and the deviations are 0.
        const bool equal = var == 0.0f && p.eps > 0.0f;
        rstd[i] = equal ? 0.0f : __frsqrt_rn(var);
        rstd_out[i] = equal ? __frsqrt_rn(p.eps) : rstd[i] * down[i];
        mean[i] *= 1.0f / down[i];
      }
    }
    if (p.stats != nullptr && t < 2 && (t == 0 || second)) {
      p.stats[t == 0 ? at[0] : at[1]] = t == 0 ? mean[0] : mean[1];
      p.stats[p.rows + (t == 0 ? at[0] : at[1])] = t == 0 ? rstd_out[0] : rstd_out[1];
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kThreads + t) * 8;
      const int n = values_of<kAligned>(c, p.cols);
      F2 w[4], b[4];
      load_pairs(static_cast<const P*>(p.w) + c, n, w);
      if (p.b != nullptr) {
        load_pairs(static_cast<const P*>(p.b) + c, n, b);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = pair(0.0f, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 y = fma2(d[i][k][j] * pair(rstd[i], rstd[i]), w[j], b[j]);
          o[j] = cvt_bf16x2(y.f.x, y.f.y);
        }
        const uint4 y = make_uint4(o[0], o[1], o[2], o[3]);
        const int m = i == 0 || second ? n : 0;
        store_values<kAligned>(p.y + at[i] * p.ldy + c, y, m);
        if (p.amax != nullptr) most = max(most, max_bits(first_values(y, m)));
      }
    }
  }
  if (p.amax != nullptr) record_max(most << 16, p.acc, p.ticket, p.amax);
}

// Columns of a row of partial sums: whole vectors.
__host__ __device__ constexpr int padded_cols(int cols) { return (cols + 7) / 8 * 8; }

struct NormBackwardParams {
  const uint16_t *dy, *x, *dres;
  uint16_t* dx;  // null: not wanted
  const void* w;
  const float* stats;
  float* partials;  // null, or a CTA's sums: padded_cols of dw, then of db
  int64_t lddy, ldx, lddres, lddx, rows;
  int cols;
  float inv_cols;
  uint32_t *amax, *acc, *ticket;
};

// Rows that a thread of the backward has on their way, in shared memory of its
// own (no thread reads another's, so its own wait for its copies is enough).
template <int kThreads, int kVecs, bool kResidual>
struct Ahead {
  static constexpr int kTensors = kResidual ? 3 : 2;
  static constexpr size_t kRowBytes = size_t(16) * kTensors * kVecs * Group<kThreads>::kBlock;
  static constexpr int kRows = 3 * kRowBytes <= 200 * 1024 ? 3 : 2;
  static constexpr size_t kBytes = kRows * kRowBytes;
};

// What lies past the row's end needs no care: x, dy and w are loaded as 0 there,
// so g and dy are 0 and add nothing to any sum as long as mean * rstd is finite, and dx
// is not stored.
template <int kThreads, int kVecs, bool kAligned, bool kResidual, typename P>
__global__ void __launch_bounds__(Group<kThreads>::kBlock)
    layer_norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  using G = Group<kThreads>;
  using A = Ahead<kThreads, kVecs, kResidual>;
  constexpr int kTensors = A::kTensors, kAhead = A::kRows;
  extern __shared__ uint4 ahead[];  // aligned rows: [kAhead][kTensors][kVecs][threads]
  griddep_wait();
  griddep_launch_dependents();
  const int t = G::kRows > 1 ? static_cast<int>(threadIdx.x & 31u) : static_cast<int>(threadIdx.x);
  const int64_t group = int64_t(blockIdx.x) * G::kRows + (G::kRows > 1 ? threadIdx.x >> 5 : 0);
  const int64_t step = int64_t(gridDim.x) * G::kRows;
  const uint16_t* const from[3] = {p.x, p.dy, p.dres};
  const int64_t ld[3] = {p.ldx, p.lddy, p.lddres};
  F2 dw[kVecs][4], db[kVecs][4];
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = pair(0.0f, 0.0f);
  uint32_t most = 0;
  int turn = 0;
  uint4 next[kTensors][kVecs];  // unaligned rows: the next row
  auto slot = [&](int stage, int tensor, int k) {
    return ahead + ((stage * kTensors + tensor) * kVecs + k) * G::kBlock + threadIdx.x;
  };
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (kAligned) {
      if (row < p.rows) {
#pragma unroll
        for (int i = 0; i < kTensors; ++i)
#pragma unroll
          for (int k = 0; k < kVecs; ++k) {
            const int c = (k * kThreads + t) * 8;
            if (c < p.cols) copy16(slot(stage, i, k), from[i] + row * ld[i] + c, true);
          }
      }
      copies_end();
    } else if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < kTensors; ++i)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = (k * kThreads + t) * 8;
          next[i][k] = load_values<false>(from[i] + row * ld[i] + c, values_of<false>(c, p.cols));
        }
    }
  };
  if constexpr (kAligned) {
    // Vectors past the row's end stay 0 in every stage.
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if ((k * kThreads + t) * 8 >= p.cols)
        for (int i = 0; i < kAhead * kTensors; ++i)
          *slot(i / kTensors, i % kTensors, k) = make_uint4(0, 0, 0, 0);
    for (int i = 0; i < kAhead - 1; ++i) fetch(group + i * step, i);
  } else {
    fetch(group, 0);
  }
  float mean = 0.0f, rstd = 0.0f;
  F2 w[kVecs][4];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int c = (k * kThreads + t) * 8;
    load_pairs(static_cast<const P*>(p.w) + c, values_of<kAligned>(c, p.cols), w[k]);
  }
  if (group < p.rows) {
    mean = p.stats[group];
    rstd = p.stats[p.rows + group];
  }
  int stage = 0;
  for (int64_t row = group; row < p.rows; row += step) {
    uint4 res[kVecs];
    F2 g[kVecs][4], xhat[kVecs][4];
    F2 s1 = pair(0.0f, 0.0f), s2 = pair(0.0f, 0.0f);
    // Only rows of equal values (xhat = 0) leave fp32's range here: different ones of 8 bits
    // deviate by 2^-9 |mean| / sqrt(cols) at least.
    const float r = fabsf(mean) * rstd < kInf ? rstd : 0.0f;
    if constexpr (kAligned) {
      copies_wait<kAhead - 2>();  // this row's; the thread's own, so no barrier
      fetch(row + (kAhead - 1) * step, stage == 0 ? kAhead - 1 : stage - 1);
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      F2 a[4];
      if constexpr (kAligned) {
        unpack(*slot(stage, 0, k), xhat[k]);
        unpack(*slot(stage, 1, k), a);
        if (kResidual) res[k] = *slot(stage, 2, k);
      } else {
        unpack(next[0][k], xhat[k]);
        unpack(next[1][k], a);
        if (kResidual) res[k] = next[kTensors - 1][k];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xhat[k][j] = (xhat[k][j] + pair(-mean, -mean)) * pair(r, r);
        g[k][j] = a[j] * w[k][j];
        dw[k][j] = fma2(a[j], xhat[k][j], dw[k][j]);
        db[k][j] = db[k][j] + a[j];
        s1 = s1 + g[k][j];
        s2 = fma2(g[k][j], xhat[k][j], s2);
      }
    }
    const float scale = rstd;
    if constexpr (!kAligned) fetch(row + step, 0);
    if (row + step < p.rows) {
      mean = p.stats[row + step];
      rstd = p.stats[p.rows + row + step];
    }
    float m1 = s1.f.x + s1.f.y, m2 = s2.f.x + s2.f.y;
    group_sum<kThreads>(m1, m2, turn++);
    m1 *= -p.inv_cols;
    m2 *= -p.inv_cols;
    if (p.dx != nullptr) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        const int n = values_of<kAligned>(c, p.cols);
        F2 b[4];
        if constexpr (kResidual) unpack(res[k], b);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 v = fma2(xhat[k][j], pair(m2, m2), g[k][j] + pair(m1, m1));
          v = kResidual ? fma2(v, pair(scale, scale), b[j]) : v * pair(scale, scale);
          o[j] = cvt_bf16x2(v.f.x, v.f.y);
        }
        const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
        store_values<kAligned>(p.dx + row * p.lddx + c, out, n);
        if (p.amax != nullptr) most = max(most, max_bits(first_values(out, n)));
      }
    }
    stage = stage == kAhead - 1 ? 0 : stage + 1;
  }
  if constexpr (kAligned) copies_wait<0>();
  if (p.partials != nullptr) {
    if constexpr (G::kRows > 1) {  // the CTA's warps together, one after another
      __shared__ float2 all[kVecs * 8 * 32];
      for (int turn_of = 0; turn_of < G::kRows; ++turn_of) {
        if (static_cast<int>(threadIdx.x >> 5) == turn_of) {
#pragma unroll
          for (int k = 0; k < kVecs; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float2& sum = all[(k * 8 + j) * 32 + t];
              const float a = j % 2 ? dw[k][j / 2].f.y : dw[k][j / 2].f.x;
              const float b = j % 2 ? db[k][j / 2].f.y : db[k][j / 2].f.x;
              sum = turn_of == 0 ? make_float2(a, b) : make_float2(sum.x + a, sum.y + b);
            }
        }
        __syncthreads();
      }
      if (threadIdx.x < 32) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = all[(k * 8 + 2 * j) * 32 + t], b = all[(k * 8 + 2 * j + 1) * 32 + t];
            dw[k][j] = pair(a.x, b.x);
            db[k][j] = pair(a.y, b.y);
          }
      }
    }
    if (G::kRows == 1 || threadIdx.x < 32) {
      const int padded = padded_cols(p.cols);
      float* to = p.partials + int64_t(blockIdx.x) * 2 * padded;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * kThreads + t) * 8;
        if (c >= p.cols) continue;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const F2 *a = dw[k] + j, *b = db[k] + j;
          *reinterpret_cast<float4*>(to + c + 2 * j) =
              make_float4(a[0].f.x, a[0].f.y, a[1].f.x, a[1].f.y);
          *reinterpret_cast<float4*>(to + padded + c + 2 * j) =
              make_float4(b[0].f.x, b[0].f.y, b[1].f.x, b[1].f.y);
        }
      }
    }
  }
  if (p.amax != nullptr) record_max(most << 16, p.acc, p.ticket, p.amax);
}

// Column sums of `groups` rows of partial sums: 32 columns a CTA, its warps
// each every kSumWarps-th row, kSumLoads of them in flight.
constexpr int kSumWarps = 32, kSumLoads = 10;

template <typename P>
__global__ void __launch_bounds__(32 * kSumWarps)
    layer_norm_sum_kernel(const float* partials, int groups, int cols, P* dw, P* db) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int padded = padded_cols(cols);
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;  // of dw and db together
  float sum = 0.0f;
  if (c < 2 * padded) {
    for (int g = warp; g < groups; g += kSumWarps * kSumLoads) {
      float v[kSumLoads];
#pragma unroll
      for (int i = 0; i < kSumLoads; ++i)
        v[i] = g + i * kSumWarps < groups
                   ? __ldcg(partials + int64_t(g + i * kSumWarps) * 2 * padded + c)
                   : 0.0f;
#pragma unroll
      for (int i = 0; i < kSumLoads; ++i) sum += v[i];
    }
  }
  __shared__ float part[kSumWarps][33];
  part[warp][lane] = sum;
  __syncthreads();
  // Warp w adds column w's numbers.
  sum = part[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const int at = static_cast<int>(blockIdx.x) * 32 + warp;
  P* out = at < padded ? dw : db;
  const int to = at < padded ? at : at - padded;
  if (lane != 0 || to >= cols || out == nullptr) return;
  if constexpr (sizeof(P) == 2)
    out[to] = static_cast<uint16_t>(cvt_bf16x2(sum, 0.0f) & 0xFFFFu);
  else
    out[to] = sum;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether all of a tensor's vectors are aligned; a null tensor's are.
bool rows_aligned(const void* p, int64_t ld) { return p == nullptr || (aligned16(p) && ld % 8 == 0); }

// Threads a row and vectors a thread.
template <int kThreads, int kVecs>
struct Shape {
  static constexpr int threads = kThreads, vecs = kVecs;
};

template <int kThreads, int kVecs, bool kAligned, bool kResidual, typename P>
cudaError_t run_backward(const NormBackwardParams& p, dim3 grid, const DeviceInfo& dev,
                         cudaStream_t stream) {
  constexpr auto* kernel = layer_norm_backward_kernel<kThreads, kVecs, kAligned, kResidual, P>;
  constexpr size_t kBytes = kAligned ? Ahead<kThreads, kVecs, kResidual>::kBytes : 0;
  if constexpr (kBytes > 40 * 1024) {  // 48 KB with the static part
    static std::mutex mu;
    static bool done[64];  // devices on which the kernel may have that much
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev.device]) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kBytes));
      if (e != cudaSuccess) return e;
      done[dev.device] = true;
    }
  }
  return launch_kernel(kernel, grid, dim3(Group<kThreads>::kBlock), kBytes, stream, 1, false, p);
}

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
    const int64_t want = (a.rows + 2 * G::kRows - 1) / (2 * G::kRows);
    const int64_t most = (int64_t(1) << 31) - 1;
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
    // Two rows a group at least (256 x 4096: 8.1 us; one 8.1, four 9.7), and no
    // more CTAs than are resident, as each leaves a row of partial sums.
    const int64_t want = (a.rows + 2 * G::kRows - 1) / (2 * G::kRows);
    int64_t most = int64_t(dev.num_sms) * (G::kBlock >= 512 ? 1 : 512 / G::kBlock);
    if (sums) {
      const int64_t room = static_cast<int64_t>(a.ws_bytes / (sizeof(float) * 2 * padded_cols(static_cast<int>(a.cols))));
      if (room < most) most = room;
    }
    if (most < 1) return cudaErrorInvalidValue;  // the caller has checked that one fits
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    groups = static_cast<int>(grid.x);
    p.partials = sums ? a.ws : nullptr;
    auto pick = [&](auto flag) {
      constexpr bool kAligned = decltype(flag)::value;
      if (a.param_f32)
        return a.dres != nullptr
                   ? run_backward<S::threads, S::vecs, kAligned, true, float>(p, grid, dev, stream)
                   : run_backward<S::threads, S::vecs, kAligned, false, float>(p, grid, dev, stream);
      return a.dres != nullptr
                 ? run_backward<S::threads, S::vecs, kAligned, true, uint16_t>(p, grid, dev, stream)
                 : run_backward<S::threads, S::vecs, kAligned, false, uint16_t>(p, grid, dev, stream);
    };
    return aligned ? pick(std::true_type()) : pick(std::false_type());
  };
  cudaError_t e;
  if (a.cols <= 256) e = run(Shape<32, 1>());
  else if (a.cols <= 512) e = run(Shape<32, 2>());
  else if (a.cols <= 1024) e = run(Shape<128, 1>());
  else if (a.cols <= 2048) e = run(Shape<256, 1>());
  else if (a.cols <= 4096) e = run(Shape<256, 2>());
  else if (a.cols <= 8192) e = run(Shape<512, 2>());
  else e = run(Shape<1024, 2>());
  *launches = 1;
  if (e != cudaSuccess || !sums) return e;
  *launches = 2;
  set_error_site("layer_norm_sum_kernel");
  const int cols = static_cast<int>(a.cols);
  const dim3 grid(static_cast<unsigned>((2 * padded_cols(cols) + 31) / 32)), block(32 * kSumWarps);
  const float* partials = a.ws;
  if (a.param_f32)
    return launch_kernel(layer_norm_sum_kernel<float>, grid, block, 0, stream, 1, false, partials,
                         groups, cols, static_cast<float*>(a.dw), static_cast<float*>(a.db));
  return launch_kernel(layer_norm_sum_kernel<uint16_t>, grid, block, 0, stream, 1, false, partials,
                       groups, cols, static_cast<uint16_t*>(a.dw), static_cast<uint16_t*>(a.db));
}

}  // namespace fp8lin
