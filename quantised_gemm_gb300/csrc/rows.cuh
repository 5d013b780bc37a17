// rows.cuh -- eight consecutive bf16 values of a row a thread, at any alignment.
//
// A row may begin at any multiple of two bytes.  A thread then reads the two
// aligned 16-byte vectors that its values lie in and shifts them into place
// (the second is its neighbour's first, so it comes from L1), and a warp
// writes aligned vectors again, each of its own values and its neighbour's.
// An aligned vector that holds a value of the tensor lies in memory that may
// be read, whatever its other bytes belong to.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace fp8lin {

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16lo_to_f32(w[j]);
    v[2 * j + 1] = bf16hi_to_f32(w[j]);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&v)[8]) {
  return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                    cvt_bf16x2(v[6], v[7]));
}

// Values off .. off + 7 of the sixteen in lo, hi.
__device__ __forceinline__ uint4 shift_values(const uint4& lo, const uint4& hi, uint32_t off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 4u) {
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
  }
  if (off & 2u) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  if (off & 1u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first n of eight values, the others 0.
__device__ __forceinline__ uint4 first_values(uint4 u, int n) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n <= 2 * j) w[j] = 0;
    if (n == 2 * j + 1) w[j] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// How many of the eight values from column c on lie in a row of `cols`.
__device__ __forceinline__ int values_at(int c, int cols) {
  return min(max(cols - c, 0), 8);
}

// The 16 bytes at p, or zeros, without a branch: loads in branches wait for one
// another at the join.
__device__ __forceinline__ uint4 load_if(const void* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<int>(on)));
  return v;
}

// Copies of 16 bytes to shared memory that are on their way while the thread goes
// on; on = false writes zeros.  Slots that only one thread writes and reads need
// no barrier but that thread's own wait.  Registers loaded ahead wait for one
// another where they share one of the warp's few scoreboards; these do not.
__device__ __forceinline__ void copy16(void* to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The n values at p, the others 0.  kAligned: p is 16-byte aligned and n 0 or 8.
template <bool kAligned>
__device__ __forceinline__ uint4 load_values(const uint16_t* p, int n) {
  if constexpr (kAligned) {
    return load_if(p, n > 0);
  } else {
    const uint32_t off = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u) >> 1;
    const uint4* v = reinterpret_cast<const uint4*>(p - off);
    const uint4 lo = load_if(v, n > 0), hi = load_if(v + 1, n > 0 && static_cast<int>(off) + n > 8);
    return first_values(shift_values(lo, hi, off), n);
  }
}

__device__ __forceinline__ uint16_t value_of(const uint4& u, int i) {
  const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
  return static_cast<uint16_t>(i & 1 ? w >> 16 : w & 0xFFFFu);
}

// The first n of the eight values to p, whose n-th place is 16-byte aligned (n < 8).
__device__ __forceinline__ void store_head(uint16_t* p, const uint4& u, int n) {
  const uint4 none = make_uint4(0, 0, 0, 0);
  if (n & 1) *p = static_cast<uint16_t>(u.x);
  const uint4 v = shift_values(u, none, n & 1);
  p += n & 1;
  if (n & 2) *reinterpret_cast<uint32_t*>(p) = v.x;
  const uint4 w = shift_values(v, none, n & 2);
  p += n & 2;
  if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
}

// The last n of the eight values to p, which is 16-byte aligned (n < 8).
__device__ __forceinline__ void store_tail(uint16_t* p, const uint4& u, int n) {
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 v = shift_values(u, none, static_cast<uint32_t>(8 - n) & 7u);
  if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
  v = shift_values(v, none, n & 4);
  p += n & 4;
  if (n & 2) *reinterpret_cast<uint32_t*>(p) = v.x;
  v = shift_values(v, none, n & 2);
  p += n & 2;
  if (n & 1) *p = static_cast<uint16_t>(v.x);
}

// What an unaligned lane writes of its n values at p and of the n_before ones before
// them (its neighbour's, at p - 8): the aligned vector that ends its neighbour's and
// begins its own.  off: values of the neighbour's in it.
__device__ __forceinline__ void store_joined(uint16_t* p, const uint4& u, int n, const uint4& before,
                                             int n_before, int off) {
  const int own = 8 - off;
  if (off == 0 && n == 8) {
    *reinterpret_cast<uint4*>(p) = u;
  } else if (off != 0 && n_before == 8 && n >= own) {
    *reinterpret_cast<uint4*>(p - off) = shift_values(before, u, own);
  } else {
    if (off != 0 && n >= own)
      store_head(p, u, own);
    else
      for (int i = 0; i < own && i < n; ++i) p[i] = value_of(u, i);
    if (off != 0 && n_before == 8)
      store_tail(p - off, before, off);
    else
      for (int i = own; i < n_before; ++i) p[i - 8] = value_of(before, i);
  }
}

// The values of a span's last lane that no lane behind it writes.
__device__ __forceinline__ void store_rest(uint16_t* p, const uint4& u, int n, int off) {
  if (off != 0 && n == 8)
    store_tail(p + 8 - off, u, off);
  else
    for (int i = 8 - off; i < n; ++i) p[i] = value_of(u, i);
}

__device__ __forceinline__ int misaligned_values(const void* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
}

// The lanes' values to p, n of them each, in spans of kSpan lanes: a lane's p lies
// 16 bytes behind that of the lane before it in the span, and no lane has values
// where one before it has fewer than eight.  All lanes of the warp call it.
template <bool kAligned, int kSpan = 32>
__device__ __forceinline__ void store_values(uint16_t* p, const uint4& u, int n) {
  if constexpr (kAligned) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = u;
  } else {
    const int off = misaligned_values(p), lane = static_cast<int>(threadIdx.x) & (kSpan - 1);
    uint4 before;
    before.x = __shfl_up_sync(0xFFFFFFFFu, u.x, 1, kSpan);
    before.y = __shfl_up_sync(0xFFFFFFFFu, u.y, 1, kSpan);
    before.z = __shfl_up_sync(0xFFFFFFFFu, u.z, 1, kSpan);
    before.w = __shfl_up_sync(0xFFFFFFFFu, u.w, 1, kSpan);
    const int n_before = __shfl_up_sync(0xFFFFFFFFu, n, 1, kSpan);
    store_joined(p, u, n, before, lane > 0 ? n_before : 0, off);
    if (lane == kSpan - 1) store_rest(p, u, n, off);
  }
}

// As store_values for unaligned rows whose spans follow one another: a span's first
// lane also has the last values of the call before, and the last lane's stay in the
// run until the next call or end().  n values a lane, 8 but at a row's end.
template <int kSpan>
struct StoreRun {
  uint4 kept = make_uint4(0, 0, 0, 0);
  int n_kept = 0;
  uint16_t* last = nullptr;

  __device__ __forceinline__ void store(uint16_t* p, const uint4& u, int n) {
    const int lane = static_cast<int>(threadIdx.x) & (kSpan - 1);
    // The lane before, or for the first one the last one's values of before.
    const bool give = lane == kSpan - 1;
    const int from = lane == 0 ? kSpan - 1 : lane - 1;
    const uint4 mine = give ? kept : u;
    uint4 before;
    before.x = __shfl_sync(0xFFFFFFFFu, mine.x, from, kSpan);
    before.y = __shfl_sync(0xFFFFFFFFu, mine.y, from, kSpan);
    before.z = __shfl_sync(0xFFFFFFFFu, mine.z, from, kSpan);
    before.w = __shfl_sync(0xFFFFFFFFu, mine.w, from, kSpan);
    const int n_before = __shfl_sync(0xFFFFFFFFu, give ? n_kept : n, from, kSpan);
    store_joined(p, u, n, before, n_before, misaligned_values(p));
    kept = u;
    n_kept = n;
    last = p;
  }
  __device__ __forceinline__ void end() const {
    if ((static_cast<int>(threadIdx.x) & (kSpan - 1)) != kSpan - 1 || last == nullptr) return;
    store_rest(last, kept, n_kept, misaligned_values(last));
  }
};

// Eight parameters (bf16 or fp32) from p on, n of them in the tensor.
template <typename P>
__device__ __forceinline__ void load_params(const P* p, int n, float (&v)[8]) {
  constexpr bool kBf16 = sizeof(P) == 2;
  if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    const uint4 a = __ldg(q);
    if constexpr (kBf16) {
      bf16x8_to_f32(a, v);
    } else {
      const uint4 b = __ldg(q + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < n) {
      if constexpr (kBf16)
        v[j] = bf16lo_to_f32(p[j]);
      else
        v[j] = p[j];
    }
  }
}

}  // namespace fp8lin
