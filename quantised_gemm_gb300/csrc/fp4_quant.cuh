// fp4_quant.cuh -- the steps of quantising 16 values of a row to 4 bits,
// shared by the quantisation kernels and the products that quantise their
// tokens on the way.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace fp8lin {
namespace {

// Eight fp32 -> eight e2m1 codes (round to nearest even, saturating), v[0] in
// the lowest four bits.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The larger magnitude of two bf16 pairs, each half with a sign that means
// nothing; a NaN wins.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two e2m1 codes in the low byte of v -> f16x2 (exact), low half first.
__device__ __forceinline__ uint32_t cvt_f16x2_e2m1x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, z;\n\t"
      "mov.b16 {b, z}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(v)));
  return r;
}

// e4m3 code -> fp32 (exact).
__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.f32.f16 %0, lo;\n\t}"
      : "=f"(f)
      : "r"(h));
  return f;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The tensorwise scale from the amax; a NaN amax gives a NaN scale.
__device__ __forceinline__ float fp4_tensor_scale(float amax, float eps) {
  return __fdiv_rn(448.0f, amax < eps ? eps : amax);
}

// Scale code and multiplier of one block from its maximum magnitude (bf16
// bits).  NVFP4: s is the tensorwise scale, and table holds the 128
// multipliers fl32(fl32(6 s) / c).
template <int kFmt>
__device__ __forceinline__ uint32_t block_scale(uint32_t max_bits, float s, const float* table,
                                                float& r) {
  if constexpr (kFmt == 0) {
    const uint32_t c = cvt_fp8x2<0>(__fmul_rn(__uint_as_float(max_bits << 16), s), 0.0f) & 0xFFu;
    r = table[c];
    return c;
  } else {
    const uint32_t e = max_bits >> 7;  // the sign bit is masked off
    const uint32_t E = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
    // 2^(127 - E): exponent field 254 - E, normal for every E up to 253.
    r = __uint_as_float((254u - (E < 253u ? E : 253u)) << 23);
    return E;
  }
}

// How a tensor's rows lie: every 16 values 32-byte aligned, 16-byte aligned,
// or neither.
enum RowAlign : int { kScalar = 0, kAlign16 = 1, kAlign32 = 2 };

// Eight values of a row as bf16 pairs: one 16-byte load, or element by
// element where the row ends inside it or the rows are not 16-byte aligned.
template <int kAlign>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t col, int64_t cols) {
  if (kAlign != kScalar && col + 8 <= cols) return ld_stream_v4(row + col);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < cols) w[j >> 1] |= static_cast<uint32_t>(row[col + j]) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sixteen values at p from the three aligned 16-byte vectors that they lie in;
// zero from the left-th on.
__device__ __forceinline__ void load16_shifted(const uint16_t* p, int64_t left, uint4 (&v)[2]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4* vec = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
  const uint4 a = __ldg(vec), b = __ldg(vec + 1), c = __ldg(vec + 2);
  uint32_t w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  const bool two = (at & 8) != 0, one = (at & 4) != 0;
#pragma unroll
  for (int j = 0; j < 10; ++j) w[j] = two ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 9; ++j) w[j] = one ? w[j + 1] : w[j];
  const uint32_t half = (at & 2) != 0 ? 16u : 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], half);
  if (left < 16) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = left >= 2 * j + 2 ? w[j] : left == 2 * j + 1 ? w[j] & 0xFFFFu : 0u;
  }
  v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  v[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Where the bytes of a tensor begin and end.
struct Span {
  const uint16_t* begin;
  const uint16_t* end;
};
__host__ __device__ __forceinline__ Span span_of(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld) {
  return {x, x + (rows - 1) * ld + cols};
}

// Sixteen values of a row (zero past its end): whole 32-byte sectors with one
// load where they are aligned; where rows are not, by the aligned vectors
// around them as long as these lie within the tensor.
template <int kAlign>
__device__ __forceinline__ void load16(const uint16_t* row, int64_t col, int64_t cols, const Span& in,
                                       uint4 (&v)[2]) {
  if (kAlign == kScalar) {
    const uint16_t* p = row + col;
    const uintptr_t low = reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15);
    if (low >= reinterpret_cast<uintptr_t>(in.begin) && low + 48 <= reinterpret_cast<uintptr_t>(in.end)) {
      load16_shifted(p, cols - col, v);
      return;
    }
  }
  if (kAlign == kAlign32 && col + 16 <= cols) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                   "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                 : "l"(row + col));
    return;
  }
  v[0] = v[1] = make_uint4(0, 0, 0, 0);
  if (col < cols) v[0] = load8<kAlign>(row, col, cols);
  if (col + 8 < cols) v[1] = load8<kAlign>(row, col + 8, cols);
}

__device__ __forceinline__ uint32_t max8(const uint4& v) {
  return max_magnitude(max_magnitude(v.x, v.y), max_magnitude(v.z, v.w));
}

// The magnitude bits of the larger half of a pair.
__device__ __forceinline__ uint32_t larger_half(uint32_t pair) {
  return max(pair & 0x7FFFu, (pair >> 16) & 0x7FFFu);
}

// One half of a bf16 pair times r in fp32.  The widening is an addition of -0
// in mixed precision, which keeps zeros' signs and leaves the integer pipe to
// the conversions; MXFP4's powers of two are bf16 numbers, so there the
// product is part of it, and exact.
template <int kFmt, int kHalf>
__device__ __forceinline__ float widen(uint32_t pair, float r) {
  float f;
  if constexpr (kFmt == 0) {
    if constexpr (kHalf == 0)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, lo, %2;\n\t}"
          : "=f"(f)
          : "r"(pair), "f"(-0.0f));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.bf16 %0, hi, %2;\n\t}"
          : "=f"(f)
          : "r"(pair), "f"(-0.0f));
  } else {
    const uint16_t m = static_cast<uint16_t>(__float_as_uint(r) >> 16);
    if constexpr (kHalf == 0)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tfma.rn.f32.bf16 %0, lo, %2, %3;\n\t}"
          : "=f"(f)
          : "r"(pair), "h"(m), "f"(-0.0f));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tfma.rn.f32.bf16 %0, hi, %2, %3;\n\t}"
          : "=f"(f)
          : "r"(pair), "h"(m), "f"(-0.0f));
  }
  return f;
}

template <int kFmt>
__device__ __forceinline__ uint32_t codes_of(float (&f)[8], float r) {
  if constexpr (kFmt == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mul2_rn(__float_as_uint(f[2 * j]), __float_as_uint(f[2 * j + 1]), r, f[2 * j], f[2 * j + 1]);
  }
  return cvt_e2m1x8(f);
}

template <int kFmt>
__device__ __forceinline__ uint32_t code8(const uint4& v, float r) {
  float f[8] = {widen<kFmt, 0>(v.x, r), widen<kFmt, 1>(v.x, r), widen<kFmt, 0>(v.y, r),
                widen<kFmt, 1>(v.y, r), widen<kFmt, 0>(v.z, r), widen<kFmt, 1>(v.z, r),
                widen<kFmt, 0>(v.w, r), widen<kFmt, 1>(v.w, r)};
  return codes_of<kFmt>(f, r);
}

// Eight values, one from each word: its low or its high half.
template <int kFmt, int kHalf>
__device__ __forceinline__ uint32_t code8_of(const uint32_t* w, float r) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = widen<kFmt, kHalf>(w[j], r);
  return codes_of<kFmt>(f, r);
}

// The multipliers fl32(fl32(6 s) / c) of the 128 block scales, 0 for c = 0.
__device__ __forceinline__ void fill_table(float s, float* table) {
  if (threadIdx.x < 128)
    table[threadIdx.x] =
        threadIdx.x == 0 ? 0.0f : __fdiv_rn(__fmul_rn(6.0f, s), e4m3_to_f32(threadIdx.x));
}

int row_align(const void* p, int64_t ld, int elem) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * elem);
  return (bits & 31u) == 0 ? kAlign32 : (bits & 15u) == 0 ? kAlign16 : kScalar;
}

}  // namespace
}  // namespace fp8lin
