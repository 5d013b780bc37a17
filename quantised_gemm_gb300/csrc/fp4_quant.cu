// fp4_quant.cu -- quantisation of bf16 tensors to microscaled 4-bit floating
// point (NVFP4 and MXFP4), with the transposed copy a backward contracts
// over, and the way back.
//
//   NVFP4  blocks of 16 along the row.  With the tensorwise scale
//          S = fl32(448 / max(amax, eps)) that an e4m3 cast of the tensor
//          would use, the block's scale is the e4m3 cast of the block's
//          maximum, c = e4m3(fl32(b * S)), and a value's code is
//          q = e2m1(fl32(x * r)), r = fl32(fl32(6 * S) / c) (0 where c is 0).
//          The code stands for q * c * fl32(inv / 6), inv = fl32(1 / S).
//   MXFP4  blocks of 32 along the row, scale 2^(E - 127) with
//          E = max(e - 2, 0), e the exponent field of the block's maximum
//          (255 where it is an infinity or a NaN); q = e2m1(x * 2^(127 - E)).
//
// Every product and quotient is one fp32 rounding, and the conversions round
// to nearest even and saturate, so the bytes are defined bit for bit.  A NaN
// makes its block's scale NaN (0x7F, 0xFF); in NVFP4 a NaN or an infinity
// anywhere also makes the tensorwise scale NaN or 0, so every value decodes
// to NaN.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kQThreads = 256;
constexpr int kQTile = 128;       // tile: 128 rows x 128 columns
constexpr int kPitch = 66;        // words of a shared bf16 tile row (64 used)
constexpr int kOutPitch = 80;     // bytes of a staged row of transposed codes (64 used)

// Two fp32 -> two e2m1 codes in a byte (round to nearest even, saturating);
// lo in the low half.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b16 %0, {b, 0};\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
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
// bits).  s: the tensorwise scale, s6 = fl32(6 s) (NVFP4 only).
template <int kFmt>
__device__ __forceinline__ uint32_t block_scale(uint32_t max_bits, float s, float s6, float& r) {
  if constexpr (kFmt == 0) {
    const float b = __uint_as_float(max_bits << 16);
    const uint32_t c = cvt_fp8x2<0>(__fmul_rn(b, s), 0.0f) & 0xFFu;
    const float cf = e4m3_to_f32(c);
    r = c == 0 ? 0.0f : __fdiv_rn(s6, cf);
    return c;
  } else {
    const uint32_t e = max_bits >> 7;  // the sign bit is masked off
    const uint32_t E = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
    // 2^(127 - E): exponent field 254 - E, normal for every E up to 253.
    r = __uint_as_float((254u - (E < 253u ? E : 253u)) << 23);
    return E;
  }
}

// Eight values of a row as bf16 pairs: one 16-byte load, or element by
// element where the row ends inside it or the rows are not 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t col, int64_t cols) {
  if (kVec && col + 8 <= cols) return ld_stream_v4(row + col);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < cols) w[j >> 1] |= static_cast<uint32_t>(row[col + j]) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t absmax8(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

__device__ __forceinline__ uint32_t code2(uint32_t pair, float r) {
  float lo, hi;
  mul2_rn(pair << 16, pair & 0xFFFF0000u, r, lo, hi);
  return cvt_e2m1x2(lo, hi);
}

__device__ __forceinline__ uint32_t code8(const uint4& v, float r) {
  return code2(v.x, r) | (code2(v.y, r) << 8) | (code2(v.z, r) << 16) | (code2(v.w, r) << 24);
}

// The tensor's amax joins a maximum over the CTAs; the last one publishes it
// and clears both words for the next call.
__device__ __forceinline__ void join_amax(uint32_t bits, uint32_t* acc, uint32_t* ticket,
                                          uint32_t* out, uint32_t ctas) {
  atomicMax(acc, bits);
  __threadfence();
  if (atomicAdd(ticket, 1u) == ctas - 1u) {
    __threadfence();
    *out = atomicExch(acc, 0u);
    atomicExch(ticket, 0u);
  }
}

// Block-wide maximum of per-thread magnitude pairs, as fp32 bits in thread 0.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t pair) {
  __shared__ uint32_t red[kQThreads / 32];
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(pair & 0xFFFFu, pair >> 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  uint32_t all = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kQThreads / 32; ++w) all = max(all, red[w]);
  return all << 16;
}

struct QuantParams {
  const uint16_t* x;
  int64_t rows, cols, ld;
  const float* amax_in;    // NVFP4: derive the scale from this amax ...
  const float* scale_in;   // ... or use this one (delayed scaling)
  float eps;
  float* scale_out;        // with amax_in: written by CTA 0
  float* inv_out;
  uint32_t* amax_rec;      // delayed scaling: the tensor's amax, through the two words
  uint32_t* rec_acc;
  uint32_t* rec_ticket;
  uint8_t* codes;          // null: only the transposed copy
  uint8_t* scales;
  int64_t ld4;
  uint8_t* codes_t;
  uint8_t* scales_t;
  int64_t ld4_t;
  int64_t tiles_c;         // 128-column tiles of a row of tiles
};

// One 128 x 128 tile a CTA.  Bound by memory: 2 bytes read and 0.56 written
// an element and copy.  Each thread holds 16 consecutive values of four rows
// (rows 32 apart, so that its scale bytes are 16 consecutive bytes of a scale
// tile); the transposed copy reads the tile again from shared memory, 32 rows
// x 2 columns a thread, and stages its codes so that they leave 64 bytes a row.
template <int kFmt, bool kTrans, bool kVec>
__global__ void __launch_bounds__(kQThreads) fp4_quantise_kernel(const QuantParams p) {
  constexpr int kBlock = kFmt == 0 ? 16 : 32;
  constexpr int kTileBlocks = 4 * kBlock;  // columns of one 512-byte scale tile
  __shared__ __align__(16) uint32_t tile[kTrans ? kQTile * kPitch : 1];
  __shared__ __align__(16) uint8_t stage[kTrans ? kQTile * kOutPitch : 16];
  __shared__ __align__(16) uint8_t sc_stage[kTrans ? 1024 : 16];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  const int64_t row0 = tr * kQTile, col0 = tc * kQTile;
  float s = 0.0f, s6 = 0.0f;
  if constexpr (kFmt == 0) {
    s = p.amax_in != nullptr ? fp4_tensor_scale(*p.amax_in, p.eps) : *p.scale_in;
    s6 = __fmul_rn(6.0f, s);
    if (p.scale_out != nullptr && blockIdx.x == 0 && tid == 0) {
      *p.scale_out = s;
      *p.inv_out = __fdiv_rn(1.0f, s);
    }
  }
  const int b = lane & 7;                    // 16-column group of the tile
  const int rr = warp * 4 + (lane >> 3);     // row modulo 32
  const int64_t col = col0 + b * 16;
  uint4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + rr + 32 * i;
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (row < p.rows) {
      const uint16_t* src = p.x + row * p.ld;
      if (col < p.cols) v[i][0] = load8<kVec>(src, col, p.cols);
      if (col + 8 < p.cols) v[i][1] = load8<kVec>(src, col + 8, p.cols);
    }
  }
  if constexpr (kTrans) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t* dst = tile + (rr + 32 * i) * kPitch + b * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<uint2*>(dst + 4 * h) = make_uint2(v[i][h].x, v[i][h].y);
        *reinterpret_cast<uint2*>(dst + 4 * h + 2) = make_uint2(v[i][h].z, v[i][h].w);
      }
    }
  }
  uint32_t all = 0;
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m2 = absmax8(absmax8(0, v[i][0]), v[i][1]);
    if (p.amax_rec != nullptr) all = __vmaxu2(all, m2);
    if (p.codes == nullptr) continue;  // uniform
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if constexpr (kFmt == 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    float r;
    const uint32_t c = block_scale<kFmt>(m, s, s6, r);
    const int64_t row = row0 + rr + 32 * i;
    if (row < p.rows && col < ((p.cols + 31) & ~int64_t(31)))
      *reinterpret_cast<uint2*>(p.codes + row * p.ld4 + (col >> 1)) =
          make_uint2(code8(v[i][0], r), code8(v[i][1], r));
    // Four block scales of one scale tile's row, low block first.
    constexpr int kStep = kFmt == 0 ? 1 : 2;
    uint32_t w = c << (8 * ((b / kStep) & 3));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, kStep);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2 * kStep);
    word[i] = w;
  }
  if (p.codes != nullptr) {
    const int64_t nblk = (p.cols + kBlock - 1) / kBlock;
    const int64_t ktiles = (nblk + 3) >> 2;
    const int64_t kt = col / kTileBlocks;
    const bool first = kFmt == 0 ? (b & 3) == 0 : b == 0;
    if (first && kt < ktiles)
      *reinterpret_cast<uint4*>(p.scales + (tr * ktiles + kt) * 512 + rr * 16) =
          make_uint4(word[0], word[1], word[2], word[3]);
  }
  if constexpr (kTrans) {
    __syncthreads();
    const int pair = lane + 32 * (warp & 1);  // columns 2 pair, 2 pair + 1
    const int rg = warp >> 1;                 // rows 32 rg .. 32 rg + 31
    const uint32_t* src = tile + (rg * 32) * kPitch + pair;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = src[j * kPitch];
    uint32_t m2[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 32; ++j) m2[j >> 4] = __vmaxu2(m2[j >> 4], w[j] & 0x7FFF7FFFu);
    if constexpr (kFmt == 1) m2[0] = m2[1] = __vmaxu2(m2[0], m2[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the low column, then the high one
      uint32_t out[4];
      const int c = 2 * pair + h;
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // 16 rows each
        const uint32_t m = h == 0 ? m2[g] & 0xFFFFu : m2[g] >> 16;
        float r;
        const uint32_t sc = block_scale<kFmt>(m, s, s6, r);
        // transposed tile: row c, block 2 rg + g (NVFP4) or rg (MXFP4)
        const int blk = kFmt == 0 ? 2 * rg + g : rg;
        if (kFmt == 0 || g == 0)
          sc_stage[(blk >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (blk & 3)] =
              static_cast<uint8_t>(sc);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t word8 = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a = w[16 * g + 8 * q + 2 * j], d = w[16 * g + 8 * q + 2 * j + 1];
            // rows 2j and 2j + 1 of this column side by side
            word8 |= code2(__byte_perm(a, d, h == 0 ? 0x5410 : 0x7632), r) << (8 * j);
          }
          out[2 * g + q] = word8;
        }
      }
      *reinterpret_cast<uint4*>(stage + c * kOutPitch + rg * 16) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
    const int64_t code_bytes = ((p.rows + 31) >> 5) << 4;  // of a transposed row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = (tid >> 2) + 64 * i, chunk = tid & 3;
      const int64_t byte = (row0 >> 1) + chunk * 16;
      if (col0 + c < p.cols && byte < code_bytes)
        *reinterpret_cast<uint4*>(p.codes_t + (col0 + c) * p.ld4_t + byte) =
            *reinterpret_cast<const uint4*>(stage + c * kOutPitch + chunk * 16);
    }
    constexpr int kScTiles = kFmt == 0 ? 2 : 1;
    if (tid < 32 * kScTiles) {
      const int64_t nblk = (p.rows + kBlock - 1) / kBlock;
      const int64_t ktiles = (nblk + 3) >> 2;
      const int64_t kt = tr * kScTiles + (tid >> 5);
      if (kt < ktiles)
        *reinterpret_cast<uint4*>(p.scales_t + (tc * ktiles + kt) * 512 + (tid & 31) * 16) =
            *reinterpret_cast<const uint4*>(sc_stage + tid * 16);
    }
  }
  if (p.amax_rec != nullptr) {
    const uint32_t bits = block_max_bits(all);
    if (tid == 0) join_amax(bits, p.rec_acc, p.rec_ticket, p.amax_rec, gridDim.x);
  }
}

// max |x| of a tensor whose rows are not whole aligned vectors.
__global__ void __launch_bounds__(kQThreads)
    fp4_amax_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, uint32_t* acc,
                    uint32_t* ticket, uint32_t* out) {
  griddep_wait();
  griddep_launch_dependents();
  uint32_t m = 0;
  const int warps = gridDim.x * (kQThreads / 32);
  const int lane = threadIdx.x & 31;
  for (int64_t r = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps)
    for (int64_t c = lane; c < cols; c += 32) m = max(m, x[r * ld + c] & 0x7FFFu);
  const uint32_t bits = block_max_bits(m);
  if (threadIdx.x == 0) join_amax(bits, acc, ticket, out, gridDim.x);
}

// Codes back to values: 16 values a thread.
template <int kFmt, typename Out, bool kVec>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantise_kernel(const uint8_t* codes, const uint8_t* scales, const float* inv,
                          int64_t rows, int64_t cols, int64_t ld4, Out* out, int64_t ldo) {
  constexpr int kBlock = kFmt == 0 ? 16 : 32;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t groups = (cols + 15) >> 4;
  const int64_t ktiles = ((cols + kBlock - 1) / kBlock + 3) >> 2;
  const float d = kFmt == 0 ? __fdiv_rn(*inv, 6.0f) : 1.0f;
  const int64_t total = rows * groups;
  for (int64_t i = blockIdx.x * int64_t(kQThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kQThreads) {
    const int64_t row = i / groups, g = i - row * groups;
    const int64_t blk = g * 16 / kBlock;
    const uint32_t code = scales[((row >> 7) * ktiles + (blk >> 2)) * 512 + (row & 31) * 16 +
                                 ((row >> 5) & 3) * 4 + (blk & 3)];
    float c;
    if constexpr (kFmt == 0)
      c = e4m3_to_f32(code);
    else  // 2^(code - 127): 0 is the subnormal 2^-127, 255 a NaN
      c = code == 0 ? __uint_as_float(0x00400000u)
                    : __uint_as_float(code == 255 ? 0x7FC00000u : code << 23);
    const uint2 q = *reinterpret_cast<const uint2*>(codes + row * ld4 + g * 8);
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = f16x2_to_f32x2(cvt_f16x2_e2m1x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xFFu));
      v[2 * j] = __fmul_rn(f.x, c);
      v[2 * j + 1] = __fmul_rn(f.y, c);
      if constexpr (kFmt == 0) {
        v[2 * j] = __fmul_rn(v[2 * j], d);
        v[2 * j + 1] = __fmul_rn(v[2 * j + 1], d);
      }
    }
    Out* dst = out + row * ldo + g * 16;
    if (kVec && g * 16 + 16 <= cols) {
      if constexpr (sizeof(Out) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          reinterpret_cast<float4*>(dst)[j] =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          reinterpret_cast<uint4*>(dst)[j] = make_uint4(
              cvt_bf16x2(v[8 * j], v[8 * j + 1]), cvt_bf16x2(v[8 * j + 2], v[8 * j + 3]),
              cvt_bf16x2(v[8 * j + 4], v[8 * j + 5]), cvt_bf16x2(v[8 * j + 6], v[8 * j + 7]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (g * 16 + j < cols) {
          if constexpr (sizeof(Out) == 4)
            dst[j] = v[j];
          else
            dst[j] = static_cast<Out>(cvt_bf16x2(v[j], 0.0f) & 0xFFFFu);
        }
    }
  }
}

template <int kFmt, bool kTrans>
cudaError_t launch_quant(const QuantParams& p, unsigned grid, bool vec, cudaStream_t stream) {
  return vec ? launch_kernel(fp4_quantise_kernel<kFmt, kTrans, true>, dim3(grid), dim3(kQThreads), 0,
                             stream, 1, false, p)
             : launch_kernel(fp4_quantise_kernel<kFmt, kTrans, false>, dim3(grid), dim3(kQThreads),
                             0, stream, 1, false, p);
}

bool rows_vectorised(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem) % 16 == 0;
}

}  // namespace

cudaError_t launch_fp4_amax(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                            uint32_t* acc, uint32_t* ticket, uint32_t* out, const DeviceInfo& dev,
                            cudaStream_t stream) {
  const int64_t want = (rows + 7) / 8, most = 8 * int64_t(dev.num_sms);
  const unsigned grid = static_cast<unsigned>(want < most ? want : most);
  set_error_site("fp4_amax_kernel");
  return launch_kernel(fp4_amax_kernel, dim3(grid), dim3(kQThreads), 0, stream, 1, false, x, rows,
                       cols, ld, acc, ticket, out);
}

cudaError_t launch_fp4_quantise(const Fp4QuantArgs& a, cudaStream_t stream) {
  QuantParams p;
  p.x = a.x;
  p.rows = a.rows;
  p.cols = a.cols;
  p.ld = a.ld;
  p.amax_in = a.amax_in;
  p.scale_in = a.scale_in;
  p.eps = a.eps;
  p.scale_out = a.scale_out;
  p.inv_out = a.inv_out;
  p.amax_rec = a.amax_rec;
  p.rec_acc = a.rec_acc;
  p.rec_ticket = a.rec_ticket;
  p.codes = a.out.codes;
  p.scales = a.out.scales;
  p.ld4 = a.out.ld;
  p.codes_t = a.out_t.codes;
  p.scales_t = a.out_t.scales;
  p.ld4_t = a.out_t.ld;
  p.tiles_c = (a.cols + kQTile - 1) / kQTile;
  const int64_t grid = (a.rows + kQTile - 1) / kQTile * p.tiles_c;
  const bool vec = rows_vectorised(a.x, a.ld, 2), trans = a.out_t.codes != nullptr;
  set_error_site("fp4_quantise_kernel");
  const unsigned g = static_cast<unsigned>(grid);
  if (a.fmt == 0)
    return trans ? launch_quant<0, true>(p, g, vec, stream) : launch_quant<0, false>(p, g, vec, stream);
  return trans ? launch_quant<1, true>(p, g, vec, stream) : launch_quant<1, false>(p, g, vec, stream);
}

cudaError_t launch_fp4_dequantise(const Fp4View& t, int fmt, const float* inv, int64_t rows,
                                  int64_t cols, void* out, int64_t ldo, bool f32,
                                  const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t want = (rows * ((cols + 15) / 16) + kQThreads - 1) / kQThreads;
  const int64_t most = 16 * int64_t(dev.num_sms);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(kQThreads);
  const bool vec = rows_vectorised(out, ldo, f32 ? 4 : 2);
  set_error_site("fp4_dequantise_kernel");
#define FP8LIN_DEQUANT(FMT, OUT, VEC)                                                            \
  launch_kernel(fp4_dequantise_kernel<FMT, OUT, VEC>, grid, block, 0, stream, 1, false,          \
                static_cast<const uint8_t*>(t.codes), static_cast<const uint8_t*>(t.scales), inv, \
                rows, cols, t.ld, static_cast<OUT*>(out), ldo)
  if (fmt == 0) {
    if (f32) return vec ? FP8LIN_DEQUANT(0, float, true) : FP8LIN_DEQUANT(0, float, false);
    return vec ? FP8LIN_DEQUANT(0, uint16_t, true) : FP8LIN_DEQUANT(0, uint16_t, false);
  }
  if (f32) return vec ? FP8LIN_DEQUANT(1, float, true) : FP8LIN_DEQUANT(1, float, false);
  return vec ? FP8LIN_DEQUANT(1, uint16_t, true) : FP8LIN_DEQUANT(1, uint16_t, false);
#undef FP8LIN_DEQUANT
}

}  // namespace fp8lin
