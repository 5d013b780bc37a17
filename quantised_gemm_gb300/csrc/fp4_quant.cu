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
// makes its block's scale NaN (0x7F, 0xFF).  In NVFP4 a NaN or an infinity
// also makes a tensorwise scale of the tensor's own amax NaN or 0, so every
// value decodes to NaN; beside a scale from elsewhere an infinity saturates.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fp4_quant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kQThreads = 256;
constexpr int kQTile = 128;       // tile: 128 rows x 128 columns
constexpr int kPitch = 68;        // words of a shared bf16 tile row (64 used)

// Thirty-two aligned bytes in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
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

struct QuantParams {
  const uint16_t* x;
  Span span;
  int64_t rows, cols, ld;
  // NVFP4's tensorwise scale: from the maximum of the amax kernel's partials,
  // from an amax, or (delayed scaling) as it is.
  const uint32_t* partials;
  int num_partials;
  const float* amax_in;
  const float* scale_in;
  const float* inv_in;
  float eps;
  float* amax_out;         // each may be null; written by the tensor's first CTA
  float* scale_out;
  float* inv_out;
  float* own_inv;          // of the tensor and its transposed copy
  float* own_inv_t;
  uint32_t* amax_rec;      // delayed scaling: the tensor's amax, through the two words
  uint32_t* rec_acc;
  uint32_t* rec_ticket;
  uint8_t* codes;          // null: only the transposed copy
  uint8_t* scales;
  int64_t ld4;
  uint8_t* codes_t;
  uint8_t* scales_t;
  int64_t ld4_t;
  uint32_t tiles_c;        // 128-column tiles of a row of tiles
  uint32_t tiles;
};
struct QuantPair {
  QuantParams p[2];        // the second tensor's tiles follow the first's
};

template <int kFmt, bool kTrans>
struct QuantSmem {
  uint32_t tile[kTrans ? kQTile * kPitch : 4];
  uint8_t stage[kTrans ? kQTile * 64 : 16];
  uint8_t scales[kTrans ? 1024 : 16];
  float table[kFmt == 0 ? 128 : 4];  // multiplier of each block scale
  uint32_t red[kQThreads / 32];
};

// This thread's part of a tile: 16 values of four rows, 32 rows apart.
template <int kAlign>
__device__ __forceinline__ void load_tile(const QuantParams& p, uint32_t tr, uint32_t tc,
                                          uint4 (&v)[4][2]) {
  const int lane = threadIdx.x & 31, rr = (threadIdx.x >> 5) * 4 + (lane >> 3);
  const int64_t col = int64_t(tc) * kQTile + (lane & 7) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = int64_t(tr) * kQTile + rr + 32 * i;
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    if (row < p.rows) load16<kAlign>(p.x + row * p.ld, col, p.cols, p.span, v[i]);
  }
}

// The block's maximum of per-thread bits, in every thread.
__device__ __forceinline__ uint32_t block_max(uint32_t bits, uint32_t* red) {
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, bits);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  uint32_t all = red[0];
#pragma unroll
  for (int w = 1; w < kQThreads / 32; ++w) all = max(all, red[w]);
  return all;
}

// State of a dynamically scaled tensor, and the inverse scale that the copies
// keep for themselves.
__device__ __forceinline__ void write_state(const QuantParams& p, float amax, float s) {
  const float inv = p.scale_in != nullptr ? *p.inv_in : __fdiv_rn(1.0f, s);
  if (p.amax_out != nullptr) *p.amax_out = amax;
  if (p.scale_out != nullptr) {
    *p.scale_out = s;
    *p.inv_out = inv;
  }
  if (p.own_inv != nullptr) *p.own_inv = inv;
  if (p.own_inv_t != nullptr) *p.own_inv_t = inv;
}

// The codes and scales of one tile held in v.
// sm.table is filled; the call synchronises before it reads it.
template <int kFmt, bool kTrans>
__device__ __forceinline__ void quantise_tile(const QuantParams& p, uint32_t tr, uint32_t tc,
                                              float s, const uint4 (&v)[4][2],
                                              QuantSmem<kFmt, kTrans>& sm) {
  constexpr int kBlock = kFmt == 0 ? 16 : 32;
  constexpr int kTileBlocks = 4 * kBlock;  // columns of one 512-byte scale tile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = int64_t(tr) * kQTile, col0 = int64_t(tc) * kQTile;
  const int b = lane & 7;                    // 16-column group of the tile
  const int rr = warp * 4 + (lane >> 3);     // row modulo 32
  const int64_t col = col0 + b * 16;
  if constexpr (kTrans) {
    const int flip = b >> 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t* dst = sm.tile + (rr + 32 * i) * kPitch + b * 8;
      *reinterpret_cast<uint4*>(dst + 4 * flip) = flip ? v[i][1] : v[i][0];
      *reinterpret_cast<uint4*>(dst + 4 * (flip ^ 1)) = flip ? v[i][0] : v[i][1];
    }
  }
  if constexpr (kTrans || kFmt == 0) __syncthreads();
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.codes == nullptr) break;  // uniform
    uint32_t m = larger_half(max_magnitude(max8(v[i][0]), max8(v[i][1])));
    if constexpr (kFmt == 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    float r;
    const uint32_t c = block_scale<kFmt>(m, s, sm.table, r);
    const int64_t row = row0 + rr + 32 * i;
    if (row < p.rows && col < ((p.cols + 31) & ~int64_t(31)))
      *reinterpret_cast<uint2*>(p.codes + row * p.ld4 + (col >> 1)) =
          make_uint2(code8<kFmt>(v[i][0], r), code8<kFmt>(v[i][1], r));
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
      *reinterpret_cast<uint4*>(p.scales + (int64_t(tr) * ktiles + kt) * 512 + rr * 16) =
          make_uint4(word[0], word[1], word[2], word[3]);
  }
  if constexpr (kTrans) {
    const int pair = lane + 32 * (warp & 1);  // columns 2 pair, 2 pair + 1
    const int rg = warp >> 1;                 // rows 32 rg .. 32 rg + 31
    const uint32_t* src = sm.tile + (rg * 32) * kPitch + pair;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = src[j * kPitch];
    uint32_t m2[2] = {w[0], w[16]};
#pragma unroll
    for (int j = 1; j < 16; ++j) {
      m2[0] = max_magnitude(m2[0], w[j]);
      m2[1] = max_magnitude(m2[1], w[16 + j]);
    }
    if constexpr (kFmt == 1) m2[0] = m2[1] = max_magnitude(m2[0], m2[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the low column, then the high one
      uint32_t out[4];
      const int c = 2 * pair + h;
      float r = 0.0f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // 16 rows each
        if (kFmt == 0 || g == 0) {
          const uint32_t sc = block_scale<kFmt>((h == 0 ? m2[g] : m2[g] >> 16) & 0x7FFFu, s, sm.table, r);
          // transposed tile: row c, block 2 rg + g (NVFP4) or rg (MXFP4)
          const int blk = kFmt == 0 ? 2 * rg + g : rg;
          sm.scales[(blk >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (blk & 3)] =
              static_cast<uint8_t>(sc);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          out[2 * g + q] = h == 0 ? code8_of<kFmt, 0>(w + 16 * g + 8 * q, r)
                                  : code8_of<kFmt, 1>(w + 16 * g + 8 * q, r);
      }
      *reinterpret_cast<uint4*>(sm.stage + pair * 128 + (((h * 4 + rg) ^ (pair & 7)) << 4)) =
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
            *reinterpret_cast<const uint4*>(
                sm.stage + (c >> 1) * 128 + ((((c & 1) * 4 + chunk) ^ ((c >> 1) & 7)) << 4));
    }
    constexpr int kScTiles = kFmt == 0 ? 2 : 1;
    if (tid < 32 * kScTiles) {
      const int64_t nblk = (p.rows + kBlock - 1) / kBlock;
      const int64_t ktiles = (nblk + 3) >> 2;
      const int64_t kt = int64_t(tr) * kScTiles + (tid >> 5);
      if (kt < ktiles)
        *reinterpret_cast<uint4*>(p.scales_t + (int64_t(tc) * ktiles + kt) * 512 + (tid & 31) * 16) =
            *reinterpret_cast<const uint4*>(sm.scales + tid * 16);
    }
  }
}

// Tile t of a tensor; kRecord: with its amax for delayed scaling, where the
// tensor has that.
template <int kFmt, bool kTrans, int kAlign, bool kRecord>
__device__ __forceinline__ void quantise_cta(const QuantParams& p, uint32_t t,
                                             QuantSmem<kFmt, kTrans>& sm) {
  const uint32_t tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
  uint4 v[4][2];
  load_tile<kAlign>(p, tr, tc, v);
  float s = 0.0f;
  if constexpr (kFmt == 0) {
    float amax = 0.0f;
    if (p.partials != nullptr) {
      uint32_t m = 0;
      for (int i = threadIdx.x; i < p.num_partials; i += kQThreads) m = max(m, p.partials[i]);
      amax = __uint_as_float(block_max(m, sm.red) << 16);
    } else if (p.amax_in != nullptr) {
      amax = *p.amax_in;
    }
    s = p.scale_in != nullptr ? *p.scale_in : fp4_tensor_scale(amax, p.eps);
    fill_table(s, sm.table);
    if (t == 0 && threadIdx.x == 0) write_state(p, amax, s);
  }
  uint32_t m = 0;
  if (kRecord) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_magnitude(m, max_magnitude(max8(v[i][0]), max8(v[i][1])));
  }
  quantise_tile<kFmt, kTrans>(p, tr, tc, s, v, sm);
  if (kRecord && p.amax_rec != nullptr) {
    // Last: at the start the CTA's warps would wait for the atomics (65536 x
    // 4096: 106 us against 101).
    const uint32_t bits = block_max(larger_half(m), sm.red) << 16;
    if (threadIdx.x == 0) join_amax(bits, p.rec_acc, p.rec_ticket, p.amax_rec, p.tiles);
  }
}

// One 128 x 128 tile a CTA.  Bound by memory: 2 bytes read and 0.56 written
// an element and copy.  Each thread holds 16 consecutive values of four rows
// (rows 32 apart, so that its scale bytes are 16 consecutive bytes of a scale
// tile); the transposed copy reads the tile again from shared memory, 32 rows
// x 2 columns a thread, and stages its codes so that they leave 64 bytes a
// row.  Shared rows are 16 bytes longer than the tile's, and the halves of
// 32 bytes and the staged chunks are permuted, so that no access conflicts.
// 65536 x 4096, MXFP4: 95 us without the transposed copy, 7.2 TB/s; 133 us
// with it, 6.2 TB/s.  Smaller tensors ramp up and down for longer than they
// run at that rate: 14336 x 4096 33 us, 5.4 TB/s, four CTAs an SM that wait
// for their loads, the conversions (60 % of the issue slots) and each other.
// Every parameter is at a constant address, so the code stands once for each
// tensor, and a single one has a kernel without the second: with indexed
// parameters 14336 x 4096 (MXFP4, both copies) took 35.1 us instead of 33.3.
// The recording of an amax is a kernel of its own too.  Five CTAs an SM
// without the transposed copy: 65536 x 4096 (NVFP4) 99 us, 102 with four.
template <int kFmt, bool kTrans, int kAlign, bool kPair, bool kRecord>
__global__ void __launch_bounds__(kQThreads, kTrans || kPair || kAlign == kScalar ? 4 : 5)
    fp4_quantise_kernel(const __grid_constant__ QuantPair pair) {
  __shared__ __align__(16) QuantSmem<kFmt, kTrans> sm;
  griddep_wait();
  griddep_launch_dependents();
  if (!kPair || blockIdx.x < pair.p[0].tiles)
    quantise_cta<kFmt, kTrans, kAlign, kRecord>(pair.p[0], blockIdx.x, sm);
  else
    quantise_cta<kFmt, kTrans, kAlign, kRecord>(pair.p[1], blockIdx.x - pair.p[0].tiles, sm);
}

// Largest magnitudes (bf16 bits) of one or two tensors, one a CTA, for the
// quantisation to join: no atomics and no last CTA.  Bound by reading them:
// 65536 x 4096 in 91 us, 5.9 TB/s.
struct AmaxParams {
  const uint16_t* x;
  Span span;
  int64_t rows, cols, ld;
  uint32_t* partials;
  int ctas;
  int lanes_log2;  // lanes of a warp that share a row
};
struct AmaxPair {
  AmaxParams p[2];
};

// share_max() of a contiguous tensor, which is one row: no rows' arithmetic
// (16 x 4096 by one CTA: 1.4 us less).
template <int kAlign, int kLoads>
__device__ __forceinline__ uint32_t contiguous_max(const AmaxParams& p, int64_t first, int64_t warps) {
  uint32_t m2 = 0;
  const int64_t step = warps * 512;
  for (int64_t c = first * 512; c < p.cols; c += kLoads * step) {
    uint4 v[kLoads][2];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      const int64_t col = c + k * step + (threadIdx.x & 31) * 16;
      if (col < p.cols) load16<kAlign>(p.x, col, p.cols, p.span, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      m2 = max_magnitude(m2, max_magnitude(max8(v[k][0]), max8(v[k][1])));
  }
  return larger_half(m2);
}

// The largest magnitude of a thread's share of a tensor: warp `first` of
// `warps` takes 512 values at a time, kLoads of these in flight: of one row,
// or 16 values a lane of several narrow ones.
template <int kAlign, int kLoads>
__device__ __forceinline__ uint32_t share_max(const AmaxParams& p, int64_t first, int64_t warps) {
  const int lane = threadIdx.x & 31, lg = p.lanes_log2;
  if (p.rows == 1) {
    if (kAlign == kScalar && (reinterpret_cast<uintptr_t>(p.x) & 31u) == 0)
      return contiguous_max<kAlign32, kLoads>(p, first, warps);
    return contiguous_max<kAlign, kLoads>(p, first, warps);
  }
  const int64_t per_row = (p.cols + (16 << lg) - 1) >> (4 + lg);
  const int64_t total = ((p.rows + (32 >> lg) - 1) >> (5 - lg)) * per_row;
  const int own_row = lane >> lg, own_col = (lane & ((1 << lg) - 1)) * 16;
  uint32_t m2 = 0;
  for (int64_t i = first; i < total; i += kLoads * warps) {
    uint4 v[kLoads][2];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      const int64_t seg = i + k * warps;
      const int64_t group = per_row == 1 ? seg : seg / per_row;
      const int64_t row = (group << (5 - lg)) + own_row;
      if (seg < total && row < p.rows)
        load16<kAlign>(p.x + row * p.ld, ((seg - group * per_row) << (4 + lg)) + own_col, p.cols, p.span,
                       v[k]);
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      m2 = max_magnitude(m2, max_magnitude(max8(v[k][0]), max8(v[k][1])));
  }
  return larger_half(m2);
}

template <int kAlign>
__global__ void __launch_bounds__(kQThreads)
    fp4_amax_kernel(const __grid_constant__ AmaxPair pair) {
  __shared__ uint32_t red[kQThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  auto run = [&](const AmaxParams& p, int cta) {
    constexpr int kWarps = kQThreads / 32;
    const uint32_t m = share_max<kAlign, 4>(p, int64_t(cta) * kWarps + (threadIdx.x >> 5),
                                            int64_t(p.ctas) * kWarps);
    const uint32_t all = block_max(m, red);
    if (threadIdx.x == 0) p.partials[cta] = all;
  };
  const int cta = static_cast<int>(blockIdx.x);
  if (cta < pair.p[0].ctas)
    run(pair.p[0], cta);
  else
    run(pair.p[1], cta - pair.p[0].ctas);
}

// A small tensor with dynamic NVFP4 scaling in one launch: every CTA finds
// the whole tensor's maximum (from L2, but for the first) before it quantises
// its tile.  Bound by the launch and two round trips to memory: 16 x 4096 in
// 3.3 us back to back in a graph (two launches: 4.1), where a cluster of eight
// CTAs that join their maxima took 1.7 us more than this.
// What it costs is the scan, in segments of 512 values that a warp loads at a
// time, and every tile's CTA scans all of them.  In a graph and by a call from
// Python, against two launches: 24 x 4096 (192 segments, 32 tiles) 3.8 and 5.6
// us against 3.7 and 7.7, 1 x 32768 (64, 256 tiles) 3.6 and 5.8 against 3.7 and
// 7.6, but 4 x 24576 (192, 192 tiles) 4.6 against 3.7 and 1 x 98304 (192, 768
// tiles) 10.6 and 10.8 against 5.2 and 7.6.  Rows with a stride, or not aligned,
// cost more a segment: 128 x 256 in wider rows (64) 4.5 against 4.6, 16 x 4096
// in wider rows (128) 6.7 against 4.3, 310 x 310 (310) 20 against 7.7.
constexpr int64_t kSmallSegments = 192;
constexpr int64_t kSmallSegmentsStrided = 64;
constexpr int64_t kSmallScans = 24576;  // segments times tiles

template <bool kTrans, int kAlign>
__global__ void __launch_bounds__(kQThreads)
    fp4_quantise_small_kernel(const __grid_constant__ QuantParams p,
                              const __grid_constant__ AmaxParams a) {
  __shared__ __align__(16) QuantSmem<0, kTrans> sm;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  const uint32_t m = share_max<kAlign, 8>(a, threadIdx.x >> 5, kQThreads / 32);
  uint4 v[4][2];
  load_tile<kAlign>(p, tr, tc, v);
  const float amax = __uint_as_float(block_max(m, sm.red) << 16);
  const float s = fp4_tensor_scale(amax, p.eps);
  fill_table(s, sm.table);
  if (blockIdx.x == 0 && threadIdx.x == 0) write_state(p, amax, s);
  quantise_tile<0, kTrans>(p, tr, tc, s, v, sm);
}

// 2^(code - 127) of an MXFP4 scale: 0 is the subnormal 2^-127, 255 a NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7FC00000u : code << 23);
}

template <int kAlign>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
  if constexpr (kAlign == kAlign32) {
    store32(p, w);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Codes back to values: a 128 x 128 tile a CTA, 16 values of four rows a
// thread, whose scales are one 16-byte load.  Bound by memory: 14336 x 4096
// into bf16 in 24 us, 6.1 TB/s.
template <int kFmt, typename Out, int kAlign>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantise_kernel(const uint8_t* codes, const uint8_t* scales, const float* inv,
                          int64_t rows, int64_t cols, int64_t ld4, Out* out, int64_t ldo,
                          uint32_t tiles_c) {
  constexpr int kBlock = kFmt == 0 ? 16 : 32;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int b = lane & 7, rr = warp * 4 + (lane >> 3);
  const int64_t col = int64_t(tc) * kQTile + b * 16;
  if (col >= cols) return;
  const int64_t ktiles = ((cols + kBlock - 1) / kBlock + 3) >> 2;
  const uint4 sc = *reinterpret_cast<const uint4*>(
      scales + (int64_t(tr) * ktiles + col / (4 * kBlock)) * 512 + rr * 16);
  const int shift = 8 * (kFmt == 0 ? b & 3 : b >> 1);
  uint2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = int64_t(tr) * kQTile + rr + 32 * i;
    q[i] = row < rows ? *reinterpret_cast<const uint2*>(codes + row * ld4 + (col >> 1))
                      : make_uint2(0, 0);
  }
  const float d = kFmt == 0 ? __fdiv_rn(*inv, 6.0f) : 1.0f;
  const uint32_t words[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = int64_t(tr) * kQTile + rr + 32 * i;
    if (row >= rows) break;
    const uint32_t code = (words[i] >> shift) & 0xFFu;
    const float c = kFmt == 0 ? e4m3_to_f32(code) : e8m0_to_f32(code);
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = f16x2_to_f32x2(
          cvt_f16x2_e2m1x2(((j < 4 ? q[i].x : q[i].y) >> (8 * (j & 3))) & 0xFFu));
      mul2_rn(__float_as_uint(f.x), __float_as_uint(f.y), c, v[2 * j], v[2 * j + 1]);
      if constexpr (kFmt == 0)
        mul2_rn(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]), d, v[2 * j], v[2 * j + 1]);
    }
    Out* dst = out + row * ldo + col;
    if (col + 16 <= cols) {
      if constexpr (sizeof(Out) == 4) {
        uint32_t w[2][8];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j >> 3][j & 7] = __float_as_uint(v[j]);
        store_words<kAlign>(dst, w[0]);
        store_words<kAlign>(dst + 8, w[1]);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = cvt_bf16x2(v[2 * j], v[2 * j + 1]);
        store_words<kAlign>(dst, w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < cols) {
          if constexpr (sizeof(Out) == 4)
            dst[j] = v[j];
          else
            dst[j] = static_cast<Out>(cvt_bf16x2(v[j], 0.0f) & 0xFFFFu);
        }
    }
  }
}

// The same for rows that are not 16-byte aligned, 32 rows a CTA: the two
// values of a byte a lane.  Where their place is not aligned to the two of
// them (bf16), the second value of the lane before goes with the first.
// 8192 x 4095 in 34 us, bound by the instructions of its short stores (a value
// a lane: 38); 1009 x 1531 in 3.4 us (4.0), much of it the launch.
template <int kFmt, typename Out>
__global__ void __launch_bounds__(kQThreads)
    fp4_dequantise_ragged_kernel(const uint8_t* codes, const uint8_t* scales, const float* inv,
                                 int64_t rows, int64_t cols, int64_t ld4, Out* out, int64_t ldo,
                                 uint32_t tiles_c) {
  constexpr int kBlock = kFmt == 0 ? 16 : 32;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t ktiles = ((cols + kBlock - 1) / kBlock + 3) >> 2;
  constexpr int kSteps = kQTile / 64;
  uint32_t code[4][kSteps], q[4][kSteps];  // all loads in flight together
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = warp + 8 * i;
    const int64_t row = int64_t(tr) * 32 + r;
    const uint8_t* row_scales = scales + int64_t(tr >> 2) * ktiles * 512 + r * 16 + (tr & 3) * 4;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t col = int64_t(tc) * kQTile + 64 * j + 2 * lane, blk = col / kBlock;
      code[i][j] = q[i][j] = 0;
      if (row < rows && col < cols) {
        code[i][j] = __ldg(row_scales + (blk >> 2) * 512 + (blk & 3));
        q[i][j] = __ldg(codes + row * ld4 + (col >> 1));
      }
    }
  }
  const float d = kFmt == 0 ? __fdiv_rn(*inv, 6.0f) : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = int64_t(tr) * 32 + warp + 8 * i;
    if (row >= rows) break;
    Out* dst = out + row * ldo;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t col = int64_t(tc) * kQTile + 64 * j + 2 * lane;
      const bool live = col < cols, two = col + 1 < cols;
      const float2 f = f16x2_to_f32x2(cvt_f16x2_e2m1x2(q[i][j]));
      const float c = kFmt == 0 ? e4m3_to_f32(code[i][j]) : e8m0_to_f32(code[i][j]);
      float v0 = __fmul_rn(f.x, c), v1 = __fmul_rn(f.y, c);
      if constexpr (kFmt == 0) {
        v0 = __fmul_rn(v0, d);
        v1 = __fmul_rn(v1, d);
      }
      if constexpr (sizeof(Out) == 4) {
        if (two && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
          *reinterpret_cast<float2*>(dst + col) = make_float2(v0, v1);
        } else {
          if (live) dst[col] = v0;
          if (two) dst[col + 1] = v1;
        }
      } else {
        const uint32_t pair = cvt_bf16x2(v0, v1);
        if ((reinterpret_cast<uintptr_t>(dst) & 3u) == 0) {
          if (two)
            *reinterpret_cast<uint32_t*>(dst + col) = pair;
          else if (live)
            dst[col] = static_cast<Out>(pair & 0xFFFFu);
        } else {
          const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, pair, 1);
          if (live && lane > 0)
            *reinterpret_cast<uint32_t*>(dst + col - 1) = before >> 16 | pair << 16;
          else if (live)
            dst[col] = static_cast<Out>(pair & 0xFFFFu);
          if (two && (lane == 31 || col + 2 >= cols)) dst[col + 1] = static_cast<Out>(pair >> 16);
        }
      }
    }
  }
}

QuantParams quant_params(const Fp4QuantArgs& a) {
  QuantParams p = {};
  p.x = a.x;
  p.span = span_of(a.x, a.rows, a.cols, a.ld);
  p.rows = a.rows;
  p.cols = a.cols;
  p.ld = a.ld;
  p.amax_in = a.amax_in;
  p.scale_in = a.scale_in;
  p.inv_in = a.inv_in;
  p.eps = a.eps;
  p.amax_out = a.amax_out;
  p.scale_out = a.scale_out;
  p.inv_out = a.inv_out;
  p.own_inv = a.own_inv;
  p.own_inv_t = a.own_inv_t;
  p.amax_rec = a.amax_rec;
  p.rec_acc = a.rec_acc;
  p.rec_ticket = a.rec_ticket;
  p.codes = a.out.codes;
  p.scales = a.out.scales;
  p.ld4 = a.out.ld;
  p.codes_t = a.out_t.codes;
  p.scales_t = a.out_t.scales;
  p.ld4_t = a.out_t.ld;
  p.tiles_c = static_cast<uint32_t>((a.cols + kQTile - 1) / kQTile);
  p.tiles = static_cast<uint32_t>((a.rows + kQTile - 1) / kQTile) * p.tiles_c;
  return p;
}

// Contiguous rows are one long row to the amax.
AmaxParams amax_params(const Fp4QuantArgs& a) {
  AmaxParams p = {};
  const bool one = a.ld == a.cols;
  p.x = a.x;
  p.span = span_of(a.x, a.rows, a.cols, a.ld);
  p.rows = one ? 1 : a.rows;
  p.cols = one ? a.rows * a.cols : a.cols;
  p.ld = one ? 0 : a.ld;
  p.lanes_log2 = 5;
  while (p.lanes_log2 > 0 && p.cols <= (8 << p.lanes_log2)) --p.lanes_log2;
  return p;
}

// The warp's loads of 512 values that share_max() makes of a tensor.
int64_t scan_segments(const AmaxParams& p) {
  if (p.rows == 1) return (p.cols + 511) / 512;
  const int64_t per_row = (p.cols + (16 << p.lanes_log2) - 1) >> (4 + p.lanes_log2);
  return ((p.rows + (32 >> p.lanes_log2) - 1) >> (5 - p.lanes_log2)) * per_row;
}

template <int kFmt, bool kTrans, bool kPair, bool kRecord>
auto* quant_kernel(int align) {
  return align == kAlign32   ? fp4_quantise_kernel<kFmt, kTrans, kAlign32, kPair, kRecord>
         : align == kAlign16 ? fp4_quantise_kernel<kFmt, kTrans, kAlign16, kPair, kRecord>
                             : fp4_quantise_kernel<kFmt, kTrans, kScalar, kPair, kRecord>;
}

template <bool kTrans>
auto* small_kernel(int align) {
  return align == kAlign32   ? fp4_quantise_small_kernel<kTrans, kAlign32>
         : align == kAlign16 ? fp4_quantise_small_kernel<kTrans, kAlign16>
                             : fp4_quantise_small_kernel<kTrans, kScalar>;
}

}  // namespace

bool fp4_quantise_small_fits(const Fp4QuantArgs& a) {
  if (a.fmt != 0 || !a.find_amax) return false;
  const AmaxParams p = amax_params(a);
  const bool whole = p.rows == 1 && ((reinterpret_cast<uintptr_t>(a.x) & 31u) == 0 ||
                                     row_align(a.x, a.ld, 2) != kScalar);
  const int64_t segments = scan_segments(p);
  if (segments > (whole ? kSmallSegments : kSmallSegmentsStrided)) return false;
  return segments * (((a.rows + kQTile - 1) / kQTile) * ((a.cols + kQTile - 1) / kQTile)) <= kSmallScans;
}

cudaError_t launch_fp4_quantise_small(const Fp4QuantArgs& a, cudaStream_t stream) {
  const int align = row_align(a.x, a.ld, 2);
  const QuantParams p = quant_params(a);
  set_error_site("fp4_quantise_small_kernel");
  return launch_kernel(a.out_t.codes != nullptr ? small_kernel<true>(align) : small_kernel<false>(align),
                       dim3(static_cast<unsigned>(p.tiles)), dim3(kQThreads), 0, stream, 1, false, p,
                       amax_params(a));
}

cudaError_t launch_fp4_amax(const Fp4QuantArgs* a, int n, uint32_t* partials, int* num_partials,
                            const DeviceInfo& dev, cudaStream_t stream) {
  AmaxPair pair = {};
  int align = kAlign32, ctas = 0;
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += a[i].rows * a[i].cols;
  // Eight CTAs an SM over all tensors: 65536 x 4096 takes 91 us, with half the
  // CTAs and twice the loads in flight 100 us.
  const int64_t most = 8 * int64_t(dev.num_sms);
  for (int i = 0; i < n; ++i) {
    pair.p[i] = amax_params(a[i]);
    // A contiguous tensor needs only its base aligned: it is one row.
    const int own = row_align(a[i].x, pair.p[i].ld, 2);
    align = own < align ? own : align;
    const int64_t size = a[i].rows * a[i].cols;
    // Four segments a warp: 16384 values, or fewer in narrow rows.
    const int64_t want = (scan_segments(pair.p[i]) + 31) / 32, share = most * size / all + 1;
    pair.p[i].ctas = static_cast<int>(want < share ? want : share);
    pair.p[i].partials = partials + i * (kMaxPartials / 2);
    num_partials[i] = pair.p[i].ctas;
    ctas += pair.p[i].ctas;
  }
  auto* kernel = align == kAlign32   ? fp4_amax_kernel<kAlign32>
                 : align == kAlign16 ? fp4_amax_kernel<kAlign16>
                                     : fp4_amax_kernel<kScalar>;
  set_error_site("fp4_amax_kernel");
  return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kQThreads), 0, stream, 1,
                       false, pair);
}

cudaError_t launch_fp4_quantise(const Fp4QuantArgs* a, int n, const uint32_t* partials,
                                const int* num_partials, cudaStream_t stream) {
  QuantPair pair = {};
  int align = kAlign32;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    pair.p[i] = quant_params(a[i]);
    if (a[i].find_amax) {
      pair.p[i].partials = partials + i * (kMaxPartials / 2);
      pair.p[i].num_partials = num_partials[i];
    }
    const int own = row_align(a[i].x, a[i].ld, 2);
    align = own < align ? own : align;
    tiles += pair.p[i].tiles;
  }
  const bool trans = a[0].out_t.codes != nullptr;
  const bool record = a[0].amax_rec != nullptr || (n == 2 && a[1].amax_rec != nullptr);
  set_error_site("fp4_quantise_kernel");
  auto pick = [&](auto two) {
    constexpr bool kPair = decltype(two)::value;
    if (a[0].fmt != 0)
      return trans ? quant_kernel<1, true, kPair, false>(align) : quant_kernel<1, false, kPair, false>(align);
    if (record)
      return trans ? quant_kernel<0, true, kPair, true>(align) : quant_kernel<0, false, kPair, true>(align);
    return trans ? quant_kernel<0, true, kPair, false>(align) : quant_kernel<0, false, kPair, false>(align);
  };
  auto* kernel = n == 2 ? pick(std::true_type()) : pick(std::false_type());
  return launch_kernel(kernel, dim3(static_cast<unsigned>(tiles)), dim3(kQThreads), 0, stream, 1,
                       false, pair);
}

cudaError_t launch_fp4_dequantise(const Fp4View& t, int fmt, const float* inv, int64_t rows,
                                  int64_t cols, void* out, int64_t ldo, bool f32,
                                  cudaStream_t stream) {
  const int64_t tiles_c = (cols + kQTile - 1) / kQTile;
  const int align = row_align(out, ldo, f32 ? 4 : 2);
  const int64_t tile_rows = align == kScalar ? 32 : kQTile;
  const dim3 grid(static_cast<unsigned>((rows + tile_rows - 1) / tile_rows * tiles_c));
  set_error_site("fp4_dequantise_kernel");
  auto run = [&](auto* scalar, auto* align16, auto* align32, auto* dst) {
    auto* kernel = align == kAlign32 ? align32 : align == kAlign16 ? align16 : scalar;
    return launch_kernel(kernel, grid, dim3(kQThreads), 0, stream, 1, false,
                         static_cast<const uint8_t*>(t.codes), static_cast<const uint8_t*>(t.scales),
                         inv, rows, cols, t.ld, dst, ldo, static_cast<uint32_t>(tiles_c));
  };
  auto run_type = [&](auto* dst) {
    using Out = std::remove_pointer_t<decltype(dst)>;
    return fmt == 0 ? run(fp4_dequantise_ragged_kernel<0, Out>, fp4_dequantise_kernel<0, Out, kAlign16>,
                          fp4_dequantise_kernel<0, Out, kAlign32>, dst)
                    : run(fp4_dequantise_ragged_kernel<1, Out>, fp4_dequantise_kernel<1, Out, kAlign16>,
                          fp4_dequantise_kernel<1, Out, kAlign32>, dst);
  };
  return f32 ? run_type(static_cast<float*>(out)) : run_type(static_cast<uint16_t*>(out));
}

}  // namespace fp8lin
