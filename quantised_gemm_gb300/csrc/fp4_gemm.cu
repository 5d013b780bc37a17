// fp4_gemm.cu -- the product of two microscaled 4-bit operands on the
// 5th-generation tensor cores:
//   D[m, n] = bf16(alpha * sum_k a[m, k] ca[m, k / B] b[n, k] cb[n, k / B])
// with e2m1 values a, b, their block scales ca, cb (e4m3 over B = 16 values:
// NVFP4; powers of two over B = 32: MXFP4), fp32 accumulation, and
// alpha = fl32(inv_a / 6) * fl32(inv_b / 6) for NVFP4, 1 for MXFP4.
//
// tcgen05.mma.kind::mxf4nvf4 / mxf4 multiplies 64 values of K at a time and
// applies the block scales itself; it reads the codes from shared memory (as
// the 8-bit kernels do: 128-byte-swizzled K-major rows, here 256 values of K
// a stage) and the scales from tensor memory, where tcgen05.cp puts each
// 512-byte scale tile as four columns: 32 rows a column, their four scales in
// its four bytes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kBM = 128;            // rows of A per CTA
constexpr int kBKBytes = 128;       // bytes of K per stage and row
constexpr int kBK = 256;            // values of K per stage
constexpr int kMmaK = 64;           // K of one MMA
constexpr int kScTile = 512;        // bytes of a scale tile: 128 rows x 4 blocks
constexpr int kThreads = 192;       // producer, MMA, 4 epilogue warps

// Scale tiles of a stage along K: 64 values of K each (NVFP4), or 128 (MXFP4).
template <int kFmt>
constexpr int stage_ktiles() {
  return kFmt == 0 ? 4 : 2;
}

struct Fp4GemmParams {
  int64_t M, N, K;            // A has M rows, B has N rows
  const uint8_t* sca;         // scale tiles
  const uint8_t* scb;
  const float* inv_a;
  const float* inv_b;
  uint16_t* d;
  int64_t ldd;
  int* err;
  bool vec;                   // D's rows take 16-byte stores
};

// Instruction descriptor of kind::mxf4nvf4 / kind::mxf4: e2m1 operands, both
// K-major, dense, K = 64; scale type ue4m3 (NVFP4) or ue8m0 (MXFP4).  The
// scale ids pick the bytes of a column that hold the blocks (MXFP4: two
// blocks an MMA, bytes 0-1 or 2-3).
template <int kFmt>
__device__ constexpr uint32_t make_idesc_fp4(uint32_t m, uint32_t n, uint32_t sf_id) {
  return (sf_id << 4)                    // [4,6)   scale id of B
         | (1u << 7)                     // [7,10)  A: e2m1
         | (1u << 10)                    // [10,12) B: e2m1
         | ((n >> 3) << 17)              // [17,23) N >> 3
         | ((kFmt == 0 ? 0u : 1u) << 23)  // [23]   scale type
         | ((m >> 4) << 24)              // [24,29) M >> 4
         | (sf_id << 29);                // [29,31) scale id of A
}

// D[tmem] (+)= A . B^T with the block scales at sa / sb in tensor memory.
template <int kFmt>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (kFmt == 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// One scale tile, shared memory -> four columns of tensor memory.
__device__ __forceinline__ void copy_scale_tile(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Descriptor of a scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups
// 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scale(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8) << 16) |
         (static_cast<uint64_t>(8) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Contiguous bulk copy global -> shared, counted in bytes on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void record_error(int* err, volatile int* abort_flag, int code) {
  atomicCAS(err, 0, code);
  *abort_flag = 1;
}

template <int BN, int STAGES>
struct Cfg {
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kBBytes = BN * kBKBytes;
  static constexpr int kScBytes = 4 * kScTile;  // of one operand and stage
  static constexpr int kStageBytes = kABytes + kBBytes + 2 * kScBytes;
  // Two accumulators, then four columns a scale tile for A and for B.
  static constexpr int kSfa = 2 * BN;
  static constexpr int kSfb = kSfa + 16;
  static constexpr int kTmemCols = kSfb + 16 <= 128 ? 128 : kSfb + 16 <= 256 ? 256 : 512;
  static constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(STAGES) * kStageBytes + 256;
  static_assert(BN % 16 == 0 && BN <= 128, "one row of scale tiles for B");
};

// One accumulator chunk (this lane's row, 16 columns from col0), scaled and
// rounded to bf16.  kTrans: the kernel's rows are D's columns.
template <bool kTrans>
__device__ __forceinline__ void store_chunk(const uint32_t (&r)[16], float alpha,
                                            const Fp4GemmParams& p, int64_t row, int64_t col0) {
  if (row >= p.M) return;
  if constexpr (kTrans) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (col0 + j < p.N)
        p.d[(col0 + j) * p.ldd + row] = static_cast<uint16_t>(
            cvt_bf16x2(__fmul_rn(__uint_as_float(r[j]), alpha), 0.0f) & 0xFFFFu);
  } else {
    uint16_t* dst = p.d + row * p.ldd + col0;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v0, v1;
      mul2_rn(r[2 * j], r[2 * j + 1], alpha, v0, v1);
      w[j] = cvt_bf16x2(v0, v1);
    }
    if (p.vec && col0 + 16 <= p.N) {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col0 + j < p.N) dst[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

template <int kFmt, int BN, int STAGES, bool kTrans>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Fp4GemmParams p) {
  using C = Cfg<BN, STAGES>;
  constexpr int kKt = stage_ktiles<kFmt>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * C::kABytes;
  uint8_t* sSa = sB + STAGES * C::kBBytes;
  uint8_t* sSb = sSa + STAGES * C::kScBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sSb + STAGES * C::kScBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2]
  uint64_t* drain = acc_empty + 2;      // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(sizeof(uint64_t) * (2 * STAGES + 5) + 8 <= 256, "barrier block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t num_n = (p.N + BN - 1) / BN;
  const int64_t num_tiles = ((p.M + kBM - 1) / kBM) * num_n;
  const int num_kb = static_cast<int>((p.K + kBK - 1) / kBK);
  const int ktiles = static_cast<int>((p.K + kBK / kKt - 1) / (kBK / kKt));  // scale tiles along K

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t fills[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) fills[s] = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const int m_blk = static_cast<int>(t / num_n), n_blk = static_cast<int>(t % num_n);
        // B's scale tile holds 128 rows: BN of them belong to this tile.
        const uint8_t* sa = p.sca + static_cast<int64_t>(m_blk) * ktiles * kScTile;
        const uint8_t* sb = p.scb + static_cast<int64_t>(n_blk) * ktiles * kScTile;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const int kt0 = kb * kKt;
          const uint32_t sc_bytes = static_cast<uint32_t>(min(kKt, ktiles - kt0)) * kScTile;
          mbar_arrive_expect_tx(&full[stage], C::kABytes + C::kBBytes + 2 * sc_bytes);
          tma_load_2d(sA + stage * C::kABytes, &tmA, &full[stage], kb * kBKBytes, m_blk * kBM);
          tma_load_2d(sB + stage * C::kBBytes, &tmB, &full[stage], kb * kBKBytes, n_blk * BN);
          bulk_load(sSa + stage * C::kScBytes, sa + static_cast<int64_t>(kt0) * kScTile, sc_bytes,
                    &full[stage]);
          bulk_load(sSb + stage * C::kScBytes, sb + static_cast<int64_t>(kt0) * kScTile, sc_bytes,
                    &full[stage]);
#pragma unroll
          for (int s = 0; s < STAGES; ++s)
            if (s == stage) ++fills[s];
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_error(p.err, abort_flag, kErrGemmProducerWait);
        volatile int never = 0;
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
          if (fills[s] > 0) mbar_wait_bounded(&full[s], (fills[s] - 1) & 1u, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool issued = false;
      for (int64_t t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        if (!mbar_wait_bounded(&acc_empty[acc], acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_bounded(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const int nkt = min(kKt, ktiles - kb * kKt);
          const int steps = static_cast<int>(min(int64_t(4), (p.K - int64_t(kb) * kBK + kMmaK - 1) / kMmaK));
          const uint64_t a_desc = smem_desc_k_sw128(smem_addr(sA + stage * C::kABytes));
          const uint64_t b_desc = smem_desc_k_sw128(smem_addr(sB + stage * C::kBBytes));
          const uint64_t sa_desc = smem_desc_scale(smem_addr(sSa + stage * C::kScBytes));
          const uint64_t sb_desc = smem_desc_scale(smem_addr(sSb + stage * C::kScBytes));
          // Copies and MMAs of one thread run in the order they are issued.
          for (int i = 0; i < nkt; ++i) {
            copy_scale_tile(tmem_base + C::kSfa + 4 * i, sa_desc + static_cast<uint64_t>(i * (kScTile >> 4)));
            copy_scale_tile(tmem_base + C::kSfb + 4 * i, sb_desc + static_cast<uint64_t>(i * (kScTile >> 4)));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;  // the rest of the stage lies past K: its scales are not loaded
            const int kt = kFmt == 0 ? k : k >> 1;
            const uint32_t idesc = make_idesc_fp4<kFmt>(kBM, BN, kFmt == 0 ? 0u : 2u * (k & 1));
            mma_fp4<kFmt>(d_tmem, a_desc + static_cast<uint64_t>(2 * k),
                          b_desc + static_cast<uint64_t>(2 * k), idesc, tmem_base + C::kSfa + 4 * kt,
                          tmem_base + C::kSfb + 4 * kt, (kb > 0 || k > 0) ? 1u : 0u);
          }
          issued = true;
          mma_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(&acc_full[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        record_error(p.err, abort_flag, kErrGemmMmaWait);
        if (issued) {
          volatile int never = 0;
          mma_commit(drain);
          mbar_wait_bounded(drain, 0, &never);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;  // TMEM lanes this warp may read
    const float alpha =
        kFmt == 0 ? __fmul_rn(__fdiv_rn(*p.inv_a, 6.0f), __fdiv_rn(*p.inv_b, 6.0f)) : 1.0f;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t t = blockIdx.x; t < num_tiles; t += gridDim.x) {
      const int64_t m_blk = t / num_n, n_blk = t % num_n;
      const bool ready =
          __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&acc_full[acc], acc_phase, abort_flag));
      if (!ready) {
        if (lane == 0) record_error(p.err, abort_flag, kErrGemmEpilogueWait);
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * BN);
      const int64_t row = m_blk * kBM + quarter * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < BN / 16; ++c) {
        uint32_t r[16];
        tmem_load_16cols(t_row + c * 16, r);
        tmem_load_wait();
        store_chunk<kTrans>(r, alpha, p, row, n_blk * BN + c * 16);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int kFmt, int BN, int STAGES, bool kTrans>
cudaError_t run_one(const Fp4View& a, const Fp4View& b, const Fp4GemmParams& p,
                    const DeviceInfo& dev, cudaStream_t stream) {
  using C = Cfg<BN, STAGES>;
  CUtensorMap tmA, tmB;
  // A row's codes to the end of its last 32 values: zero past that.
  const uint64_t inner = static_cast<uint64_t>((p.K + 31) / 32 * 16);
  if (!make_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, inner, p.M, a.ld, kBKBytes, kBM,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, b.codes, inner, p.N, b.ld, kBKBytes, BN,
                   CU_TENSOR_MAP_SWIZZLE_128B))
    return map_failed("fp4 gemm operand");
  auto* kernel = gemm_fp4_kernel<kFmt, BN, STAGES, kTrans>;
  static std::mutex mu;
  static bool done[64] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    if (!done[dev.device]) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(C::kSmemBytes));
      if (e != cudaSuccess) return e;
      done[dev.device] = true;
    }
  }
  const int64_t tiles = ((p.M + kBM - 1) / kBM) * ((p.N + BN - 1) / BN);
  const unsigned grid = static_cast<unsigned>(tiles < dev.num_sms ? tiles : dev.num_sms);
  set_error_site("gemm_fp4_kernel");
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, 1, false, tmA, tmB,
                       p);
}

template <int kFmt>
cudaError_t run_fmt(const Fp4GemmArgs& g, Fp4GemmParams p, const DeviceInfo& dev,
                    cudaStream_t stream) {
  if (g.M <= 128) {
    // Few rows: the weight's rows fill the MMA's 128, the tokens are its columns.
    p.M = g.N;
    p.N = g.M;
    p.sca = g.b.scales;
    p.scb = g.a.scales;
    p.inv_a = g.inv_b;
    p.inv_b = g.inv_a;
    if (g.M <= 16) return run_one<kFmt, 16, 8, true>(g.b, g.a, p, dev, stream);
    if (g.M <= 32) return run_one<kFmt, 32, 8, true>(g.b, g.a, p, dev, stream);
    if (g.M <= 64) return run_one<kFmt, 64, 6, true>(g.b, g.a, p, dev, stream);
    return run_one<kFmt, 128, 5, true>(g.b, g.a, p, dev, stream);
  }
  return run_one<kFmt, 128, 5, false>(g.a, g.b, p, dev, stream);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4GemmArgs& g, const DeviceInfo& dev, cudaStream_t stream) {
  Fp4GemmParams p;
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.sca = g.a.scales;
  p.scb = g.b.scales;
  p.inv_a = g.inv_a;
  p.inv_b = g.inv_b;
  p.d = static_cast<uint16_t*>(g.d);
  p.ldd = g.ldd;
  p.err = g.ws_error;
  p.vec = (reinterpret_cast<uintptr_t>(g.d) & 15u) == 0 && g.ldd % 8 == 0;
  return g.fmt == 0 ? run_fmt<0>(g, p, dev, stream) : run_fmt<1>(g, p, dev, stream);
}

}  // namespace fp8lin
