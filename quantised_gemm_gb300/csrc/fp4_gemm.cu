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

#include "fp4_quant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kBM = 128;            // rows of A per CTA
constexpr int kBKBytes = 128;       // bytes of K per stage and row
constexpr int kBK = 256;            // values of K per stage
constexpr int kMmaK = 64;           // K of one MMA
constexpr int kScTile = 512;        // bytes of a scale tile: 128 rows x 4 blocks
constexpr int kScElems = kScTile / 8;  // its 8-byte elements, as the tensor maps see it
constexpr int kThreads = 192;       // producer, MMA, 4 epilogue warps

// Scale tiles of a stage along K: 64 values of K each (NVFP4), or 128 (MXFP4).
template <int kFmt>
constexpr int stage_ktiles() {
  return kFmt == 0 ? 4 : 2;
}

struct Fp4GemmParams {
  int64_t M, N, K;            // A has M rows, B has N rows
  const float* inv_a;
  const float* inv_b;
  uint16_t* d;
  int64_t ldd;
  int* err;
  bool vec;                   // D's rows take 16-byte stores
  // Pair kernel: tiles [0, t_full) run whole, each one after them as s_tail
  // slices of the K loop that join through fp32 partials, tickets (two ints
  // for each epilogue warp of a tile) and the number of pairs with a slice that
  // have begun; all counters are zero between launches.
  int64_t t_full;
  int s_tail;
  int slice_pairs;  // pairs whose last unit is a slice: the first ones
  float* partials;
  int* tickets;
  int* begun;       // [2]: those that have begun, epilogue warps that have read it
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

// The same over a CTA pair.
template <int kFmt>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (kFmt == 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// One scale tile, shared memory -> four columns of tensor memory (the pair
// form: in both CTAs, each from its own shared memory).
__device__ __forceinline__ void copy_scale_tile(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void copy_scale_tile_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Descriptor of a scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups
// 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scale(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8) << 16) |
         (static_cast<uint64_t>(8) << 32) | (static_cast<uint64_t>(1) << 46);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, P;\n\t}"
               : "=r"(p));
  return p != 0;
}

// The two halves of a cluster barrier, without ordering memory: after the
// wait, every CTA of the cluster has started, and its shared memory may be
// written.
__device__ __forceinline__ void cluster_started_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on a barrier of the pair with a release at CTA scope, which waits for
// no memory operation of this thread outside the CTA: for an arrival that
// hands over tensor memory, ordered by the tcgen05 fences around it.  The
// cluster-scope release costs about a microsecond beside TMA stores in flight.
__device__ __forceinline__ void mbar_arrive_cluster_tmem(uint32_t cluster_saddr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_saddr)
               : "memory");
}

// A bounded wait of the whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag));
}

__device__ __forceinline__ void record_error(int* err, volatile int* abort_flag, int code) {
  atomicCAS(err, 0, code);
  *abort_flag = 1;
}

// Where a K loop is shared by a cluster, its CTAs own the rows of the tile in
// turn: `split` parts of kBM / split rows.  Each CTA's `joined` holds the
// partials of its own rows, [split][BN][rows] floats, which the CTAs write
// into it: one cluster barrier, and nothing is read across CTAs.
template <int BN>
constexpr size_t joined_bytes(int split) {
  return split > 1 ? static_cast<size_t>(kBM) * BN * 4 : 0;
}

// The epilogue of one tile for one of four warps: its 32 rows of the
// accumulator to D, or, where the K loop is shared, to their owners.
template <int BN>
__device__ __forceinline__ void few_epilogue(const Fp4GemmParams& p, uint32_t tmem_base, float* joined,
                                             int split, int rank, bool any, int64_t row0, int cols,
                                             float alpha, uint16_t* d, int quarter, int lane) {
  const int r = quarter * 32 + lane;
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
  const int rows = kBM / split;
  const uint32_t to = split > 1 ? map_to_cta(smem_addr(joined + (rank * BN * rows + r % rows)),
                                             static_cast<uint32_t>(r / rows))
                                : 0u;
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 16) {
    uint32_t v[16];
    tmem_load_16cols(t_row + c0, v);
    tmem_load_wait();
    if (split > 1) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < cols)
          st_shared_cluster_u32(to + static_cast<uint32_t>((c0 + j) * rows) * 4u, any ? v[j] : 0u);
    } else if (row0 + r < p.M) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < cols)
          d[(c0 + j) * p.ldd + r] = static_cast<uint16_t>(
              cvt_bf16x2(__fmul_rn(__uint_as_float(v[j]), alpha), 0.0f) & 0xFFFFu);
    }
  }
}

// This CTA's rows of a tile, added up over the partials in rank order, four
// rows a thread.
template <int BN>
__device__ __forceinline__ void join_partials(const Fp4GemmParams& p, const float* joined, int split,
                                              int rank, int64_t row0, int cols, float alpha,
                                              uint16_t* d) {
  const int rows = kBM / split, quads = rows / 4;
  const bool wide = p.vec && row0 + kBM <= p.M;
  for (int e = threadIdx.x; e < quads * cols; e += blockDim.x) {
    const int c = e / quads, q = e % quads * 4;
    const float* src = joined + c * rows + q;
    float4 sum = *reinterpret_cast<const float4*>(src);
    for (int s = 1; s < split; ++s) {
      const float4 v = *reinterpret_cast<const float4*>(src + s * BN * rows);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    const uint32_t lo = cvt_bf16x2(__fmul_rn(sum.x, alpha), __fmul_rn(sum.y, alpha));
    const uint32_t hi = cvt_bf16x2(__fmul_rn(sum.z, alpha), __fmul_rn(sum.w, alpha));
    const int r = rank * rows + q;
    uint16_t* dst = d + c * p.ldd + r;
    if (wide) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row0 + r + j < p.M)
          dst[j] = static_cast<uint16_t>((j < 2 ? lo : hi) >> (16 * (j & 1)));
    }
  }
}

// ------------------------------------------------------------------ few tiles
//
// One 128 x BN tile of D^T a cluster: A, the operand that fills the MMA's 128
// rows, is the weight, and B the tokens, BN of them.  The cluster's CTAs
// share the K loop: each multiplies its share of the stages into an fp32
// partial and writes the rows of it to their owners' shared memory; after a
// cluster barrier each CTA adds up its own rows in rank order -- the same
// bits every time -- and writes D.  No workspace and no second launch.
// (Reading the other CTAs' partials after the barrier instead took 1.5 us
// more of 32 x 4096 x 14336.)
//
// Bound by reading the weight (0.56 bytes a value): the split brings enough
// CTAs, two an SM, to keep that many loads in flight.  With `early` the
// preceding kernel of the stream is known not to write A, so its first
// stages are loaded before that kernel has finished.
//
// 32 x 4096 x 14336 9.5 us in NVFP4, the weight at 3.5 TB/s (the launch and
// the join take 4 us of it); 1 x 4096 x 4096 5.6 us; 128 x 4096 x 4096 7.7 and
// 512 x 4096 x 4096 10.4 us, where every 64 tokens read the weight from L2
// again.
template <int kFmt, int BN, int STAGES>
struct FewCfg {
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kBBytes = BN * kBKBytes;
  static constexpr int kScBytes = stage_ktiles<kFmt>() * kScTile;
  static constexpr int kStageBytes = kABytes + kBBytes + 2 * kScBytes;
  static constexpr int kSfa = BN;
  static constexpr int kSfb = kSfa + 16;
  static constexpr int kTmemCols = BN + 32 <= 64 ? 64 : 128;
  static constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(STAGES) * kStageBytes + 256;
  static_assert(BN % 16 == 0 && BN + 32 <= 128, "one row of scale tiles for B");
  // Two CTAs an SM, or one with a deep ring.
  static constexpr int kPerSm = STAGES <= 4 ? 2 : 1;
  static_assert(kPerSm * (kSmemBytes + (BN <= 32 || kPerSm == 1 ? joined_bytes<BN>(2) : 0) + 1024) <= 233472,
                "fits");
};

template <int kFmt, int BN, int STAGES>
__global__ void __launch_bounds__(kThreads, FewCfg<kFmt, BN, STAGES>::kPerSm)
    gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSa,
                        const __grid_constant__ CUtensorMap tmSb,
                        const __grid_constant__ Fp4GemmParams p, const int split, const bool early) {
  using C = FewCfg<kFmt, BN, STAGES>;
  constexpr int kKt = stage_ktiles<kFmt>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * C::kABytes;
  uint8_t* sSa = sB + STAGES * C::kBBytes;
  uint8_t* sSb = sSa + STAGES * C::kScBytes;
  float* joined = reinterpret_cast<float*>(sSb + STAGES * C::kScBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(joined) + joined_bytes<BN>(split));
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t tile = blockIdx.x / split;
  const int64_t num_n = (p.N + BN - 1) / BN;  // tiles of tokens
  const int m_blk = static_cast<int>(tile / num_n), n_blk = static_cast<int>(tile % num_n);
  const int num_kb = static_cast<int>((p.K + kBK - 1) / kBK);
  const int per = (num_kb + split - 1) / split;
  const int kb0 = min(num_kb, rank * per), nkb = min(num_kb, kb0 + per) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  auto load_a = [&](int stage, int kb) {
    mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
    tma_load_2d(sA + stage * C::kABytes, &tmA, &full[stage], kb * kBKBytes, m_blk * kBM);
    tma_load_2d(sSa + stage * C::kScBytes, &tmSa, &full[stage], kb * kKt * kScElems, m_blk);
  };
  if (threadIdx.x == 0) {  // the weight's first stages, before anything else
    if (!early) griddep_wait();
    for (int i = 0; i < nkb && i < STAGES; ++i) load_a(i, kb0 + i);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (split > 1) cluster_started_arrive();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int i = 0;
      for (; i < nkb; ++i) {
        const int stage = i % STAGES, kb = kb0 + i;
        if (i >= STAGES && !mbar_wait_bounded(&empty[stage], (i / STAGES - 1) & 1u, abort_flag)) break;
        if (i >= STAGES) load_a(stage, kb);
        tma_load_2d(sB + stage * C::kBBytes, &tmB, &full[stage], kb * kBKBytes, n_blk * BN);
        // B's scale tile holds 128 rows: BN of them belong to this tile.
        tma_load_2d(sSb + stage * C::kScBytes, &tmSb, &full[stage], kb * kKt * kScElems,
                    n_blk * BN / 128);
      }
      if (i < nkb) {
        record_error(p.err, abort_flag, kErrGemmProducerWait);
        // Let the copies in flight land before the CTA exits.
        volatile int never = 0;
        for (int j = max(0, i - STAGES); j < i; ++j)
          mbar_wait_bounded(&full[j % STAGES], (j / STAGES) & 1u, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The tile's tokens may start inside a scale tile: 32 rows a column.
    const uint32_t sfb = tmem_base + C::kSfb + static_cast<uint32_t>(n_blk * BN % 128 / 32);
    bool ok = true;
    int i = 0;
    for (; i < nkb; ++i) {
      const int stage = i % STAGES;
      ok = warp_wait(&full[stage], (i / STAGES) & 1u, abort_flag);
      if (!ok) break;
      tc_fence_after_sync();
      const uint64_t a_desc = smem_desc_k_sw128(smem_addr(sA + stage * C::kABytes));
      const uint64_t b_desc = smem_desc_k_sw128(smem_addr(sB + stage * C::kBBytes));
      const uint64_t sa_desc = smem_desc_scale(smem_addr(sSa + stage * C::kScBytes));
      const uint64_t sb_desc = smem_desc_scale(smem_addr(sSb + stage * C::kScBytes));
      const int64_t left = p.K - int64_t(kb0 + i) * kBK;
      const int steps = left >= kBK ? 4 : static_cast<int>((left + kMmaK - 1) / kMmaK);
      if (elect_one()) {
        // Copies and MMAs of one thread run in the order they are issued.
#pragma unroll
        for (int t = 0; t < kKt; ++t) {
          copy_scale_tile(tmem_base + C::kSfa + 4 * t, sa_desc + static_cast<uint64_t>(t * (kScTile >> 4)));
          copy_scale_tile(tmem_base + C::kSfb + 4 * t, sb_desc + static_cast<uint64_t>(t * (kScTile >> 4)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int kt = kFmt == 0 ? k : k >> 1;
          const uint32_t idesc = make_idesc_fp4<kFmt>(kBM, BN, kFmt == 0 ? 0u : 2u * (k & 1));
          if (k < steps)  // the rest of the stage lies past K
            mma_fp4<kFmt>(tmem_base, a_desc + static_cast<uint64_t>(2 * k),
                          b_desc + static_cast<uint64_t>(2 * k), idesc, tmem_base + C::kSfa + 4 * kt,
                          sfb + 4 * kt, (i > 0 || k > 0) ? 1u : 0u);
        }
        if (i + STAGES < nkb) mma_commit(&empty[stage]);  // no load follows into the other stages
      }
      __syncwarp();
    }
    if (elect_one()) {
      if (ok) {
        mma_commit(acc_full);
      } else {
        record_error(p.err, abort_flag, kErrGemmMmaWait);
        if (i > 0) {
          volatile int never = 0;
          mma_commit(drain);
          mbar_wait_bounded(drain, 0, &never);
        }
      }
    }
    __syncwarp();
  }

  __syncwarp();
  if (split > 1) cluster_started_wait();  // before anything is written to another CTA
  const int cols = static_cast<int>(min(int64_t(BN), p.N - int64_t(n_blk) * BN));  // live tokens
  const int64_t row0 = static_cast<int64_t>(m_blk) * kBM;
  const float alpha =
      kFmt == 0 ? __fmul_rn(__fdiv_rn(*p.inv_a, 6.0f), __fdiv_rn(*p.inv_b, 6.0f)) : 1.0f;
  uint16_t* d = p.d + static_cast<int64_t>(n_blk) * BN * p.ldd + row0;
  if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;  // TMEM lanes this warp may read
    const bool ready = warp_wait(acc_full, 0, abort_flag);
    if (!ready) {
      if (lane == 0) record_error(p.err, abort_flag, kErrGemmEpilogueWait);
    } else {
      tc_fence_after_sync();
      few_epilogue<BN>(p, tmem_base, joined, split, rank, nkb > 0, row0, cols, alpha, d, quarter, lane);
    }
  }
  if (split > 1) {
    tc_fence_before_sync();
    cluster_sync_all();  // every partial is with its rows' owner
    join_partials<BN>(p, joined, split, rank, row0, cols, alpha, d);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ few tokens, quantised on the way
//
// The few-tile product of up to 32 tokens straight from their bf16 values:
// one launch instead of a quantisation and a product.  While the first stages
// of the weight are on their way, each CTA quantises its K slice of the
// tokens into shared memory, in the places that the codes and scale tiles of
// a stage have; a cluster covers all of K, so its CTAs join their maxima for
// the tensorwise scale.  The first tile's cluster also writes the quantised
// tokens and their state.  Every thread holds its values in registers between
// the maximum and the conversion, which is what bounds the slice.
// Bound by reading the weight and by the launch.  In a graph, NVFP4: 1 x 14336
// x 4096 9.1 us, 3.6 TB/s (10.2 in two launches), 1 x 4096 x 4096 5.7 us (6.4),
// 32 x 4096 x 4096 8.3 us (11.0); MXFP4: 4.5 us (5.9) and 7.1 us (6.6, but two
// launches take the host 2 us longer).  What does not need the launches before
// this one is done before the wait for them: 2 us of each.
constexpr int kFusedThreads = 256;
constexpr int kFusedUnits = 4 * kFusedThreads;  // of 16 values, of a CTA
constexpr size_t kFusedSmemHalf = 114688;       // two CTAs an SM
constexpr size_t kFusedSmemFull = 229376;       // one

template <int kFmt, int BN>
struct FusedCfg {
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kBBytes = BN * kBKBytes;                  // of a K block
  static constexpr int kScBytes = stage_ktiles<kFmt>() * kScTile;
  static constexpr int kRingBytes = kABytes + kScBytes;          // of a stage
  static constexpr int kMaxStages = 10;
  static constexpr int kFixed = 1024 + 512 + 256;                // alignment, table, barriers
  static constexpr int kSfa = BN;
  static constexpr int kSfb = kSfa + 16;
  static constexpr int kTmemCols = 64;
  static_assert(BN + 32 <= kTmemCols, "accumulator and scales");
  // Stages beside the tokens of nkb K blocks.
  static int stages(int64_t nkb, int split, size_t smem) {
    const int64_t left = int64_t(smem) - kFixed - int64_t(joined_bytes<BN>(split)) -
                         nkb * (kBBytes + kScBytes);
    const int64_t n = left / kRingBytes;
    return static_cast<int>(n < 0 ? 0 : n > nkb ? nkb : n > kMaxStages ? kMaxStages : n);
  }
};

struct FusedTokens {
  const uint16_t* x;
  Span span;
  int64_t ldx;
  const float* amax_in;    // NVFP4: precomputed amax, or
  const float* scale_in;   // the stored scale, or (neither) the tokens' own amax
  const float* inv_in;     // beside scale_in
  float eps;
  float* amax_out;         // each may be null
  float* scale_out;
  float* inv_out;
  float* own_inv;          // of the quantised tokens
  uint8_t* codes;          // the quantised tokens
  int64_t ld4;
  uint8_t* scales;
};

template <int kFmt, int BN, int kAlign>
__global__ void __launch_bounds__(kFusedThreads, 2)
    gemm_fp4_fused_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmSa,
                          const __grid_constant__ Fp4GemmParams p,
                          const __grid_constant__ FusedTokens x, const int split, const int stages) {
  using C = FusedCfg<kFmt, BN>;
  constexpr int kKt = stage_ktiles<kFmt>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int m_blk = static_cast<int>(blockIdx.x / split);
  const int num_kb = static_cast<int>((p.K + kBK - 1) / kBK);
  const int per = (num_kb + split - 1) / split;
  const int kb0 = min(num_kb, rank * per), nkb = min(num_kb, kb0 + per) - kb0;
  uint8_t* sA = smem;
  uint8_t* sB = sA + stages * C::kABytes;    // [per] K blocks of the tokens' codes
  uint8_t* sSa = sB + per * C::kBBytes;
  uint8_t* sSb = sSa + stages * C::kScBytes;  // [per] K blocks of their scale tiles
  float* joined = reinterpret_cast<float*>(sSb + per * C::kScBytes);
  float* table = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(joined) + joined_bytes<BN>(split));
  uint64_t* full = reinterpret_cast<uint64_t*>(table + 128);
  uint64_t* empty = full + C::kMaxStages;
  uint64_t* acc_full = empty + C::kMaxStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* red = tmem_slot + 2;   // [8] warps' maxima
  uint32_t* cta_max = red + 8;     // read by the cluster

  auto load_a = [&](int stage, int kb) {
    mbar_arrive_expect_tx(&full[stage], C::kRingBytes);
    tma_load_2d(sA + stage * C::kABytes, &tmA, &full[stage], kb * kBKBytes, m_blk * kBM);
    tma_load_2d(sSa + stage * C::kScBytes, &tmSa, &full[stage], kb * kKt * kScElems, m_blk);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (split > 1) cluster_started_arrive();
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  // Scale tiles hold 128 rows; those past the tokens are zero.
  for (int i = threadIdx.x; i < nkb * C::kScBytes / 16; i += kFusedThreads)
    reinterpret_cast<uint4*>(sSb)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
  griddep_wait();

  // ------------------------------------------------------------ the tokens
  // Their loads go out before the weight's, behind which they would wait.
  const int row_units = nkb * 16, units = static_cast<int>(p.N) * row_units;
  const int64_t col0 = static_cast<int64_t>(kb0) * kBK;
  auto load_units = [&](uint4 (&v)[4][2], int per_row, int count, int64_t first) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = threadIdx.x + k * kFusedThreads;
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      if (u < count) {
        const int row = u / per_row, c = u - row * per_row;
        load16<kAlign>(x.x + row * x.ldx, first + c * 16, p.K, x.span, v[k]);
      }
    }
  };
  // The tensorwise maximum: every CTA's own where all tokens fit its
  // registers, else the cluster's.
  const int all_units = static_cast<int>(p.N) * num_kb * 16;
  const bool find = kFmt == 0 && x.amax_in == nullptr;
  const bool whole = split == 1 || all_units <= kFusedUnits;
  uint4 v[4][2], w[4][2];
  load_units(v, row_units, units, col0);
  if (find && whole && split > 1) load_units(w, num_kb * 16, all_units, 0);
  if (threadIdx.x == 0)
    for (int i = 0; i < nkb && i < stages; ++i) load_a(i, kb0 + i);
  __syncwarp();
  if (split > 1) cluster_started_wait();  // before anything is written to another CTA
  uint32_t largest[4], pairs = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t own = max_magnitude(max8(v[k][0]), max8(v[k][1]));
    pairs = max_magnitude(pairs, own);
    largest[k] = larger_half(own);
  }
  if (find && whole && split > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      pairs = max_magnitude(pairs, max_magnitude(max8(w[k][0]), max8(w[k][1])));
  }
  uint32_t m = larger_half(pairs);
  float s = 0.0f, inv = 1.0f;
  if constexpr (kFmt == 0) {
    float amax = 0.0f;
    if (!find) {
      amax = *x.amax_in;
    } else {
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (lane == 0) red[warp] = m;
      __syncthreads();
      uint32_t all = red[0];
#pragma unroll
      for (int w = 1; w < kFusedThreads / 32; ++w) all = max(all, red[w]);
      if (!whole) {
        if (threadIdx.x == 0) *cta_max = all;
        cluster_sync_all();
        for (int r = 0; r < split; ++r)
          all = max(all, ld_shared_cluster_u32(map_to_cta(smem_addr(cta_max), r)));
      }
      amax = __uint_as_float(all << 16);
    }
    s = x.scale_in != nullptr ? *x.scale_in : fp4_tensor_scale(amax, x.eps);
    inv = x.scale_in != nullptr ? *x.inv_in : __fdiv_rn(1.0f, s);
    fill_table(s, table);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      if (x.amax_out != nullptr) *x.amax_out = amax;
      if (x.scale_out != nullptr) {
        *x.scale_out = s;
        *x.inv_out = inv;
      }
      if (x.own_inv != nullptr) *x.own_inv = inv;
    }
  }
  __syncthreads();  // the table is filled and the scale tiles are zero
  // Only now that this CTA has its tensor memory: a CTA of the next launch
  // that took the last of it while waiting for this grid would never get on.
  griddep_launch_dependents();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = threadIdx.x + k * kFusedThreads;
    // A block of 32 is two units of neighbouring lanes.
    const uint32_t top =
        kFmt == 0 ? largest[k] : max(largest[k], __shfl_xor_sync(0xFFFFFFFFu, largest[k], 1));
    float r;
    const uint32_t sc = block_scale<kFmt>(top, s, table, r);
    const uint2 codes = make_uint2(code8<kFmt>(v[k][0], r), code8<kFmt>(v[k][1], r));
    if (u >= units) continue;
    const int row = u / row_units, c = u - row * row_units;
    const int kb = c >> 4, byte = (c & 15) * 8;  // of a 128-byte swizzled row
    *reinterpret_cast<uint2*>(sB + kb * C::kBBytes + row * kBKBytes +
                              (((byte >> 4) ^ (row & 7)) << 4) + (byte & 8)) = codes;
    const int blk = kFmt == 0 ? c & 15 : (c & 15) >> 1;
    if (kFmt == 0 || (c & 1) == 0)
      sSb[kb * C::kScBytes + (blk >> 2) * kScTile + row * 16 + (blk & 3)] = static_cast<uint8_t>(sc);
    const int64_t col = col0 + c * 16;
    if (m_blk == 0 && col < (p.K + 31) / 32 * 32)
      *reinterpret_cast<uint2*>(x.codes + row * x.ld4 + (col >> 1)) = codes;
  }
  fence_proxy_async_shared();  // the tensor core reads what was written here
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  if (m_blk == 0) {
    const int64_t ktiles = (p.K + kBK / kKt - 1) / (kBK / kKt), first = static_cast<int64_t>(kb0) * kKt;
    const int mine = static_cast<int>(min(ktiles - first, static_cast<int64_t>(nkb) * kKt)) * (kScTile / 16);
    for (int i = threadIdx.x; i < mine; i += kFusedThreads)
      reinterpret_cast<uint4*>(x.scales + first * kScTile)[i] = reinterpret_cast<const uint4*>(sSb)[i];
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int i = min(nkb, stages);
      for (; i < nkb; ++i) {
        if (!mbar_wait_bounded(&empty[i % stages], (i / stages - 1) & 1u, abort_flag)) break;
        load_a(i % stages, kb0 + i);
      }
      if (i < nkb) {
        record_error(p.err, abort_flag, kErrGemmProducerWait);
        volatile int never = 0;
        for (int j = max(0, i - stages); j < i; ++j)
          mbar_wait_bounded(&full[j % stages], (j / stages) & 1u, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    int i = 0, stage = 0;
    uint32_t phase = 0;
    for (; i < nkb; ++i) {
      ok = warp_wait(&full[stage], phase, abort_flag);
      if (!ok) break;
      tc_fence_after_sync();
      const uint64_t a_desc = smem_desc_k_sw128(smem_addr(sA + stage * C::kABytes));
      const uint64_t b_desc = smem_desc_k_sw128(smem_addr(sB + i * C::kBBytes));
      const uint64_t sa_desc = smem_desc_scale(smem_addr(sSa + stage * C::kScBytes));
      const uint64_t sb_desc = smem_desc_scale(smem_addr(sSb + i * C::kScBytes));
      const int64_t left = p.K - int64_t(kb0 + i) * kBK;
      const int steps = left >= kBK ? 4 : static_cast<int>((left + kMmaK - 1) / kMmaK);
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < kKt; ++t) {
          copy_scale_tile(tmem_base + C::kSfa + 4 * t, sa_desc + static_cast<uint64_t>(t * (kScTile >> 4)));
          copy_scale_tile(tmem_base + C::kSfb + 4 * t, sb_desc + static_cast<uint64_t>(t * (kScTile >> 4)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int kt = kFmt == 0 ? k : k >> 1;
          const uint32_t idesc = make_idesc_fp4<kFmt>(kBM, BN, kFmt == 0 ? 0u : 2u * (k & 1));
          if (k < steps)
            mma_fp4<kFmt>(tmem_base, a_desc + static_cast<uint64_t>(2 * k),
                          b_desc + static_cast<uint64_t>(2 * k), idesc, tmem_base + C::kSfa + 4 * kt,
                          tmem_base + C::kSfb + 4 * kt, (i > 0 || k > 0) ? 1u : 0u);
        }
        if (i + stages < nkb) mma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) {
      if (ok) {
        mma_commit(acc_full);
      } else {
        record_error(p.err, abort_flag, kErrGemmMmaWait);
        if (i > 0) {
          volatile int never = 0;
          mma_commit(drain);
          mbar_wait_bounded(drain, 0, &never);
        }
      }
    }
    __syncwarp();
  }

  const int cols = static_cast<int>(p.N);
  const int64_t row0 = static_cast<int64_t>(m_blk) * kBM;
  const float alpha =
      kFmt == 0 ? __fmul_rn(__fdiv_rn(*p.inv_a, 6.0f), __fdiv_rn(inv, 6.0f)) : 1.0f;
  uint16_t* d = p.d + row0;
  if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------ epilogue
    const bool ready = warp_wait(acc_full, 0, abort_flag);
    if (!ready) {
      if (lane == 0) record_error(p.err, abort_flag, kErrGemmEpilogueWait);
    } else {
      tc_fence_after_sync();
      few_epilogue<BN>(p, tmem_base, joined, split, rank, nkb > 0, row0, cols, alpha, d, warp & 3, lane);
    }
  }
  if (split > 1) {
    tc_fence_before_sync();
    cluster_sync_all();  // every partial is with its rows' owner
    join_partials<BN>(p, joined, split, rank, row0, cols, alpha, d);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// 32 rows x 64 columns of the accumulator (this lane's row in ra and rb),
// scaled, rounded to bf16 and staged in shared memory as the 128-byte TMA
// swizzle has them.  Rows that are 16-byte aligned leave by TMA (clipped to
// D); others, and a row's end inside 16 bytes, four bytes a lane where the row
// is aligned to that and two elsewhere, consecutive lanes on consecutive
// columns: 6183 x 2821 x 176 in 17.7 us, x 2822 in 15.3, x 2824, by TMA, in
// 11.0.  The loops are unrolled no further than eight epilogue warps' registers
// go (twice as far: 20.7, 15.9 and 11.2).
__device__ __forceinline__ void store_box(const uint32_t (&ra)[32], const uint32_t (&rb)[32],
                                          float alpha, uint8_t* box, const CUtensorMap* tmD,
                                          const Fp4GemmParams& p, int row0, int64_t col0, int lane) {
  uint32_t w[32];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v0, v1;
    mul2_rn(ra[2 * j], ra[2 * j + 1], alpha, v0, v1);
    w[j] = cvt_bf16x2(v0, v1);
    mul2_rn(rb[2 * j], rb[2 * j + 1], alpha, v0, v1);
    w[16 + j] = cvt_bf16x2(v0, v1);
  }
  if (lane == 0) bulk_wait_group_read<0>();  // the box's last store has read it
  __syncwarp();
  const int sw = lane & 7;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((q ^ sw) << 4)) =
        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  // TMA writes whole 16 bytes, past the last column too.
  if (p.vec && (col0 + 64 <= p.N || (p.N & 7) == 0)) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmD, box, static_cast<int32_t>(col0), row0);
      bulk_commit_group();
    }
    return;
  }
  __syncwarp();
  const int rows = static_cast<int>(min(int64_t(32), p.M - row0));
  uint16_t* dst = p.d + static_cast<int64_t>(row0) * p.ldd + col0;
  if (rows == 32 && col0 + 64 <= p.N) {
    // Rows that are 4-byte aligned: all, every other one, or none.
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
    const bool alternate = (p.ldd & 1) != 0;
    auto words = [&](int r, uint16_t* to) {
      reinterpret_cast<uint32_t*>(to)[lane] = *reinterpret_cast<const uint32_t*>(
          box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    };
    auto halves = [&](int r, uint16_t* to) {
      const uint32_t at = r * 128 + (((lane >> 3) ^ (r & 7)) << 4) + (lane & 7) * 2;
      to[lane] = *reinterpret_cast<const uint16_t*>(box + at);
      to[lane + 32] = *reinterpret_cast<const uint16_t*>(box + (at ^ 64u));
    };
    if (alternate) {
      uint16_t* even_to = dst + odd * p.ldd;
      uint16_t* odd_to = dst + (odd ^ 1) * p.ldd;
#pragma unroll 2
      for (int r = 0; r < 32; r += 2, even_to += 2 * p.ldd, odd_to += 2 * p.ldd) {
        words(r + odd, even_to);
        halves(r + (odd ^ 1), odd_to);
      }
    } else if (odd == 0) {
#pragma unroll 4
      for (int r = 0; r < 32; ++r, dst += p.ldd) words(r, dst);
    } else {
#pragma unroll 4
      for (int r = 0; r < 32; ++r, dst += p.ldd) halves(r, dst);
    }
    __syncwarp();
    return;
  }
  const bool in0 = col0 + lane < p.N, in1 = col0 + lane + 32 < p.N;
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    const uint8_t* src = box + r * 128 + (lane & 7) * 2;
    const uint16_t v0 = *reinterpret_cast<const uint16_t*>(src + (((lane >> 3) ^ (r & 7)) << 4));
    const uint16_t v1 = *reinterpret_cast<const uint16_t*>(src + (((lane >> 3) + 4 ^ (r & 7)) << 4));
    if (r < rows) {
      if (in0) dst[r * p.ldd + lane] = v0;
      if (in1) dst[r * p.ldd + lane + 32] = v1;
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ CTA pairs
//
// Two CTAs share a 256 x BN tile as in the 8-bit pair kernel: each loads its
// 128 rows of A and half of B's rows, and the even CTA issues
// tcgen05.mma.cta_group::2 over both.  Each CTA's tensor memory holds the
// scales of its own rows of A and of all BN rows of B, so both load B's scale
// tiles whole.
//
// Two accumulators of BN = 256 columns and the scales do not fit the 512 columns
// of tensor memory, so the accumulators overlap by BN - kAcc1: the epilogue
// reads the shared columns first and announces them on `shared_free`, and the
// next tile's MMAs wait for that.
//
// Where the last wave of tiles fills at most half of the pairs and the K loop
// is long, each of its tiles runs as slices of the K loop on several pairs.
// A slice waits for the others of its tile only once every pair with a slice
// has begun.  Until then -- fewer SMs than the launch counted on, or another
// stream's kernels on them -- it leaves all of its partials and goes, and
// another one adds up what was left: no slice waits for one that may need its
// SM to start.  Products without slices have a kernel without that
// code (8192 x 14336 x 4096, MXFP4: 131 us, 134 with it).
//
// Bound by the tensor cores: 8192 x 14336 x 4096 takes 137 us in NVFP4 (7.0
// PFLOP/s) and 131 us in MXFP4 (7.3), which copies half as many scale tiles;
// the MMAs alone, without loads, take 133.  16384 x 4096 x 4096: 82 and 79 us.
// With short K loops (12288 x 6400 x 1600: 57 us) writing D bounds it.  Tiles
// of 128 and 192 columns need more loads an MMA than L2 delivers, and a second
// box for each epilogue warp's stores slows the MMAs by 1 %.
template <int kFmt, int BN, int STAGES, int EPI>
struct PairCfg {
  static constexpr int kKt = stage_ktiles<kFmt>();
  static constexpr int kRowTiles = 2;                    // rows of scale tiles under BN rows of B
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kBBytes = BN / 2 * kBKBytes;
  static constexpr int kSaBytes = kKt * kScTile;
  static constexpr int kSbBytes = kRowTiles * kKt * kScTile;
  static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr int kSfCols = 4 * kKt * (1 + kRowTiles);
  static constexpr int kSfa = 512 - kSfCols;
  static constexpr int kSfb = kSfa + 4 * kKt;
  static constexpr int kAcc1 = kSfa - BN;                // second accumulator's first column
  static constexpr int kBoxBytes = 32 * 128;             // 32 rows x 64 bf16 columns
  static constexpr int kGroups = BN / 64 / (EPI / 4);    // boxes an epilogue warp writes
  static constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(STAGES) * kStageBytes +
                                       static_cast<size_t>(EPI) * kBoxBytes + 256;
  static_assert(BN % 128 == 0 && BN <= 256 && kBBytes % 1024 == 0, "tile, whole scale tiles");
  static_assert(BN / 64 % (EPI / 4) == 0, "the epilogue warps of a quarter share the boxes");
  static_assert(kAcc1 < BN && BN - kAcc1 <= 64, "the overlap lies in one box");
  static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
};

// The t-th tile.  The larger operand is read once and the smaller again and
// again from L2: with at least as many columns as rows, all rows of tiles
// within a column of them; else groups of four rows of tiles, column by
// column.  8192 x 14336 x 4096: 137.6 us, 144.0 in groups of four; 16384 x
// 4096 x 4096: 82.1 us, 83.5 by whole columns.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int64_t t, int64_t num_m, int64_t num_n, int64_t group) {
  const int64_t g = t / (group * num_n);
  const int64_t r = t - g * group * num_n;
  const int64_t rows = min(group, num_m - g * group);
  return {static_cast<int>(g * group + r % rows), static_cast<int>(r / rows)};
}

// The t-th unit of work: a whole tile, or a slice of a tail tile's K loop.
struct Unit {
  int64_t tile;
  int kb0, kb1, slice;
  bool sliced;
};
template <bool kSliced>
__device__ __forceinline__ Unit unit_at(const Fp4GemmParams& p, int64_t t, int num_kb) {
  if (!kSliced || t < p.t_full) return {t, 0, num_kb, 0, false};
  const int64_t v = t - p.t_full;
  const int per = (num_kb + p.s_tail - 1) / p.s_tail;
  const int slice = static_cast<int>(v % p.s_tail);
  const int kb0 = min(num_kb, slice * per);
  return {p.t_full + v / p.s_tail, kb0, min(num_kb, kb0 + per), slice, true};
}

// One box of a slice's accumulator: 16-byte accesses, lane after lane.
__device__ __forceinline__ void store_partial(float* region, const uint32_t (&ra)[32],
                                              const uint32_t (&rb)[32], int lane) {
  uint4* dst = reinterpret_cast<uint4*>(region) + lane;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    __stcg(dst + q * 32, make_uint4(ra[4 * q], ra[4 * q + 1], ra[4 * q + 2], ra[4 * q + 3]));
    __stcg(dst + (8 + q) * 32, make_uint4(rb[4 * q], rb[4 * q + 1], rb[4 * q + 2], rb[4 * q + 3]));
  }
}

__device__ __forceinline__ void load_partial(const float* region, uint32_t (&ra)[32],
                                             uint32_t (&rb)[32], int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(region) + lane;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    uint32_t* r = q < 8 ? ra + 4 * q : rb + 4 * (q - 8);
    const uint4 v = __ldcg(src + q * 32);
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  }
}

// Adds one slice's partial of a box to the accumulator in ra and rb.
__device__ __forceinline__ void add_partial(const float* region, uint32_t (&ra)[32],
                                            uint32_t (&rb)[32], int lane) {
  const float4* src = reinterpret_cast<const float4*>(region) + lane;
  float4 v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] = __ldcg(src + q * 32);  // all in flight
  auto add = [](uint32_t& r, float x) { r = __float_as_uint(__uint_as_float(r) + x); };
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    uint32_t* r = q < 8 ? ra + 4 * q : rb + 4 * (q - 8);
    add(r[0], v[q].x);
    add(r[1], v[q].y);
    add(r[2], v[q].z);
    add(r[3], v[q].w);
  }
}

// A ticket counts the slices that have arrived in units of kArrived; below
// them it has a bit for each slice that left its own boxes too.
constexpr int kArrived = 256;

// Whether every pair with a slice is running: none of them waits for anything
// but the other slices, so a slice may then wait for these.  The last of the
// launch's epilogue warps to ask clears both counters for the next one.
__device__ __forceinline__ bool all_begun(int* begun, int pairs, int warps, int lane) {
  int seen = 0;
  if (lane == 0) {
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(begun) : "memory");
    if (atomicAdd(begun + 1, 1) == pairs * warps - 1) {
      atomicExch(begun, 0);
      atomicExch(begun + 1, 0);
    }
  }
  return __shfl_sync(0xFFFFFFFFu, seen, 0) >= pairs;
}

// Announce this warp's partials, and wait, bounded, for those of all slices:
// the ticket then, or -1.
__device__ __forceinline__ int wait_for_slices(int* ticket, int slices, volatile int* abort_flag,
                                               int lane) {
  __threadfence();
  __syncwarp();
  int seen = 0;
  if (lane == 0) {
    atomicAdd(ticket, kArrived);
    const uint64_t t0 = global_timer_ns();
    while (true) {
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(seen) : "l"(ticket) : "memory");
      if (seen >= slices * kArrived) break;
      if (*abort_flag || global_timer_ns() - t0 > kWaitLimitNs) {
        seen = -1;
        break;
      }
      __nanosleep(64);
    }
  }
  __syncwarp();  // lane 0's acquire holds for the warp
  return __shfl_sync(0xFFFFFFFFu, seen, 0);
}

// The same without the wait; the ticket with this slice.
__device__ __forceinline__ int leave_slice(int* ticket, int slice, int lane) {
  __threadfence();
  __syncwarp();
  int seen = 0;
  if (lane == 0) seen = atomicAdd(ticket, kArrived + (1 << slice)) + kArrived + (1 << slice);
  seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
  __threadfence();
  return seen;
}

// The last slice to finish clears both counters for the next call.
__device__ __forceinline__ void finish_slices(int* ticket, int slices, int lane) {
  __syncwarp();
  if (lane == 0 && atomicAdd(ticket + 1, 1) == slices - 1) {
    atomicExch(ticket, 0);
    atomicExch(ticket + 1, 0);
  }
}

template <int kFmt, int BN, int STAGES, int EPI, bool kSliced>
__global__ void __launch_bounds__(64 + 32 * EPI, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSa,
                         const __grid_constant__ CUtensorMap tmSb,
                         const __grid_constant__ CUtensorMap tmD,
                         const __grid_constant__ Fp4GemmParams p) {
  using C = PairCfg<kFmt, BN, STAGES, EPI>;
  constexpr int kKt = C::kKt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * C::kABytes;
  uint8_t* sEpi = sB + STAGES * C::kBBytes;
  uint8_t* sSa = sEpi + EPI * C::kBoxBytes;
  uint8_t* sSb = sSa + STAGES * C::kSaBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sSb + STAGES * C::kSbBytes);  // even CTA: both CTAs' loads
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;   // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2] even CTA: every epilogue warp of the pair
  uint64_t* shared_free = acc_empty + 2;  // [1] even CTA: the accumulators' shared columns
  uint64_t* drain = shared_free + 1;     // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // Written by the peer CTA before the closing cluster barrier: whether it
  // gave up, and (odd CTA -> even CTA) how many loads it issued into a stage.
  volatile uint32_t* peer_abort = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);
  volatile uint32_t* peer_fills = peer_abort + 1;      // [STAGES]
  volatile uint32_t* own_fills = peer_fills + STAGES;  // [STAGES]
  static_assert(sizeof(uint64_t) * (2 * STAGES + 6) + sizeof(uint32_t) * (3 + 2 * STAGES) <= 256,
                "barrier block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t pair = cluster_id_x(), num_pairs = cluster_count_x();
  const int64_t num_n = (p.N + BN - 1) / BN;
  const int64_t num_m = (p.M + 2 * kBM - 1) / (2 * kBM);
  const int64_t num_tiles = num_m * num_n;
  const int64_t group = p.N >= p.M ? num_m : 4;
  const int num_kb = static_cast<int>((p.K + kBK - 1) / kBK);
  const int64_t num_units = kSliced ? p.t_full + (num_tiles - p.t_full) * p.s_tail : num_tiles;
  // MMAs of the last stage; what follows K is zero in the codes and is not multiplied.
  const int last_steps = static_cast<int>((p.K - int64_t(num_kb - 1) * kBK + kMmaK - 1) / kMmaK);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 2 * EPI);
    }
    mbar_init(shared_free, 2 * EPI);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *peer_abort = 0;
    for (int s = 0; s < STAGES; ++s) peer_fills[s] = own_fills[s] = 0;
    fence_barrier_init();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmSa);
    tma_prefetch_map(&tmSb);
    tma_prefetch_map(&tmD);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync_all();  // barriers of both CTAs initialised before any remote use
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  if (kSliced && rank == 0 && threadIdx.x == 64 && pair < p.slice_pairs) atomicAdd(p.begun, 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producers (both CTAs)
    // The whole warp runs the loop and one elected lane issues, as below: one
    // lane alone took 45 ns more a K block, which bound the kernel.
    uint32_t fills[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES; ++s) fills[s] = 0;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = pair; ok && t < num_units; t += num_pairs) {
      const Unit u = unit_at<kSliced>(p, t, num_kb);
      const TileAt at = tile_at(u.tile, num_m, num_n, group);
      const int m0 = at.m * 2 * kBM + static_cast<int>(rank) * kBM;
      const int n0 = at.n * BN;
      for (int kb = u.kb0; kb < u.kb1; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t full_even = map_to_cta(smem_addr(&full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          tma_load_2d_pair(sA + stage * C::kABytes, &tmA, full_even, kb * kBKBytes, m0);
          tma_load_2d_pair(sB + stage * C::kBBytes, &tmB, full_even, kb * kBKBytes,
                           n0 + static_cast<int>(rank) * (BN / 2));
          tma_load_2d_pair(sSa + stage * C::kSaBytes, &tmSa, full_even, kb * kKt * kScElems,
                           m0 / kBM);
          tma_load_2d_pair(sSb + stage * C::kSbBytes, &tmSb, full_even, kb * kKt * kScElems,
                           n0 / 128);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
          if (s == stage) ++fills[s];
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      if (!ok) record_error(p.err, abort_flag, kErrGemmProducerWait);
      if (rank == 1) {
        const uint32_t even_fills = map_to_cta(smem_addr(const_cast<uint32_t*>(peer_fills)), 0);
#pragma unroll
        for (int s = 0; s < STAGES; ++s) st_shared_cluster_u32(even_fills + 4u * s, fills[s]);
      } else {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) own_fills[s] = fills[s];
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp runs the loop and one elected lane issues, so that the
    // operands of the copies and MMAs stay in uniform registers.
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0, shared_phase = 0;
      bool ok = true;
      bool issued = false;
      for (int64_t t = pair; ok && t < num_units; t += num_pairs) {
        ok = warp_wait(&acc_empty[acc], acc_phase ^ 1u, abort_flag);
        // The columns shared with the tile before this one (none before the first).
        if (ok && issued) {
          ok = warp_wait(shared_free, shared_phase, abort_flag);
          shared_phase ^= 1u;
        }
        if (!ok) break;
        tc_fence_after_sync();
        const Unit u = unit_at<kSliced>(p, t, num_kb);
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::kAcc1);
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          ok = warp_wait(&full[stage], phase, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t a_desc = smem_desc_k_sw128(smem_addr(sA + stage * C::kABytes));
          const uint64_t b_desc = smem_desc_k_sw128(smem_addr(sB + stage * C::kBBytes));
          const uint64_t sa_desc = smem_desc_scale(smem_addr(sSa + stage * C::kSaBytes));
          const uint64_t sb_desc = smem_desc_scale(smem_addr(sSb + stage * C::kSbBytes));
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kKt; ++i) {
              copy_scale_tile_pair(tmem_base + C::kSfa + 4 * i,
                                   sa_desc + static_cast<uint64_t>(i * (kScTile >> 4)));
#pragma unroll
              for (int r = 0; r < C::kRowTiles; ++r)
                copy_scale_tile_pair(
                    tmem_base + C::kSfb + 4 * (i * C::kRowTiles + r),
                    sb_desc + static_cast<uint64_t>((r * kKt + i) * (kScTile >> 4)));
            }
            auto step = [&](int k) {
              const int kt = kFmt == 0 ? k : k >> 1;
              const uint32_t idesc =
                  make_idesc_fp4<kFmt>(2 * kBM, BN, kFmt == 0 ? 0u : 2u * (k & 1));
              mma_fp4_pair<kFmt>(d_tmem, a_desc + static_cast<uint64_t>(2 * k),
                                 b_desc + static_cast<uint64_t>(2 * k), idesc,
                                 tmem_base + C::kSfa + 4 * kt,
                                 tmem_base + C::kSfb + 4 * C::kRowTiles * kt,
                                 (kb > u.kb0 || k > 0) ? 1u : 0u);
            };
            if (kb + 1 < num_kb || last_steps == 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k) step(k);
            } else {
#pragma unroll 1
              for (int k = 0; k < last_steps; ++k) step(k);
            }
            mma_commit_pair_multicast(&empty[stage], 0x3);
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair_multicast(&acc_full[acc], 0x3);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && elect_one()) {
        record_error(p.err, abort_flag, kErrGemmMmaWait);
        if (issued) {
          volatile int never = 0;
          mma_commit_pair_multicast(drain, 0x1);
          mbar_wait_bounded(drain, 0, &never);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;  // which of the quarter's warps (0 when EPI == 4)
    const float alpha =
        kFmt == 0 ? __fmul_rn(__fdiv_rn(*p.inv_a, 6.0f), __fdiv_rn(*p.inv_b, 6.0f)) : 1.0f;
    const uint32_t acc_empty_even = map_to_cta(smem_addr(acc_empty), 0);
    const uint32_t shared_free_even = map_to_cta(smem_addr(shared_free), 0);
    uint8_t* box = sEpi + (warp - 2) * C::kBoxBytes;
    int acc = 0;
    uint32_t acc_phase = 0;
    // This warp's place among the epilogue warps of the tail tiles, and one of
    // its boxes' partial (2048 floats) of a slice.
    auto warp_slot = [&](const Unit& u) {
      return static_cast<int>(u.tile - p.t_full) * 2 * EPI + static_cast<int>(rank) * EPI + part * 4 + quarter;
    };
    auto partial_of = [&](const Unit& u, int slice, int i) {
      const int64_t tail = (u.tile - p.t_full) * p.s_tail + slice;
      return p.partials + ((tail * 8 + static_cast<int>(rank) * 4 + quarter) * (BN / 64) + i) * 2048;
    };
    for (int64_t t = pair; t < num_units; t += num_pairs) {
      const Unit u = unit_at<kSliced>(p, t, num_kb);
      const TileAt at = tile_at(u.tile, num_m, num_n, group);
      const int row0 = at.m * 2 * kBM + static_cast<int>(rank) * kBM + quarter * 32;
      const int64_t n0 = static_cast<int64_t>(at.n) * BN;
      // Asked while the slice's MMAs run, which hides the counter's round trips.
      const bool meet = kSliced && u.sliced && all_begun(p.begun, p.slice_pairs, 2 * EPI, lane);
      const bool ready =
          __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&acc_full[acc], acc_phase, abort_flag));
      if (!ready) {
        if (lane == 0) record_error(p.err, abort_flag, kErrGemmEpilogueWait);
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * C::kAcc1);
#pragma unroll 1
      for (int g = 0; g < C::kGroups; ++g) {
        // The first accumulator's shared columns are its last, the second's its first.
        const int i = part * C::kGroups + (acc == 0 ? C::kGroups - 1 - g : g);
        const int64_t col0 = n0 + 64 * i;
        const bool live = row0 < p.M && col0 < p.N;
        // A slice owns every s_tail-th box of a warp and hands over the others;
        // its own too where it may not wait for the other slices.
        const bool kept = meet && i % p.s_tail == u.slice;
        uint32_t ra[32], rb[32];
        if (live && !kept) {
          tmem_load_32cols(t_row + 64 * i, ra);
          tmem_load_32cols(t_row + 64 * i + 32, rb);
          tmem_load_wait();
        }
        if (g == 0 || g == C::kGroups - 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (g == 0) mbar_arrive_cluster_tmem(shared_free_even);
            if (g == C::kGroups - 1) mbar_arrive_cluster_tmem(acc_empty_even + 8u * acc);
          }
        }
        if (live && !(kSliced && u.sliced)) store_box(ra, rb, alpha, box, &tmD, p, row0, col0, lane);
        if constexpr (kSliced)
          if (live && u.sliced && !kept) store_partial(partial_of(u, u.slice, i), ra, rb, lane);
      }
      if (kSliced && u.sliced && row0 < p.M) {
        // The pair's last unit: its accumulator stays where it is.  A box is
        // its owner's partial plus the others in order, whoever adds them up:
        // the owner, or, where that has left, the first slice that waited, or
        // the last one to arrive if none did.
        int* ticket = p.tickets + 2 * warp_slot(u);
        const int all = (1 << p.s_tail) - 1;
        int left;
        if (meet) {
          const int seen = wait_for_slices(ticket, p.s_tail, abort_flag, lane);
          if (seen < 0) {
            if (lane == 0) record_error(p.err, abort_flag, kErrGemmEpilogueWait);
            break;
          }
          left = seen & (kArrived - 1);
          if (__ffs(~left & all) - 1 != u.slice) left = 0;
        } else {
          left = leave_slice(ticket, u.slice, lane) == p.s_tail * kArrived + all ? all : 0;
        }
#pragma unroll 1
        for (int i = part * C::kGroups; i < (part + 1) * C::kGroups; ++i) {
          const int64_t col0 = n0 + 64 * i;
          const int owner = i % p.s_tail;
          const bool kept = meet && owner == u.slice;
          if ((!kept && (left >> owner & 1) == 0) || col0 >= p.N) continue;
          uint32_t ra[32], rb[32];
          if (kept) {
            tmem_load_32cols(t_row + 64 * i, ra);
            tmem_load_32cols(t_row + 64 * i + 32, rb);
            tmem_load_wait();
          } else {
            load_partial(partial_of(u, owner, i), ra, rb, lane);
          }
          for (int o = 0; o < p.s_tail; ++o)
            if (o != owner) add_partial(partial_of(u, o, i), ra, rb, lane);
          store_box(ra, rb, alpha, box, &tmD, p, row0, col0, lane);
        }
        finish_slices(ticket, p.s_tail, lane);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  __syncwarp();
  __syncthreads();  // every role of this CTA is done: its abort flag is final
  if (threadIdx.x == 0)
    st_shared_cluster_u32(map_to_cta(smem_addr(const_cast<uint32_t*>(peer_abort)), rank ^ 1u),
                          *abort_flag != 0 ? 1u : 0u);
  tc_fence_before_sync();
  cluster_sync_all();  // no CTA leaves while its peer may still read its shared memory
  // After a failure, loads may be in flight: the even CTA balances each
  // stage's last phase (its full[] counts both CTAs' bytes) and waits,
  // bounded, for it, as the 8-bit pair kernel does.
  if (*abort_flag != 0 || *peer_abort != 0) {
    if (rank == 0 && threadIdx.x == 0) {
      volatile int never = 0;
#pragma unroll
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t fe = own_fills[s], fo = peer_fills[s];
        if (fo > fe) mbar_arrive_expect_tx(&full[s], C::kStageBytes);
        if (fe > fo) mbar_complete_tx(&full[s], C::kStageBytes);
        const uint32_t last = fe > fo ? fe : fo;
        if (last > 0) mbar_wait_bounded(&full[s], (last - 1) & 1u, &never);
      }
    }
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Shared memory of a kernel instance, allowed once a device.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t bytes, const DeviceInfo& dev, bool (&done)[64]) {
  static std::mutex mu;
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev.device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(bytes));
  done[dev.device] = e == cudaSuccess;
  return e;
}

// The same for a kernel of CTA pairs, and how many pairs are resident at once.
template <typename Kernel>
cudaError_t pair_setup(Kernel kernel, size_t bytes, int threads, const DeviceInfo& dev, int (&slots)[64],
                       bool (&done)[64]) {
  const cudaError_t e = allow_smem(kernel, bytes, dev, done);
  if (e != cudaSuccess) return e;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (slots[dev.device] > 0) return cudaSuccess;
  cudaLaunchConfig_t probe = {};
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = 2;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  probe.gridDim = dim3(2 * (dev.num_sms / 2));
  probe.blockDim = dim3(threads);
  probe.dynamicSmemBytes = bytes;
  probe.attrs = &cluster;
  probe.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &probe) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = dev.num_sms / 2;
  }
  slots[dev.device] = n;
  return cudaSuccess;
}

// Codes of one operand: boxes of 128 bytes of K.  The rows end at their last
// 32 values; the box is zero past that, and past the last row.
bool make_code_map(CUtensorMap* map, const Fp4View& v, int64_t rows, int64_t K, int box_rows) {
  return make_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, v.codes,
                     static_cast<uint64_t>((K + 31) / 32 * 16), static_cast<uint64_t>(rows),
                     static_cast<uint64_t>(v.ld), kBKBytes, static_cast<uint32_t>(box_rows),
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles of one operand, a row of tiles for 128 rows: boxes of a
// stage's tiles along K and `box_rows` rows of tiles, zero past the last.
template <int kFmt>
bool make_scale_map(CUtensorMap* map, const Fp4View& v, int64_t rows, int64_t K, int box_rows) {
  const uint64_t elems = static_cast<uint64_t>(fp4_scale_ktiles(K, kFmt)) * kScElems;
  return make_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, v.scales, elems,
                     static_cast<uint64_t>((rows + 127) / 128), elems * 8,
                     stage_ktiles<kFmt>() * kScElems, static_cast<uint32_t>(box_rows),
                     CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The K split of the few-tile kernel: a power of two, at most `most` CTAs and
// at least two stages each.
int few_split(int64_t tiles, int64_t K, int64_t most) {
  const int64_t num_kb = (K + kBK - 1) / kBK;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= most && num_kb >= split * 4) split *= 2;
  return split;
}

template <int kFmt, int BN, int STAGES>
cudaError_t run_few(const Fp4GemmArgs& g, Fp4GemmParams p, const DeviceInfo& dev,
                    cudaStream_t stream) {
  using C = FewCfg<kFmt, BN, STAGES>;
  p.M = g.N;
  p.N = g.M;
  CUtensorMap tmA, tmB, tmSa, tmSb;
  if (!make_code_map(&tmA, g.b, p.M, p.K, kBM) || !make_code_map(&tmB, g.a, p.N, p.K, BN) ||
      !make_scale_map<kFmt>(&tmSa, g.b, p.M, p.K, 1) || !make_scale_map<kFmt>(&tmSb, g.a, p.N, p.K, 1))
    return map_failed("fp4 gemm operand");
  auto* kernel = gemm_fp4_few_kernel<kFmt, BN, STAGES>;
  static bool done[64] = {};
  cudaError_t e = allow_smem(kernel, C::kSmemBytes + joined_bytes<BN>(2), dev, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.M + kBM - 1) / kBM) * ((p.N + BN - 1) / BN);
  // Two CTAs an SM where the weight's loads bound it (up to 32 tokens); one
  // where the partials are larger: 64 x 4096 x 4096 6.7 us against 8.3.
  const int split = few_split(tiles, p.K, (BN <= 32 ? 2 : 1) * int64_t(dev.num_sms));
  set_error_site("gemm_fp4_few_kernel");
  return launch_kernel(kernel, dim3(static_cast<unsigned>(tiles * split)), dim3(kThreads),
                       C::kSmemBytes + joined_bytes<BN>(split), stream, split, false, tmA, tmB, tmSa,
                       tmSb, p, split, g.b_early);
}

// How the fused product runs these sizes; stages 0: it does not.
struct FusedPlan {
  int split, per, stages;
};

template <int kFmt, int BN>
FusedPlan plan_fused(const Fp4GemmArgs& g, const DeviceInfo& dev) {
  using C = FusedCfg<kFmt, BN>;
  const int64_t num_kb = (g.K + kBK - 1) / kBK, tiles = (g.N + kBM - 1) / kBM;
  // Tiles for most SMs: one CTA each, with all of its shared memory for loads
  // in flight and nothing to join.
  if (2 * tiles > dev.num_sms && g.M * num_kb * 16 <= kFusedUnits) {
    const int n = C::stages(num_kb, 1, kFusedSmemFull);
    if (n >= num_kb || n >= 6) return {1, static_cast<int>(num_kb), n};
  }
  const int split = few_split(tiles, g.K, 2 * int64_t(dev.num_sms));
  const int64_t per = (num_kb + split - 1) / split;
  if (g.M * per * 16 > kFusedUnits) return {split, 0, 0};  // the values would not stay in registers
  const int n = C::stages(per, split, kFusedSmemHalf);
  return {split, static_cast<int>(per), n >= per || n >= 3 ? n : 0};
}

template <int kFmt, int BN>
cudaError_t run_fused(const Fp4GemmArgs& g, const Fp4QuantArgs& x, Fp4GemmParams p,
                      const DeviceInfo& dev, cudaStream_t stream) {
  using C = FusedCfg<kFmt, BN>;
  p.M = g.N;
  p.N = g.M;
  const FusedPlan f = plan_fused<kFmt, BN>(g, dev);
  CUtensorMap tmA, tmSa;
  if (!make_code_map(&tmA, g.b, p.M, p.K, kBM) || !make_scale_map<kFmt>(&tmSa, g.b, p.M, p.K, 1))
    return map_failed("fp4 gemm operand");
  FusedTokens t;
  t.x = x.x;
  t.span = span_of(x.x, x.rows, x.cols, x.ld);
  t.ldx = x.ld;
  t.amax_in = x.amax_in;
  t.scale_in = x.scale_in;
  t.inv_in = x.inv_in;
  t.eps = x.eps;
  // A stored scale's call records the amax beside it.
  t.amax_out = x.scale_in != nullptr ? reinterpret_cast<float*>(x.amax_rec) : x.amax_out;
  t.scale_out = x.scale_out;
  t.inv_out = x.inv_out;
  t.own_inv = x.own_inv;
  t.codes = x.out.codes;
  t.ld4 = x.out.ld;
  t.scales = x.out.scales;
  const int align = row_align(x.x, x.ld, 2);
  auto* kernel = align == kAlign32   ? gemm_fp4_fused_kernel<kFmt, BN, kAlign32>
                 : align == kAlign16 ? gemm_fp4_fused_kernel<kFmt, BN, kAlign16>
                                     : gemm_fp4_fused_kernel<kFmt, BN, kScalar>;
  static bool done[3][64] = {};
  cudaError_t e = allow_smem(kernel, kFusedSmemFull, dev, done[align]);
  if (e != cudaSuccess) return e;
  const size_t bytes = C::kFixed + joined_bytes<BN>(f.split) +
                       static_cast<size_t>(f.stages) * C::kRingBytes +
                       static_cast<size_t>(f.per) * (C::kBBytes + C::kScBytes);
  const int64_t tiles = (p.M + kBM - 1) / kBM;
  set_error_site("gemm_fp4_fused_kernel");
  return launch_kernel(kernel, dim3(static_cast<unsigned>(tiles * f.split)), dim3(kFusedThreads),
                       bytes, stream, f.split, false, tmA, tmSa, p, t, f.split, f.stages);
}

template <int kFmt, int BN, int STAGES, int EPI, bool kSliced>
cudaError_t pair_slots(const DeviceInfo& dev, int64_t* slots) {
  static bool done[64] = {};
  static int resident[64] = {};
  const cudaError_t e = pair_setup(gemm_fp4_pair_kernel<kFmt, BN, STAGES, EPI, kSliced>,
                                   PairCfg<kFmt, BN, STAGES, EPI>::kSmemBytes, 64 + 32 * EPI, dev,
                                   resident, done);
  if (e == cudaSuccess) *slots = resident[dev.device];
  return e;
}

template <int kFmt, int BN, int STAGES, int EPI, bool kSliced>
cudaError_t run_pair(const Fp4View& a, const Fp4View& b, const Fp4GemmParams& p, const DeviceInfo& dev,
                     cudaStream_t stream) {
  using C = PairCfg<kFmt, BN, STAGES, EPI>;
  CUtensorMap tmA, tmB, tmSa, tmSb, tmD;
  if (!make_code_map(&tmA, a, p.M, p.K, kBM) || !make_code_map(&tmB, b, p.N, p.K, BN / 2) ||
      !make_scale_map<kFmt>(&tmSa, a, p.M, p.K, 1) ||
      !make_scale_map<kFmt>(&tmSb, b, p.N, p.K, C::kRowTiles))
    return map_failed("fp4 pair gemm operand");
  // Rows that TMA cannot store are written from shared memory: no map then.
  if (!p.vec)
    tmD = tmA;
  else if (!make_map_2d(&tmD, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.d, static_cast<uint64_t>(p.N),
                        static_cast<uint64_t>(p.M), static_cast<uint64_t>(p.ldd) * 2, 64, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B))
    return map_failed("fp4 pair gemm output");
  int64_t slots = 0;
  const cudaError_t e = pair_slots<kFmt, BN, STAGES, EPI, kSliced>(dev, &slots);
  if (e != cudaSuccess) return e;
  const int64_t units = p.t_full + p.slice_pairs;
  const unsigned pairs = static_cast<unsigned>(units < slots ? units : slots);
  set_error_site("gemm_fp4_pair_kernel");
  return launch_kernel(gemm_fp4_pair_kernel<kFmt, BN, STAGES, EPI, kSliced>, dim3(2 * pairs),
                       dim3(64 + 32 * EPI), C::kSmemBytes, stream, 2, false, tmA, tmB, tmSa, tmSb,
                       tmD, p);
}

// What joining the slices of the last wave costs, in K blocks of a tile: 6 us
// for two or four slices and 8 for three, whose warps have two boxes to add up
// in one slice and one in the others; four have more to wait for where TMA
// cannot write y's rows.  A block takes 0.3 us, 0.43 where the rows of codes
// are not whole 128-byte lines.  Sliced against whole, us, around the limits:
//   4096 x 1600 (two slices)   8192 25.1 24.2, 10240 28.3 28.3, 12288 31.8 32.6
//   2560 x 2560 (three)        8192 25.5 24.1, 10240 28.3 28.4, 12288 31.3 32.6
//   2500 x 2504 (three)        7000 28.7 29.1;  2500 x 2500: 30.8 30.2
//   2304 x 2304 (four)         6144 21.2 20.0, 7168 22.2 22.0, 8192 23.4 24.2
//   2200 x 2250 (four)         8192 28.3 25.7, 12288 32.4 34.1
int join_blocks(int64_t ways, bool vec) {
  return ways == 2 ? 20 : ways == 3 ? 26 : vec ? 21 : 31;
}

// Whole tiles, and the last wave's as K slices where that saves more than it costs.
void plan_tail(Fp4GemmParams& p, int64_t slots, int BN, size_t split_bytes, bool whole_lines) {
  const int64_t tiles = ((p.M + 2 * kBM - 1) / (2 * kBM)) * ((p.N + BN - 1) / BN);
  p.t_full = tiles;
  p.s_tail = 1;
  p.slice_pairs = 0;
  const int64_t tail = tiles % slots, num_kb = (p.K + kBK - 1) / kBK;
  if (tail == 0 || p.partials == nullptr) return;
  int64_t ways = slots / tail < 4 ? slots / tail : 4;
  const int64_t fit = static_cast<int64_t>(split_bytes) / (tail * 2 * kBM * BN * 4);
  if (fit < ways) ways = fit;
  if (ways < 2 || tail * 32 > kWsTickets) return;
  if (num_kb * (ways - 1) * (whole_lines ? 30 : 43) < join_blocks(ways, p.vec) * 30 * ways) return;
  p.t_full = tiles - tail;
  p.s_tail = static_cast<int>(ways);
  p.slice_pairs = static_cast<int>(tail * ways);  // t_full is a multiple of slots, or 0
}

constexpr int64_t kDeepK = 24 * kBK;

template <int kFmt>
cudaError_t run_fmt(const Fp4GemmArgs& g, Fp4GemmParams p, const DeviceInfo& dev,
                    cudaStream_t stream) {
  // The few-tile kernel while its tiles are one wave, two CTAs an SM:
  // 512 x 4096 x 4096 takes 10.6 us there and 11.7 us in pairs, 1024 x 4096 x
  // 4096 (two waves) 20.0 and 11.7.
  if (g.M <= 16) return run_few<kFmt, 16, 4>(g, p, dev, stream);
  if (g.M <= 32) return run_few<kFmt, 32, kFmt == 0 ? 3 : 4>(g, p, dev, stream);
  const int64_t tiles = (g.M + 63) / 64 * ((g.N + kBM - 1) / kBM);
  // Long K loops, one CTA an SM: the second CTA's shared memory as stages too.
  // 256 x 4096 x 16384: 22.8 us against 27.2, 256 x 4096 x 6144 11.1 against
  // 11.8, but 256 x 4096 x 4096 8.8 against 8.6.
  if (tiles <= dev.num_sms && g.K >= kDeepK)
    return run_few<kFmt, 64, 6>(g, p, dev, stream);
  if (tiles <= 2 * int64_t(dev.num_sms)) return run_few<kFmt, 64, 3>(g, p, dev, stream);
  constexpr int kTileN = 256, kStages = 5;
  int64_t slots = 0;
  const cudaError_t e = pair_slots<kFmt, kTileN, kStages, 4, true>(dev, &slots);
  if (e != cudaSuccess) return e;
  plan_tail(p, slots, kTileN, g.ws_split_bytes, ((g.a.ld | g.b.ld) & 127) == 0);
  if (p.s_tail > 1)
    return p.vec ? run_pair<kFmt, kTileN, kStages, 4, true>(g.a, g.b, p, dev, stream)
                 : run_pair<kFmt, kTileN, kStages, 8, true>(g.a, g.b, p, dev, stream);
  // Eight epilogue warps where writing a tile takes longer than multiplying
  // it -- a short K, or rows that TMA cannot store -- and four elsewhere:
  // 4096 x 4096 x 512 11.1 us against 13.2, 8192 x 8192 x 1024 35.9 against
  // 37.7, 777 x 4801 x 1600 9.8 against 11.6, but 8192 x 8192 x 2048 55.1
  // against 50.9.
  if (!p.vec || g.K <= 4 * kBK)
    return run_pair<kFmt, kTileN, kStages, 8, false>(g.a, g.b, p, dev, stream);
  return run_pair<kFmt, kTileN, kStages, 4, false>(g.a, g.b, p, dev, stream);
}

}  // namespace

namespace {

Fp4GemmParams base_params(const Fp4GemmArgs& g) {
  Fp4GemmParams p;
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.inv_a = g.inv_a;
  p.inv_b = g.inv_b;
  p.d = static_cast<uint16_t*>(g.d);
  p.ldd = g.ldd;
  p.err = g.ws_error;
  p.partials = g.ws_split;
  p.tickets = g.ws_tickets;
  p.begun = g.ws_begun;
  p.vec = (reinterpret_cast<uintptr_t>(g.d) & 15u) == 0 && g.ldd % 8 == 0;
  return p;
}

// The few-tile kernels take the weight as their A.
Fp4GemmParams swapped(Fp4GemmParams p) {
  const float* a = p.inv_a;
  p.inv_a = p.inv_b;
  p.inv_b = a;
  return p;
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4GemmArgs& g, const DeviceInfo& dev, cudaStream_t stream) {
  const Fp4GemmParams p = base_params(g);
  return g.fmt == 0 ? run_fmt<0>(g, p, dev, stream) : run_fmt<1>(g, p, dev, stream);
}

bool fp4_fused_fits(const Fp4GemmArgs& g, const DeviceInfo& dev) {
  if (g.M > 32) return false;
  const FusedPlan f = g.fmt == 0 ? (g.M <= 16 ? plan_fused<0, 16>(g, dev) : plan_fused<0, 32>(g, dev))
                                 : (g.M <= 16 ? plan_fused<1, 16>(g, dev) : plan_fused<1, 32>(g, dev));
  return f.stages > 0;
}

cudaError_t launch_fp4_fused(const Fp4GemmArgs& g, const Fp4QuantArgs& x, const DeviceInfo& dev,
                             cudaStream_t stream) {
  const Fp4GemmParams p = swapped(base_params(g));
  if (g.fmt == 0)
    return g.M <= 16 ? run_fused<0, 16>(g, x, p, dev, stream) : run_fused<0, 32>(g, x, p, dev, stream);
  return g.M <= 16 ? run_fused<1, 16>(g, x, p, dev, stream) : run_fused<1, 32>(g, x, p, dev, stream);
}

}  // namespace fp8lin
