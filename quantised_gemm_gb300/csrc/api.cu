// api.cu -- the C ABI of libfp8lin: argument checks, orchestration of the
// forward and backward of the fp8 Linear on the caller's stream, workspace
// layout, error reporting and the measurement hooks.  No device memory is
// allocated here; every buffer comes from the caller.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/fp8lin.h"
#include "internal.h"

namespace fp8lin {
namespace {

thread_local int g_last_cuda_error = 0;
thread_local const char* g_error_site = nullptr;
thread_local char g_error_detail[256];
std::atomic<uint64_t> g_launches{0};

// Record a failed CUDA call: its error, and where (the site a launcher named
// with set_error_site, else the line of this file that saw the failure).
fp8lin_status cuda_fail(cudaError_t e, int line = __builtin_LINE()) {
  g_last_cuda_error = static_cast<int>(e);
  if (g_error_site != nullptr)
    std::snprintf(g_error_detail, sizeof(g_error_detail), "%s in %s", cudaGetErrorName(e),
                  g_error_site);
  else
    std::snprintf(g_error_detail, sizeof(g_error_detail), "%s at api.cu:%d", cudaGetErrorName(e),
                  line);
  g_error_site = nullptr;
  return FP8LIN_ECUDA;
}

// ---------------------------------------------------------------- profiling

constexpr int kProfPairs = 8192;
struct ProfRecord {
  cudaEvent_t start, stop;
  int kind;
};
bool g_prof_on = false;
int g_prof_used = 0;
ProfRecord g_prof[kProfPairs];
bool g_prof_created[kProfPairs];

struct ProfScope {
  ProfRecord* rec = nullptr;
  cudaStream_t stream;
  ProfScope(int kind, cudaStream_t s) : stream(s) {
    g_launches.fetch_add(1, std::memory_order_relaxed);
    if (!g_prof_on || g_prof_used >= kProfPairs) return;
    const int i = g_prof_used;
    if (!g_prof_created[i]) {
      if (cudaEventCreate(&g_prof[i].start) != cudaSuccess) return;
      if (cudaEventCreate(&g_prof[i].stop) != cudaSuccess) return;
      g_prof_created[i] = true;
    }
    rec = &g_prof[i];
    rec->kind = kind;
    ++g_prof_used;
    cudaEventRecord(rec->start, stream);
  }
  ~ProfScope() {
    if (rec) cudaEventRecord(rec->stop, stream);
  }
};

// ---------------------------------------------------------------- helpers

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int* ws_error(void* ws) {
  return reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsErrorOffset);
}
uint32_t* ws_u32(void* ws, size_t off) {
  return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + off);
}

bool valid_fmt(int32_t f) { return f == FP8LIN_E4M3 || f == FP8LIN_E5M2; }

// Checks shared by amax and cast: bf16 [rows, cols] with row stride ld.
fp8lin_status check_bf16(const void* x, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0) return FP8LIN_EINVAL;
  if (rows == 0 || cols == 0) return FP8LIN_OK;
  if (x == nullptr || !aligned16(x)) return FP8LIN_EINVAL;
  if (ld < cols) return FP8LIN_EINVAL;
  if (cols % 16 != 0 || ld % 8 != 0) return FP8LIN_EUNSUPPORTED;
  if (rows > (int64_t(1) << 31) || cols > (int64_t(1) << 31)) return FP8LIN_EUNSUPPORTED;
  return FP8LIN_OK;
}

fp8lin_status check_state(const fp8lin_scaling_state* st, bool need_delayed_buffers) {
  if (st == nullptr) return FP8LIN_EINVAL;
  if (!valid_fmt(st->fmt)) return FP8LIN_EUNSUPPORTED;
  if (st->kind != FP8LIN_DYNAMIC && st->kind != FP8LIN_DELAYED) return FP8LIN_EUNSUPPORTED;
  if (st->amax == nullptr || st->scale == nullptr || st->inv_scale == nullptr)
    return FP8LIN_EINVAL;
  if (!(st->eps > 0.0f)) return FP8LIN_EINVAL;
  if (st->kind == FP8LIN_DELAYED && need_delayed_buffers) {
    if (st->history_len < 1) return FP8LIN_EINVAL;
    if (st->amax_history == nullptr || st->head == nullptr) return FP8LIN_EINVAL;
  }
  if (st->amax_algo < FP8LIN_AMAX_ATOMIC || st->amax_algo > FP8LIN_AMAX_PRECOMPUTED)
    return FP8LIN_EUNSUPPORTED;
  if (st->amax_algo == FP8LIN_AMAX_PRECOMPUTED && st->kind != FP8LIN_DYNAMIC)
    return FP8LIN_EUNSUPPORTED;  // delayed scaling records the amax in its own cast pass
  return FP8LIN_OK;
}

// amax into a device fp32 (ATOMIC or REDUCTION).
fp8lin_status do_amax(const void* x, int64_t rows, int64_t cols, int64_t ld, float* amax_out,
                      int32_t algo, void* ws, const DeviceInfo& dev, cudaStream_t stream) {
  uint32_t* out_bits = reinterpret_cast<uint32_t*>(amax_out);
  if (rows == 0 || cols == 0) {
    cudaError_t e = cudaMemsetAsync(amax_out, 0, sizeof(float), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  const int grid = amax_grid(dev, rows, cols);
  if (algo == FP8LIN_AMAX_REDUCTION) {
    uint32_t* part = ws_u32(ws, kWsPartialOffset);
    {
      ProfScope ps(FP8LIN_PROF_AMAX, stream);
      cudaError_t e = launch_amax(static_cast<const uint16_t*>(x), rows, cols, ld, part, false,
                                  grid, stream);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    ProfScope ps(FP8LIN_PROF_AMAX, stream);
    cudaError_t e = launch_amax_final(part, grid, out_bits, stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  if (ws != nullptr) {
    // One atomic max per CTA through the workspace's self-cleaning words.
    ProfScope ps(FP8LIN_PROF_AMAX, stream);
    cudaError_t e = launch_amax(static_cast<const uint16_t*>(x), rows, cols, ld, out_bits, true,
                                grid, stream, ws_u32(ws, kWsAtomicAccOffset),
                                ws_u32(ws, kWsAtomicTicketOffset));
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  cudaError_t e = cudaMemsetAsync(amax_out, 0, sizeof(float), stream);
  if (e != cudaSuccess) return cuda_fail(e);
  ProfScope ps(FP8LIN_PROF_AMAX, stream);
  e = launch_amax(static_cast<const uint16_t*>(x), rows, cols, ld, out_bits, true, grid, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status do_cast(const CastArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return FP8LIN_OK;
  ProfScope ps(FP8LIN_PROF_CAST, stream);
  cudaError_t e = launch_cast(a, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

// Dynamic scaling of one tensor: amax -> scale -> cast (+T) per st->amax_algo.
// FP8LIN_PAIR_CAST=0 casts x and W of the forward in separate launches even
// where one paired single pass would take both.
bool pair_cast_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("FP8LIN_PAIR_CAST");
    return !(v != nullptr && v[0] == '0');
  }();
  return on;
}

bool single_pass_algo(int32_t algo) {
  return algo == FP8LIN_AMAX_AUTO || algo == FP8LIN_AMAX_SINGLE_PASS;
}

SinglePassArgs single_pass_args(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                const fp8lin_scaling_state* st, uint8_t* out, uint8_t* out_t,
                                void* ws) {
  SinglePassArgs sp;
  sp.x = static_cast<const uint16_t*>(x);
  sp.rows = rows;
  sp.cols = cols;
  sp.ld = ld;
  sp.fmt = st->fmt;
  sp.eps = st->eps;
  sp.amax_out = st->amax;
  sp.scale_out = st->scale;
  sp.inv_out = st->inv_scale;
  sp.out = out;
  sp.out_t = out_t;
  sp.ws_barrier = ws_u32(ws, kWsBarrierOffset);
  sp.ws_exits = ws_u32(ws, kWsExitsOffset);
  sp.ws_amax = ws_u32(ws, kWsAmaxOffset);
  sp.ws_error = ws_error(ws);
  return sp;
}

// SINGLE_PASS falls back to ATOMIC when the tensor does not fit on chip and
// `allow_fallback` is set.  PRECOMPUTED takes *st->amax as given (written by
// the producer of x, e.g. a GEMM epilogue) and runs scale + cast only.
fp8lin_status cast_dynamic_scaled(const void* x, int64_t rows, int64_t cols, int64_t ld,
                           const fp8lin_scaling_state* st, uint8_t* out, uint8_t* out_t, void* ws,
                           const DeviceInfo& dev, cudaStream_t stream, bool allow_fallback) {
  int32_t algo = st->amax_algo;
  if ((algo == FP8LIN_AMAX_SINGLE_PASS || algo == FP8LIN_AMAX_AUTO) && rows > 0 && cols > 0) {
    const bool cluster = cluster_cast_fits(rows, cols);
    if (cluster || single_pass_fits(dev, rows, cols)) {
      SinglePassArgs sp;
      sp.x = static_cast<const uint16_t*>(x);
      sp.rows = rows;
      sp.cols = cols;
      sp.ld = ld;
      sp.fmt = st->fmt;
      sp.eps = st->eps;
      sp.amax_out = st->amax;
      sp.scale_out = st->scale;
      sp.inv_out = st->inv_scale;
      sp.out = out;
      sp.out_t = out_t;
      sp.ws_barrier = ws_u32(ws, kWsBarrierOffset);
      sp.ws_exits = ws_u32(ws, kWsExitsOffset);
      sp.ws_amax = ws_u32(ws, kWsAmaxOffset);
      sp.ws_error = ws_error(ws);
      ProfScope ps(FP8LIN_PROF_CAST_FUSED, stream);
      cudaError_t e =
          cluster ? launch_cast_cluster(sp, stream) : launch_cast_single_pass(sp, dev, stream);
      return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
    }
    if (!allow_fallback && algo == FP8LIN_AMAX_SINGLE_PASS) return FP8LIN_EUNSUPPORTED;
    algo = FP8LIN_AMAX_ATOMIC;
  }
  if (algo != FP8LIN_AMAX_PRECOMPUTED) {
    fp8lin_status s = do_amax(x, rows, cols, ld, st->amax, algo, ws, dev, stream);
    if (s != FP8LIN_OK) return s;
  }
  if (rows == 0 || cols == 0) {
    ProfScope ps(FP8LIN_PROF_SCALE, stream);
    cudaError_t e = launch_scale(st->amax, st->scale, st->inv_scale, nullptr, nullptr, 1, false,
                                 st->fmt, st->eps, stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  CastArgs c;
  c.x = static_cast<const uint16_t*>(x);
  c.rows = rows;
  c.cols = cols;
  c.ld = ld;
  c.fmt = st->fmt;
  c.scale_in = nullptr;
  c.amax_in = st->amax;
  c.derive_scale = true;
  c.eps = st->eps;
  c.scale_out = st->scale;
  c.inv_out = st->inv_scale;
  c.out = out;
  c.out_t = out_t;
  c.amax_rec = nullptr;
  c.err = ws_error(ws);
  return do_cast(c, dev, stream);
}

// Delayed scaling of one tensor inside forward/backward: cast with the stored
// scale and record this tensor's amax in the same pass; on the first step
// (needs_init) take the scale from the tensor's own amax first.
fp8lin_status delayed_cast(const void* x, int64_t rows, int64_t cols, int64_t ld,
                           fp8lin_scaling_state* st, uint8_t* out, uint8_t* out_t, void* ws,
                           const DeviceInfo& dev, cudaStream_t stream) {
  if (st->needs_init) {
    fp8lin_status s = do_amax(x, rows, cols, ld, st->amax, FP8LIN_AMAX_ATOMIC, ws, dev, stream);
    if (s != FP8LIN_OK) return s;
    ProfScope ps(FP8LIN_PROF_SCALE, stream);
    cudaError_t e = launch_scale(st->amax, st->scale, st->inv_scale, nullptr, nullptr, 1, false,
                                 st->fmt, st->eps, stream);
    if (e != cudaSuccess) return cuda_fail(e);
    st->needs_init = 0;
  }
  if (rows == 0 || cols == 0) {
    cudaError_t e = cudaMemsetAsync(st->amax, 0, sizeof(float), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  CastArgs c;
  c.x = static_cast<const uint16_t*>(x);
  c.rows = rows;
  c.cols = cols;
  c.ld = ld;
  c.fmt = st->fmt;
  c.scale_in = st->scale;
  c.amax_in = nullptr;
  c.derive_scale = false;
  c.eps = st->eps;
  c.scale_out = nullptr;
  c.inv_out = nullptr;
  c.out = out;
  c.out_t = out_t;
  c.amax_rec = reinterpret_cast<uint32_t*>(st->amax);
  c.rec_acc = ws_u32(ws, kWsAtomicAccOffset);
  c.rec_ticket = ws_u32(ws, kWsAtomicTicketOffset);
  c.err = ws_error(ws);
  return do_cast(c, dev, stream);
}

GemmArgs gemm_args(const uint8_t* a, const uint8_t* b, int64_t M, int64_t N, int64_t K,
                   int64_t lda, int64_t ldb, int32_t fa, int32_t fb, const float* inv_a,
                   const float* inv_b, void* d, int64_t ldd, float* d_amax, void* ws,
                   size_t ws_bytes) {
  GemmArgs g;
  g.a = a;
  g.b = b;
  g.M = M;
  g.N = N;
  g.K = K;
  g.lda = lda;
  g.ldb = ldb;
  g.fmt_a = fa;
  g.fmt_b = fb;
  g.inv_a = inv_a;
  g.inv_b = inv_b;
  g.d = d;
  g.ldd = ldd;
  g.d_amax = reinterpret_cast<uint32_t*>(d_amax);
  g.ws_amax_acc = ws_u32(ws, kWsGemmAmaxAccOffset);
  g.ws_amax_ticket = ws_u32(ws, kWsGemmAmaxTicketOffset);
  g.ws_error = ws_error(ws);
  if (ws_bytes > kWsSplitOffset) {
    g.ws_tickets = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsTicketOffset);
    g.ws_split = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsSplitOffset);
    g.ws_split_bytes = ws_bytes - kWsSplitOffset;
  } else {
    g.ws_tickets = nullptr;
    g.ws_split = nullptr;
    g.ws_split_bytes = 0;
  }
  return g;
}

fp8lin_status do_gemm(const uint8_t* a, const uint8_t* b, int64_t M, int64_t N, int64_t K,
                      int64_t lda, int64_t ldb, int32_t fa, int32_t fb, const float* inv_a,
                      const float* inv_b, void* d, int64_t ldd, float* d_amax, void* ws,
                      size_t ws_bytes, const DeviceInfo& dev, cudaStream_t stream) {
  if (M == 0 || N == 0 || K == 0) {
    // Nothing to multiply: D (if any) is zeros, and so is its amax.
    cudaError_t e = cudaSuccess;
    if (M > 0 && N > 0)
      e = cudaMemset2DAsync(d, static_cast<size_t>(ldd) * 2, 0, static_cast<size_t>(N) * 2,
                            static_cast<size_t>(M), stream);
    if (e == cudaSuccess && d_amax != nullptr)
      e = cudaMemsetAsync(d_amax, 0, sizeof(float), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  const GemmArgs g = gemm_args(a, b, M, N, K, lda, ldb, fa, fb, inv_a, inv_b, d, ldd, d_amax, ws,
                               ws_bytes);
  ProfScope ps(FP8LIN_PROF_GEMM, stream);
  cudaError_t e = launch_gemm(g, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status get_dev(DeviceInfo* dev) {
  cudaError_t e = current_device_info(dev);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

bool ws_ok(const void* ws) {
  return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

fp8lin_status run_scale(const fp8lin_scaling_state* st, cudaStream_t stream) {
  const bool delayed = st->kind == FP8LIN_DELAYED;
  ProfScope ps(FP8LIN_PROF_SCALE, stream);
  cudaError_t e = launch_scale(st->amax, st->scale, st->inv_scale, st->amax_history, st->head,
                               delayed ? st->history_len : 1, delayed, st->fmt, st->eps, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

}  // namespace

void set_error_site(const char* site) { g_error_site = site; }

bool pdl_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("FP8LIN_PDL");
    return !(v != nullptr && v[0] == '0');
  }();
  return on;
}

cudaError_t current_device_info(DeviceInfo* info) {
  static std::mutex mu;
  static DeviceInfo cache[64];
  static bool have[64] = {};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  // Bind the device's primary context to this thread: a thread that never
  // called cudaSetDevice (e.g. an autograd worker) may have none current, and
  // the driver-level tensor-map encoding needs one.
  e = cudaSetDevice(d);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[d]) {
    DeviceInfo x;
    x.device = d;
    e = cudaDeviceGetAttribute(&x.num_sms, cudaDevAttrMultiProcessorCount, d);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&x.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d);
    if (e != cudaSuccess) return e;
    cache[d] = x;
    have[d] = true;
  }
  *info = cache[d];
  return cudaSuccess;
}

namespace {

// Calls run(list, n) over the gradients that match, at most kClipMaxTensors at a time.
template <typename Match, typename Run>
fp8lin_status for_lists(const fp8lin_grad* grads, int32_t count, Match match, Run run) {
  GradTensor list[kClipMaxTensors];
  int n = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (grads[i].n == 0 || !match(grads[i])) continue;
    if (n == kClipMaxTensors) {
      fp8lin_status s = run(list, n);
      if (s != FP8LIN_OK) return s;
      n = 0;
    }
    list[n].g = grads[i].g;
    list[n].out = grads[i].out;
    list[n].n = grads[i].n;
    ++n;
  }
  return n > 0 ? run(list, n) : FP8LIN_OK;
}

}  // namespace
}  // namespace fp8lin

using namespace fp8lin;

extern "C" {

const char* fp8lin_status_string(int status) {
  switch (status) {
    case FP8LIN_OK: return "FP8LIN_OK";
    case FP8LIN_EINVAL: return "FP8LIN_EINVAL: invalid argument";
    case FP8LIN_EUNSUPPORTED: return "FP8LIN_EUNSUPPORTED: shape, format or size not supported";
    case FP8LIN_ECUDA: return "FP8LIN_ECUDA: a CUDA call failed";
    case FP8LIN_ETIMEOUT: return "FP8LIN_ETIMEOUT: a bounded device wait ran out";
    default: return "unknown fp8lin status";
  }
}

int fp8lin_last_cuda_error(void) { return g_last_cuda_error; }

const char* fp8lin_last_error_detail(void) {
  return g_last_cuda_error == 0 ? "" : g_error_detail;
}

int fp8lin_version(void) { return 101; }

size_t fp8lin_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  (void)M;
  (void)K;
  (void)N;
  // Fixed part (error word, grid barrier, amax partials), the K-split tickets
  // and room for the K-split partials of the GEMMs' tail wave.
  int num_sms = 152;
  DeviceInfo dev;
  if (current_device_info(&dev) == cudaSuccess) num_sms = dev.num_sms;
  else cudaGetLastError();
  return kWsSplitOffset + gemm_split_workspace_bytes(num_sms);
}

int64_t fp8lin_single_pass_max_elems(void) {
  DeviceInfo dev;
  if (current_device_info(&dev) != cudaSuccess) return 0;
  return single_pass_capacity_elems(dev);
}

fp8lin_status fp8lin_check(void* ws, cudaStream_t stream) {
  if (!ws_ok(ws)) return FP8LIN_EINVAL;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e);
  int code = 0;
  e = cudaMemcpy(&code, ws_error(ws), sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e);
  if (code == 0) return FP8LIN_OK;
  // A wait that ran out can leave counters of the workspace mid-count: clear
  // the error word and the GEMM split tickets so the workspace is usable again.
  e = cudaMemset(ws_error(ws), 0, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaMemset(static_cast<uint8_t*>(ws) + kWsTicketOffset, 0, sizeof(int) * kWsTickets);
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaMemset(static_cast<uint8_t*>(ws) + kWsScratchBegin, 0,
                 kWsPartialOffset - kWsScratchBegin);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8LIN_ETIMEOUT;
}

fp8lin_status fp8lin_amax(const void* x, int64_t rows, int64_t cols, int64_t ld,
                          float* amax_out, int32_t algo, void* ws, cudaStream_t stream) {
  fp8lin_status s = check_bf16(x, rows, cols, ld);
  if (s != FP8LIN_OK) return s;
  if (amax_out == nullptr || (reinterpret_cast<uintptr_t>(amax_out) & 3u)) return FP8LIN_EINVAL;
  if (algo != FP8LIN_AMAX_ATOMIC && algo != FP8LIN_AMAX_REDUCTION) return FP8LIN_EUNSUPPORTED;
  if (algo == FP8LIN_AMAX_REDUCTION && !ws_ok(ws)) return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return do_amax(x, rows, cols, ld, amax_out, algo, ws, dev, stream);
}

fp8lin_status fp8lin_amax_noalloc(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                  float* amax_out, cudaStream_t stream) {
  fp8lin_status s = check_bf16(x, rows, cols, ld);
  if (s != FP8LIN_OK) return s;
  if (amax_out == nullptr || (reinterpret_cast<uintptr_t>(amax_out) & 3u)) return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  if (rows == 0 || cols == 0) {
    cudaError_t e = cudaMemsetAsync(amax_out, 0, sizeof(float), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  const int grid = amax_grid(dev, rows, cols);
  if (grid > kStaticAmaxPartials) return FP8LIN_EUNSUPPORTED;  // more CTAs than scratch slots
  g_launches.fetch_add(2, std::memory_order_relaxed);
  cudaError_t e = launch_amax_static_scratch(static_cast<const uint16_t*>(x), rows, cols, ld,
                                             amax_out, grid, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_scale(const fp8lin_scaling_state* st, cudaStream_t stream) {
  fp8lin_status s = check_state(st, true);
  if (s != FP8LIN_OK) return s;
  return run_scale(st, stream);
}

// The device byte ranges the scale update of one state writes (scale, inverse
// and, delayed, the ring and its head); it reads only these and *amax.
struct ByteRange {
  uintptr_t lo, hi;
};

int scale_written_ranges(const fp8lin_scaling_state* st, ByteRange* r) {
  auto at = [](const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return ByteRange{lo, lo + bytes};
  };
  int n = 0;
  r[n++] = at(st->scale, sizeof(float));
  r[n++] = at(st->inv_scale, sizeof(float));
  if (st->kind == FP8LIN_DELAYED) {
    r[n++] = at(st->amax_history, sizeof(float) * static_cast<size_t>(st->history_len));
    r[n++] = at(st->head, sizeof(int32_t));
  }
  return n;
}

bool ranges_overlap(const ByteRange& a, const ByteRange& b) { return a.lo < b.hi && b.lo < a.hi; }

// True if a buffer that one of the n states' updates writes overlaps any
// buffer of another state (one thread per state would race on it).  States
// may share an amax, which the update only reads.
bool scale_states_overlap(const fp8lin_scaling_state* states, int n) {
  for (int i = 0; i < n; ++i) {
    ByteRange wi[4];
    const int ni = scale_written_ranges(&states[i], wi);
    for (int j = 0; j < n; ++j) {
      if (j == i) continue;
      ByteRange bj[5];
      int nj = scale_written_ranges(&states[j], bj);
      const uintptr_t amax = reinterpret_cast<uintptr_t>(states[j].amax);
      bj[nj++] = {amax, amax + sizeof(float)};
      for (int x = 0; x < ni; ++x)
        for (int y = 0; y < nj; ++y)
          if (ranges_overlap(wi[x], bj[y])) return true;
    }
  }
  return false;
}

fp8lin_status fp8lin_scale_many(const fp8lin_scaling_state* states, int32_t n,
                                cudaStream_t stream) {
  if (n < 0 || n > 8 || (n > 0 && states == nullptr)) return FP8LIN_EINVAL;
  ScaleArgs a[8];
  for (int i = 0; i < n; ++i) {
    const fp8lin_scaling_state* st = &states[i];
    fp8lin_status s = check_state(st, true);
    if (s != FP8LIN_OK) return s;
    const bool delayed = st->kind == FP8LIN_DELAYED;
    a[i] = {st->amax, st->scale, st->inv_scale, st->amax_history, st->head,
            delayed ? st->history_len : 1, delayed, st->fmt, st->eps};
  }
  if (n == 0) return FP8LIN_OK;
  if (scale_states_overlap(states, n)) return FP8LIN_EINVAL;
  ProfScope ps(FP8LIN_PROF_SCALE, stream);
  cudaError_t e = launch_scale_batch(a, n, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_cast(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t fmt,
                          const float* scale, uint8_t* out, uint8_t* out_t, float* amax_out,
                          cudaStream_t stream) {
  fp8lin_status s = check_bf16(x, rows, cols, ld);
  if (s != FP8LIN_OK) return s;
  if (!valid_fmt(fmt)) return FP8LIN_EUNSUPPORTED;
  if (scale == nullptr) return FP8LIN_EINVAL;
  if (out == nullptr && out_t == nullptr) return FP8LIN_EINVAL;
  if (out != nullptr && !aligned16(out)) return FP8LIN_EINVAL;
  if (out_t != nullptr) {
    if (!aligned16(out_t)) return FP8LIN_EINVAL;
    if (rows % 16 != 0) return FP8LIN_EUNSUPPORTED;
  }
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  if (amax_out != nullptr) {
    cudaError_t e = cudaMemsetAsync(amax_out, 0, sizeof(float), stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  CastArgs c;
  c.x = static_cast<const uint16_t*>(x);
  c.rows = rows;
  c.cols = cols;
  c.ld = ld;
  c.fmt = fmt;
  c.scale_in = scale;
  c.amax_in = nullptr;
  c.derive_scale = false;
  c.eps = 1e-12f;
  c.scale_out = nullptr;
  c.inv_out = nullptr;
  c.out = out;
  c.out_t = out_t;
  c.amax_rec = reinterpret_cast<uint32_t*>(amax_out);
  return do_cast(c, dev, stream);
}

fp8lin_status fp8lin_cast_dynamic(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                  const fp8lin_scaling_state* st, uint8_t* out, uint8_t* out_t,
                                  void* ws, cudaStream_t stream) {
  fp8lin_status s = check_bf16(x, rows, cols, ld);
  if (s != FP8LIN_OK) return s;
  if ((s = check_state(st, false)) != FP8LIN_OK) return s;
  if (st->kind != FP8LIN_DYNAMIC) return FP8LIN_EINVAL;
  if (!ws_ok(ws)) return FP8LIN_EINVAL;
  if (out == nullptr && out_t == nullptr) return FP8LIN_EINVAL;
  if (out != nullptr && !aligned16(out)) return FP8LIN_EINVAL;
  if (out_t != nullptr) {
    if (!aligned16(out_t)) return FP8LIN_EINVAL;
    if (rows % 16 != 0) return FP8LIN_EUNSUPPORTED;
  }
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return cast_dynamic_scaled(x, rows, cols, ld, st, out, out_t, ws, dev, stream, false);
}

fp8lin_status fp8lin_cast_delayed(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                  fp8lin_scaling_state* st, uint8_t* out, uint8_t* out_t,
                                  void* ws, cudaStream_t stream) {
  fp8lin_status s = check_bf16(x, rows, cols, ld);
  if (s != FP8LIN_OK) return s;
  if ((s = check_state(st, false)) != FP8LIN_OK) return s;
  if (st->kind != FP8LIN_DELAYED) return FP8LIN_EINVAL;
  if (!ws_ok(ws)) return FP8LIN_EINVAL;
  if (out == nullptr && out_t == nullptr) return FP8LIN_EINVAL;
  if (out != nullptr && !aligned16(out)) return FP8LIN_EINVAL;
  if (out_t != nullptr) {
    if (!aligned16(out_t)) return FP8LIN_EINVAL;
    if (rows % 16 != 0) return FP8LIN_EUNSUPPORTED;
  }
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return delayed_cast(x, rows, cols, ld, st, out, out_t, ws, dev, stream);
}

fp8lin_status fp8lin_gemm(const uint8_t* a, const uint8_t* b, int64_t M, int64_t N, int64_t K,
                          int64_t lda, int64_t ldb, int32_t fmt_a, int32_t fmt_b,
                          const float* inv_a, const float* inv_b, void* d, int64_t ldd,
                          float* d_amax, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return FP8LIN_EINVAL;
  if (!valid_fmt(fmt_a) || !valid_fmt(fmt_b)) return FP8LIN_EUNSUPPORTED;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  if (d_amax != nullptr && (reinterpret_cast<uintptr_t>(d_amax) & 3u) != 0) return FP8LIN_EINVAL;
  if (M == 0 || N == 0) {
    if (d_amax == nullptr) return FP8LIN_OK;
    DeviceInfo dev;
    fp8lin_status s = get_dev(&dev);
    if (s != FP8LIN_OK) return s;
    return do_gemm(a, b, M, N, K, lda, ldb, fmt_a, fmt_b, inv_a, inv_b, d, ldd, d_amax, ws,
                   ws_bytes, dev, stream);
  }
  if (d == nullptr || !aligned16(d) || ldd < N) return FP8LIN_EINVAL;
  if (inv_a == nullptr || inv_b == nullptr) return FP8LIN_EINVAL;
  if (K > 0) {
    if (a == nullptr || b == nullptr || !aligned16(a) || !aligned16(b)) return FP8LIN_EINVAL;
    if (lda < K || ldb < K) return FP8LIN_EINVAL;
    if (lda % 16 != 0 || ldb % 16 != 0 || K % 16 != 0) return FP8LIN_EUNSUPPORTED;
  }
  if (N % 16 != 0 || ldd % 8 != 0) return FP8LIN_EUNSUPPORTED;
  if (M > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256 || K > (int64_t(1) << 31) - 256)
    return FP8LIN_EUNSUPPORTED;
  DeviceInfo dev;
  fp8lin_status s = get_dev(&dev);
  if (s != FP8LIN_OK) return s;
  return do_gemm(a, b, M, N, K, lda, ldb, fmt_a, fmt_b, inv_a, inv_b, d, ldd, d_amax, ws, ws_bytes,
                 dev, stream);
}

fp8lin_status fp8lin_gemm_describe(int64_t M, int64_t N, int64_t K, char* buf, size_t buf_len) {
  if (M < 0 || N < 0 || K < 0 || buf == nullptr || buf_len == 0) return FP8LIN_EINVAL;
  buf[0] = '\0';
  DeviceInfo dev;
  fp8lin_status s = get_dev(&dev);
  if (s != FP8LIN_OK) return s;
  cudaError_t e = describe_gemm(M, N, K, dev, buf, buf_len);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_gemm_describe_for(int64_t M, int64_t N, int64_t K, int32_t num_sms,
                                       char* buf, size_t buf_len) {
  if (M < 0 || N < 0 || K < 0 || num_sms < 2 || buf == nullptr || buf_len == 0)
    return FP8LIN_EINVAL;
  describe_plan(M, N, K, num_sms, num_sms / 2, buf, buf_len);
  return FP8LIN_OK;
}

fp8lin_status fp8lin_gemm_group_describe_for(int64_t Ma, int64_t Na, int64_t Ka, int64_t Mb,
                                             int64_t Nb, int64_t Kb, int32_t num_sms, char* buf,
                                             size_t buf_len) {
  if (Ma < 1 || Na < 1 || Ka < 1 || Mb < 1 || Nb < 1 || Kb < 1 || num_sms < 2 || buf == nullptr ||
      buf_len == 0)
    return FP8LIN_EINVAL;
  describe_group_plan(Ma, Na, Ka, Mb, Nb, Kb, num_sms, num_sms / 2, buf, buf_len);
  return FP8LIN_OK;
}

static fp8lin_status check_linear_sizes(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K < 0 || N < 0) return FP8LIN_EINVAL;
  if (M % 16 != 0 || K % 16 != 0 || N % 16 != 0) return FP8LIN_EUNSUPPORTED;
  if (M > (int64_t(1) << 31) - 256 || K > (int64_t(1) << 31) - 256 ||
      N > (int64_t(1) << 31) - 256)
    return FP8LIN_EUNSUPPORTED;
  return FP8LIN_OK;
}

static bool dev_ptrs_ok(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr || !aligned16(p)) return false;
  return true;
}

}  // extern "C"

namespace {

fp8lin_status check_forward(const void* x, const void* w, int64_t M, int64_t K, int64_t N,
                            const fp8lin_scaling_state* sx, const fp8lin_scaling_state* sw,
                            const void* y, const float* y_amax, const uint8_t* x8,
                            const uint8_t* x8t, const uint8_t* w8, const uint8_t* w8t,
                            const void* ws, size_t ws_bytes) {
  fp8lin_status s = check_linear_sizes(M, K, N);
  if (s != FP8LIN_OK) return s;
  if ((s = check_state(sx, true)) != FP8LIN_OK) return s;
  if ((s = check_state(sw, true)) != FP8LIN_OK) return s;
  if (sx->fmt != FP8LIN_E4M3 || sw->fmt != FP8LIN_E4M3) return FP8LIN_EUNSUPPORTED;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  if (M * K > 0 && !dev_ptrs_ok({x, x8, x8t})) return FP8LIN_EINVAL;
  if (N * K > 0 && !dev_ptrs_ok({w8, w8t})) return FP8LIN_EINVAL;
  if (w != nullptr && N * K > 0 && !dev_ptrs_ok({w})) return FP8LIN_EINVAL;
  // w == NULL reuses w8 / w8t / sw from an earlier call: there must have been one.
  if (w == nullptr && sw->kind == FP8LIN_DELAYED && sw->needs_init) return FP8LIN_EINVAL;
  if (M * N > 0 && !dev_ptrs_ok({y})) return FP8LIN_EINVAL;
  if (y_amax != nullptr && (reinterpret_cast<uintptr_t>(y_amax) & 3u) != 0) return FP8LIN_EINVAL;
  return FP8LIN_OK;
}

// Few-token products run as one fused launch each (small_m.cu) when the
// token side has dynamic scaling; FP8LIN_SMALL_M=0 turns this off.
bool small_m_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("FP8LIN_SMALL_M");
    return !(v != nullptr && v[0] == '0');
  }();
  return on;
}

// The backward's few-token product also computes dW unless FP8LIN_SMALL_M_DW=0.
bool small_m_dw_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("FP8LIN_SMALL_M_DW");
    return !(v != nullptr && v[0] == '0');
  }();
  return on;
}

bool few_token_state(const fp8lin_scaling_state* st, int64_t M) {
  return small_m_enabled() && M >= 1 && M <= kSmallMaxRows && st->kind == FP8LIN_DYNAMIC &&
         (st->amax_algo == FP8LIN_AMAX_AUTO || st->amax_algo == FP8LIN_AMAX_SINGLE_PASS ||
          st->amax_algo == FP8LIN_AMAX_PRECOMPUTED);
}

size_t split_bytes(size_t ws_bytes) {
  return ws_bytes > kWsSplitOffset ? ws_bytes - kWsSplitOffset : 0;
}

// The fused few-token product D = B8 . A8^T (token side B cast in the launch).
SmallMArgs small_m_args(const fp8lin_scaling_state* sb, const void* b, int64_t M, uint8_t* b8,
                        uint8_t* b8t, void* d, int64_t ldd, float* d_amax, void* ws,
                        size_t ws_bytes) {
  SmallMArgs a = {};
  a.MB = M;
  a.b = static_cast<const uint16_t*>(b);
  a.eps = sb->eps;
  a.fmt_b = sb->fmt;
  a.b_amax_in = sb->amax_algo == FP8LIN_AMAX_PRECOMPUTED ? sb->amax : nullptr;
  a.b_amax = sb->amax;
  a.b_scale = sb->scale;
  a.b_inv = sb->inv_scale;
  a.b8 = b8;
  a.b8t = b8t;
  a.d = d;
  a.ldd = ldd;
  a.d_amax = reinterpret_cast<uint32_t*>(d_amax);
  a.ws_amax_acc = ws_u32(ws, kWsGemmAmaxAccOffset);
  a.ws_amax_ticket = ws_u32(ws, kWsGemmAmaxTicketOffset);
  a.ws_partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsSplitOffset);
  a.ws_partial_bytes = split_bytes(ws_bytes);
  a.ws_tickets = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsTicketOffset);
  a.ws_barrier = ws_u32(ws, kWsBarrierOffset);
  a.ws_exits = ws_u32(ws, kWsExitsOffset);
  a.ws_amax = ws_u32(ws, kWsAmaxOffset);
  a.ws_b_amax = ws_u32(ws, kWsSmallBAmaxOffset);
  a.ws_error = ws_error(ws);
  return a;
}

fp8lin_status run_small_m(const SmallMArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  ProfScope ps(FP8LIN_PROF_SMALL_M, stream);
  cudaError_t e = launch_small_m(a, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status run_forward(const void* x, const void* w, int64_t M, int64_t K, int64_t N,
                          fp8lin_scaling_state* sx, fp8lin_scaling_state* sw, void* y,
                          float* y_amax, uint8_t* x8, uint8_t* x8t, uint8_t* w8, uint8_t* w8t,
                          void* ws, size_t ws_bytes, const DeviceInfo& dev, cudaStream_t stream) {
  // A few tokens: x's cast, W's cast (unless W8 is reused) and y in one launch.
  if (K > 0 && N > 0 && few_token_state(sx, M)) {
    const bool cast_w = w != nullptr;
    const bool w_ok = !cast_w || (sw->kind == FP8LIN_DYNAMIC &&
                                  (sw->amax_algo == FP8LIN_AMAX_AUTO ||
                                   sw->amax_algo == FP8LIN_AMAX_SINGLE_PASS));
    if (w_ok && small_m_fits(dev, cast_w, 0, M, N, K, split_bytes(ws_bytes))) {
      SmallMArgs a = small_m_args(sx, x, M, x8, x8t, y, N, y_amax, ws, ws_bytes);
      a.cast_a = cast_w;
      a.NA = N;
      a.KA = K;
      a.ldb = K;
      if (cast_w) {
        a.a = w;
        a.a8 = w8;
        a.a8t = w8t;
        a.a_amax = sw->amax;
        a.a_scale = sw->scale;
        a.a_inv = sw->inv_scale;
      } else {
        a.a = w8;
        a.a_inv_in = sw->inv_scale;
      }
      return run_small_m(a, dev, stream);
    }
  }
  // W's single pass with x's cast in the same launch, where x has at most one
  // tile for each of its CTAs (a few hundred tokens): one launch and one grid
  // barrier fewer.
  if (w != nullptr && pair_cast_enabled() && sx->kind == FP8LIN_DYNAMIC &&
      sw->kind == FP8LIN_DYNAMIC && single_pass_algo(sx->amax_algo) &&
      single_pass_algo(sw->amax_algo) && x8t != nullptr && w8t != nullptr &&
      single_pass_pair_fits(dev, N, K, M, K)) {
    SinglePassArgs wa = single_pass_args(w, N, K, K, sw, w8, w8t, ws);
    SinglePassArgs xa = single_pass_args(x, M, K, K, sx, x8, x8t, ws);
    xa.ws_amax = ws_u32(ws, kWsAmax2Offset);
    {
      ProfScope ps(FP8LIN_PROF_CAST_FUSED, stream);
      cudaError_t e = launch_cast_single_pass_pair(wa, xa, dev, stream);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    return do_gemm(x8, w8, M, N, K, K, K, FP8LIN_E4M3, FP8LIN_E4M3, sx->inv_scale, sw->inv_scale,
                   y, N, y_amax, ws, ws_bytes, dev, stream);
  }
  fp8lin_status s;
  if (sx->kind == FP8LIN_DYNAMIC)
    s = cast_dynamic_scaled(x, M, K, K, sx, x8, x8t, ws, dev, stream, true);
  else
    s = delayed_cast(x, M, K, K, sx, x8, x8t, ws, dev, stream);
  if (s != FP8LIN_OK) return s;
  if (w != nullptr) {
    if (sw->kind == FP8LIN_DYNAMIC)
      s = cast_dynamic_scaled(w, N, K, K, sw, w8, w8t, ws, dev, stream, true);
    else
      s = delayed_cast(w, N, K, K, sw, w8, w8t, ws, dev, stream);
    if (s != FP8LIN_OK) return s;
  }
  // y = x8 . W8^T : A = x8 [M, K], B = W8 [N, K]
  return do_gemm(x8, w8, M, N, K, K, K, FP8LIN_E4M3, FP8LIN_E4M3, sx->inv_scale, sw->inv_scale, y,
                 N, y_amax, ws, ws_bytes, dev, stream);
}

fp8lin_status check_backward(const void* dy, int64_t M, int64_t K, int64_t N, const uint8_t* x8t,
                             const uint8_t* w8t, const fp8lin_scaling_state* sx,
                             const fp8lin_scaling_state* sw, const fp8lin_scaling_state* sdy,
                             const uint8_t* dy8, const uint8_t* dy8t, const void* dx,
                             const void* dw, const float* dx_amax, const float* dw_amax,
                             const void* ws, size_t ws_bytes) {
  fp8lin_status s = check_linear_sizes(M, K, N);
  if (s != FP8LIN_OK) return s;
  if ((s = check_state(sx, false)) != FP8LIN_OK) return s;
  if ((s = check_state(sw, false)) != FP8LIN_OK) return s;
  if ((s = check_state(sdy, true)) != FP8LIN_OK) return s;
  if (sdy->fmt != FP8LIN_E5M2) return FP8LIN_EUNSUPPORTED;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  if (M * N > 0 && !dev_ptrs_ok({dy, dy8, dy8t})) return FP8LIN_EINVAL;
  if (dx != nullptr && M * K > 0 && !dev_ptrs_ok({dx})) return FP8LIN_EINVAL;
  if (dx != nullptr && N * K > 0 && !dev_ptrs_ok({w8t})) return FP8LIN_EINVAL;
  if (dw != nullptr && N * K > 0 && !dev_ptrs_ok({dw})) return FP8LIN_EINVAL;
  if (dw != nullptr && M * K > 0 && !dev_ptrs_ok({x8t})) return FP8LIN_EINVAL;
  if ((dx_amax != nullptr && (dx == nullptr || (reinterpret_cast<uintptr_t>(dx_amax) & 3u))) ||
      (dw_amax != nullptr && (dw == nullptr || (reinterpret_cast<uintptr_t>(dw_amax) & 3u))))
    return FP8LIN_EINVAL;
  return FP8LIN_OK;
}

fp8lin_status run_backward(const void* dy, int64_t M, int64_t K, int64_t N, const uint8_t* x8t,
                           const uint8_t* w8t, const fp8lin_scaling_state* sx,
                           const fp8lin_scaling_state* sw, fp8lin_scaling_state* sdy,
                           uint8_t* dy8, uint8_t* dy8t, void* dx, void* dw, float* dx_amax,
                           float* dw_amax, void* ws, size_t ws_bytes, const DeviceInfo& dev,
                           cudaStream_t stream) {
  fp8lin_status s;
  bool dx_done = false, dw_done = false;
  if (dx != nullptr && K > 0 && N > 0 && few_token_state(sdy, M) &&
      small_m_fits(dev, false, FP8LIN_E5M2, M, K, N, split_bytes(ws_bytes))) {
    // A few tokens: dY's cast and dX = dY8 . W8 (A = W8^T [K, N]) in one launch,
    // and dW = dY8^T . x8 in the same launch when its amax is not wanted.
    SmallMArgs a = small_m_args(sdy, dy, M, dy8, dy8t, dx, K, dx_amax, ws, ws_bytes);
    a.cast_a = false;
    a.NA = K;
    a.KA = N;
    a.ldb = N;
    a.a = w8t;
    a.a_inv_in = sw->inv_scale;
    if (dw != nullptr && dw_amax == nullptr && small_m_dw_enabled() &&
        small_m_fits(dev, false, FP8LIN_E5M2, M, K, N, split_bytes(ws_bytes), true)) {
      a.fuse_dw = true;
      a.x8t = x8t;
      a.x_inv = sx->inv_scale;
      a.dw = dw;
      dw_done = true;
    }
    if ((s = run_small_m(a, dev, stream)) != FP8LIN_OK) return s;
    dx_done = true;
  } else if (sdy->kind == FP8LIN_DYNAMIC) {
    s = cast_dynamic_scaled(dy, M, N, N, sdy, dy8, dy8t, ws, dev, stream, true);
  } else {
    s = delayed_cast(dy, M, N, N, sdy, dy8, dy8t, ws, dev, stream);
  }
  if (!dx_done && s != FP8LIN_OK) return s;
  if (dx != nullptr && !dx_done && dw != nullptr && !dw_done && M > 0 && N > 0 && K > 0) {
    // dX and dW in one launch when the grouped plan expects it to be faster
    const GemmArgs gx = gemm_args(dy8, w8t, M, K, N, N, N, FP8LIN_E5M2, FP8LIN_E4M3,
                                  sdy->inv_scale, sw->inv_scale, dx, K, dx_amax, ws, ws_bytes);
    const GemmArgs gw = gemm_args(dy8t, x8t, N, K, M, M, M, FP8LIN_E5M2, FP8LIN_E4M3,
                                  sdy->inv_scale, sx->inv_scale, dw, K, dw_amax, ws, ws_bytes);
    bool grouped = false;
    cudaError_t e = plan_gemm_pair2(gx, gw, dev, &grouped);
    if (e != cudaSuccess) return cuda_fail(e);
    if (grouped) {
      ProfScope ps(FP8LIN_PROF_GEMM, stream);
      e = launch_gemm_pair2(gx, gw, dev, stream);
      if (e != cudaSuccess) return cuda_fail(e);
      dx_done = dw_done = true;
    }
  }
  if (dx != nullptr && !dx_done) {
    // dX = dY8 . W8 : A = dY8 [M, N], B = W8^T [K, N], contract over N
    s = do_gemm(dy8, w8t, M, K, N, N, N, FP8LIN_E5M2, FP8LIN_E4M3, sdy->inv_scale, sw->inv_scale,
                dx, K, dx_amax, ws, ws_bytes, dev, stream);
    if (s != FP8LIN_OK) return s;
  }
  if (dw != nullptr && !dw_done) {
    // dW = dY8^T . x8 : A = dY8^T [N, M], B = x8^T [K, M], contract over M
    s = do_gemm(dy8t, x8t, N, K, M, M, M, FP8LIN_E5M2, FP8LIN_E4M3, sdy->inv_scale, sx->inv_scale,
                dw, K, dw_amax, ws, ws_bytes, dev, stream);
    if (s != FP8LIN_OK) return s;
  }
  return FP8LIN_OK;
}

}  // namespace

extern "C" {

fp8lin_status fp8lin_forward(const void* x, const void* w, int64_t M, int64_t K, int64_t N,
                             fp8lin_scaling_state* sx, fp8lin_scaling_state* sw, void* y,
                             float* y_amax, uint8_t* x8, uint8_t* x8t, uint8_t* w8, uint8_t* w8t,
                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  fp8lin_status s =
      check_forward(x, w, M, K, N, sx, sw, y, y_amax, x8, x8t, w8, w8t, ws, ws_bytes);
  if (s != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return run_forward(x, w, M, K, N, sx, sw, y, y_amax, x8, x8t, w8, w8t, ws, ws_bytes, dev,
                     stream);
}

fp8lin_status fp8lin_backward(const void* dy, int64_t M, int64_t K, int64_t N,
                              const uint8_t* x8t, const uint8_t* w8t,
                              const fp8lin_scaling_state* sx, const fp8lin_scaling_state* sw,
                              fp8lin_scaling_state* sdy, uint8_t* dy8, uint8_t* dy8t, void* dx,
                              void* dw, float* dx_amax, float* dw_amax, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
  fp8lin_status s = check_backward(dy, M, K, N, x8t, w8t, sx, sw, sdy, dy8, dy8t, dx, dw, dx_amax,
                                   dw_amax, ws, ws_bytes);
  if (s != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return run_backward(dy, M, K, N, x8t, w8t, sx, sw, sdy, dy8, dy8t, dx, dw, dx_amax, dw_amax, ws,
                      ws_bytes, dev, stream);
}

fp8lin_status fp8lin_step_host(const void* x_h, const void* w_h, const void* dy_h, void* y_h,
                               void* dx_h, void* dw_h, int64_t M, int64_t K, int64_t N,
                               fp8lin_scaling_state* sx, fp8lin_scaling_state* sw,
                               fp8lin_scaling_state* sdy, const fp8lin_step_slot* slot,
                               cudaStream_t compute, cudaStream_t h2d, cudaStream_t d2h,
                               int wait) {
  if (slot == nullptr) return FP8LIN_EINVAL;
  const fp8lin_step_slot& d = *slot;
  fp8lin_status s = check_forward(d.x, d.w, M, K, N, sx, sw, d.y, nullptr, d.x8, d.x8t, d.w8,
                                  d.w8t, d.ws, d.ws_bytes);
  if (s != FP8LIN_OK) return s;
  if ((s = check_backward(d.dy, M, K, N, d.x8t, d.w8t, sx, sw, sdy, d.dy8, d.dy8t, d.dx, d.dw,
                          nullptr, nullptr, d.ws, d.ws_bytes)) != FP8LIN_OK)
    return s;
  if (M * K > 0 && (x_h == nullptr || dx_h == nullptr || d.dx == nullptr)) return FP8LIN_EINVAL;
  if (N * K > 0 && (w_h == nullptr || dw_h == nullptr || d.w == nullptr || d.dw == nullptr))
    return FP8LIN_EINVAL;
  if (M * N > 0 && (dy_h == nullptr || y_h == nullptr)) return FP8LIN_EINVAL;
  for (cudaEvent_t e : d.ev)
    if (e == nullptr) return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;

  enum { kXwIn = 0, kDyIn = 1, kFwdDone = 2, kBwdDone = 3, kOutDone = 4 };
  const size_t bx = static_cast<size_t>(M) * K * 2, bw = static_cast<size_t>(N) * K * 2,
               by = static_cast<size_t>(M) * N * 2;
  cudaError_t e;
  // Uploads: x and W once this slot's previous forward has read them; dY once
  // its previous backward has.
  if ((e = cudaStreamWaitEvent(h2d, d.ev[kFwdDone], 0)) != cudaSuccess) return cuda_fail(e);
  if (bx > 0 && (e = cudaMemcpyAsync(d.x, x_h, bx, cudaMemcpyHostToDevice, h2d)) != cudaSuccess)
    return cuda_fail(e);
  if (bw > 0 && (e = cudaMemcpyAsync(d.w, w_h, bw, cudaMemcpyHostToDevice, h2d)) != cudaSuccess)
    return cuda_fail(e);
  if ((e = cudaEventRecord(d.ev[kXwIn], h2d)) != cudaSuccess) return cuda_fail(e);
  if ((e = cudaStreamWaitEvent(h2d, d.ev[kBwdDone], 0)) != cudaSuccess) return cuda_fail(e);
  if (by > 0 && (e = cudaMemcpyAsync(d.dy, dy_h, by, cudaMemcpyHostToDevice, h2d)) != cudaSuccess)
    return cuda_fail(e);
  if ((e = cudaEventRecord(d.ev[kDyIn], h2d)) != cudaSuccess) return cuda_fail(e);
  // Forward once x and W are in and this slot's outputs have gone out.
  if ((e = cudaStreamWaitEvent(compute, d.ev[kXwIn], 0)) != cudaSuccess) return cuda_fail(e);
  if ((e = cudaStreamWaitEvent(compute, d.ev[kOutDone], 0)) != cudaSuccess) return cuda_fail(e);
  s = run_forward(d.x, d.w, M, K, N, sx, sw, d.y, nullptr, d.x8, d.x8t, d.w8, d.w8t, d.ws,
                  d.ws_bytes, dev, compute);
  if (s != FP8LIN_OK) return s;
  if ((e = cudaEventRecord(d.ev[kFwdDone], compute)) != cudaSuccess) return cuda_fail(e);
  if ((e = cudaStreamWaitEvent(d2h, d.ev[kFwdDone], 0)) != cudaSuccess) return cuda_fail(e);
  if (by > 0 && (e = cudaMemcpyAsync(y_h, d.y, by, cudaMemcpyDeviceToHost, d2h)) != cudaSuccess)
    return cuda_fail(e);
  // Backward once dY is in, then the delayed states' history sync.
  if ((e = cudaStreamWaitEvent(compute, d.ev[kDyIn], 0)) != cudaSuccess) return cuda_fail(e);
  s = run_backward(d.dy, M, K, N, d.x8t, d.w8t, sx, sw, sdy, d.dy8, d.dy8t, d.dx, d.dw, nullptr,
                   nullptr, d.ws, d.ws_bytes, dev, compute);
  if (s != FP8LIN_OK) return s;
  for (const fp8lin_scaling_state* st : {static_cast<const fp8lin_scaling_state*>(sx),
                                         static_cast<const fp8lin_scaling_state*>(sw),
                                         static_cast<const fp8lin_scaling_state*>(sdy)}) {
    if (st->kind != FP8LIN_DELAYED) continue;
    if ((s = run_scale(st, compute)) != FP8LIN_OK) return s;
  }
  if ((e = cudaEventRecord(d.ev[kBwdDone], compute)) != cudaSuccess) return cuda_fail(e);
  if ((e = cudaStreamWaitEvent(d2h, d.ev[kBwdDone], 0)) != cudaSuccess) return cuda_fail(e);
  if (bx > 0 && (e = cudaMemcpyAsync(dx_h, d.dx, bx, cudaMemcpyDeviceToHost, d2h)) != cudaSuccess)
    return cuda_fail(e);
  if (bw > 0 && (e = cudaMemcpyAsync(dw_h, d.dw, bw, cudaMemcpyDeviceToHost, d2h)) != cudaSuccess)
    return cuda_fail(e);
  if ((e = cudaEventRecord(d.ev[kOutDone], d2h)) != cudaSuccess) return cuda_fail(e);
  if (wait && (e = cudaStreamWaitEvent(compute, d.ev[kOutDone], 0)) != cudaSuccess)
    return cuda_fail(e);
  return FP8LIN_OK;
}

// ---- 4-bit operands

namespace {

constexpr int64_t kFp4MaxDim = (int64_t(1) << 31) - 256;

bool valid_fp4(int32_t fmt) { return fmt == FP8LIN_NVFP4 || fmt == FP8LIN_MXFP4; }

// A 4-bit tensor that a call reads or writes.
fp8lin_status check_fp4(const fp8lin_fp4_tensor* t) {
  if (t == nullptr || t->rows < 0 || t->cols < 0) return FP8LIN_EINVAL;
  if (!valid_fp4(t->fmt)) return FP8LIN_EUNSUPPORTED;
  if (t->rows > kFp4MaxDim || t->cols > kFp4MaxDim) return FP8LIN_EUNSUPPORTED;
  if ((t->fmt == FP8LIN_NVFP4) != (t->inv_scale != nullptr)) return FP8LIN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(t->inv_scale) & 3u) != 0) return FP8LIN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(t->own_inv) & 3u) != 0) return FP8LIN_EINVAL;
  if (t->fmt == FP8LIN_MXFP4 && t->own_inv != nullptr) return FP8LIN_EINVAL;
  if (t->rows == 0 || t->cols == 0) return FP8LIN_OK;
  if (t->codes == nullptr || t->scales == nullptr || !aligned16(t->codes) || !aligned16(t->scales))
    return FP8LIN_EINVAL;
  if (t->ld % 16 != 0 || t->ld < (t->cols + 31) / 32 * 16) return FP8LIN_EINVAL;
  return FP8LIN_OK;
}

Fp4View fp4_view(const fp8lin_fp4_tensor* t) {
  Fp4View v;
  if (t != nullptr && t->rows > 0 && t->cols > 0) {
    v.codes = t->codes;
    v.scales = t->scales;
    v.ld = t->ld;
  }
  return v;
}

// The inverse scale that a tensor's codes were made with.
const float* inv_of(const fp8lin_fp4_tensor* t) {
  return t->own_inv != nullptr ? t->own_inv : t->inv_scale;
}

// The source and the destinations of a quantisation.
fp8lin_status check_quantise(const void* x, int64_t rows, int64_t cols, int64_t ld,
                             const fp8lin_scaling_state* st, const fp8lin_fp4_tensor* out,
                             const fp8lin_fp4_tensor* out_t, const void* ws) {
  if (rows < 0 || cols < 0 || (out == nullptr && out_t == nullptr)) return FP8LIN_EINVAL;
  const int32_t fmt = (out != nullptr ? out : out_t)->fmt;
  if (!valid_fp4(fmt)) return FP8LIN_EUNSUPPORTED;
  fp8lin_status s;
  if (fmt == FP8LIN_NVFP4) {
    if ((s = check_state(st, false)) != FP8LIN_OK) return s;
    if (st->fmt != FP8LIN_E4M3) return FP8LIN_EUNSUPPORTED;
  } else if (st != nullptr) {
    return FP8LIN_EINVAL;
  }
  if (out != nullptr) {
    if ((s = check_fp4(out)) != FP8LIN_OK) return s;
    if (out->rows != rows || out->cols != cols) return FP8LIN_EINVAL;
  }
  if (out_t != nullptr) {
    if ((s = check_fp4(out_t)) != FP8LIN_OK) return s;
    if (out_t->rows != cols || out_t->cols != rows || out_t->fmt != fmt) return FP8LIN_EINVAL;
  }
  for (const fp8lin_fp4_tensor* t : {out, out_t})
    if (t != nullptr && st != nullptr && t->inv_scale != st->inv_scale) return FP8LIN_EINVAL;
  if (!ws_ok(ws)) return FP8LIN_EINVAL;
  if (rows > 0 && cols > 0) {
    if (x == nullptr || (reinterpret_cast<uintptr_t>(x) & 1u) != 0 || ld < cols)
      return FP8LIN_EINVAL;
    // Half a launch's CTAs: two tensors may share one.
    if (((rows + 127) / 128) > kFp4MaxDim / 2 / ((cols + 127) / 128)) return FP8LIN_EUNSUPPORTED;
  }
  return FP8LIN_OK;
}

// One tensor's quantisation.
struct QuantJob {
  const void* x;
  int64_t rows, cols, ld;
  fp8lin_scaling_state* st;
  const fp8lin_fp4_tensor* out;
  const fp8lin_fp4_tensor* out_t;
};

bool empty_job(const QuantJob& j) { return j.rows == 0 || j.cols == 0; }

// An empty tensor's state: as an amax of 0 leaves it.
fp8lin_status quantise_empty(const QuantJob& j, cudaStream_t stream) {
  if (j.st == nullptr) return FP8LIN_OK;
  cudaError_t e = cudaSuccess;
  const bool delayed = j.st->kind == FP8LIN_DELAYED;
  if (delayed || j.st->amax_algo != FP8LIN_AMAX_PRECOMPUTED)
    e = cudaMemsetAsync(j.st->amax, 0, sizeof(float), stream);
  if (e == cudaSuccess && (!delayed || j.st->needs_init)) {
    ProfScope ps(FP8LIN_PROF_SCALE, stream);
    e = launch_scale(j.st->amax, j.st->scale, j.st->inv_scale, nullptr, nullptr, 1, false,
                     j.st->fmt, j.st->eps, stream);
    j.st->needs_init = 0;
  }
  for (const fp8lin_fp4_tensor* t : {j.out, j.out_t})
    if (e == cudaSuccess && t != nullptr && t->own_inv != nullptr)
      e = cudaMemcpyAsync(t->own_inv, j.st->inv_scale, sizeof(float), cudaMemcpyDeviceToDevice, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

Fp4QuantArgs quant_args(const QuantJob& j, void* ws) {
  Fp4QuantArgs q;
  q.x = static_cast<const uint16_t*>(j.x);
  q.rows = j.rows;
  q.cols = j.cols;
  q.ld = j.ld;
  q.fmt = (j.out != nullptr ? j.out : j.out_t)->fmt;
  q.out = fp4_view(j.out);
  q.out_t = fp4_view(j.out_t);
  if (j.st == nullptr) return q;
  q.eps = j.st->eps;
  if (j.out != nullptr) q.own_inv = j.out->own_inv;
  if (j.out_t != nullptr) q.own_inv_t = j.out_t->own_inv;
  if (j.st->kind == FP8LIN_DELAYED && !j.st->needs_init) {
    q.scale_in = j.st->scale;
    q.inv_in = j.st->inv_scale;
    q.amax_rec = reinterpret_cast<uint32_t*>(j.st->amax);
    q.rec_acc = ws_u32(ws, kWsAtomicAccOffset);
    q.rec_ticket = ws_u32(ws, kWsAtomicTicketOffset);
    return q;
  }
  // Dynamic scaling, and delayed scaling's first step.
  q.scale_out = j.st->scale;
  q.inv_out = j.st->inv_scale;
  if (j.st->kind == FP8LIN_DYNAMIC && j.st->amax_algo == FP8LIN_AMAX_PRECOMPUTED) {
    q.amax_in = j.st->amax;
  } else {
    q.find_amax = true;
    q.amax_out = j.st->amax;
  }
  return q;
}

// One or two tensors, in as few launches as they allow: two of one format go
// through one amax and one quantisation (x and W of 256 x 4096 x 4096: the
// small one's launches are hidden), unless both record a delayed amax through
// the workspace's one pair of words.
fp8lin_status run_quantise(const QuantJob* jobs, int n, void* ws, const DeviceInfo& dev,
                           cudaStream_t stream) {
  Fp4QuantArgs q[2];
  fp8lin_status s;
  if (n == 2) {
    bool apart = empty_job(jobs[0]) || empty_job(jobs[1]);
    if (!apart) {
      for (int i = 0; i < 2; ++i) q[i] = quant_args(jobs[i], ws);
      apart = q[0].fmt != q[1].fmt || (q[0].out_t.codes != nullptr) != (q[1].out_t.codes != nullptr) ||
              (q[0].amax_rec != nullptr && q[1].amax_rec != nullptr);
    }
    if (apart) {
      if ((s = run_quantise(jobs, 1, ws, dev, stream)) != FP8LIN_OK) return s;
      return run_quantise(jobs + 1, 1, ws, dev, stream);
    }
  } else {
    if (empty_job(jobs[0])) return quantise_empty(jobs[0], stream);
    q[0] = quant_args(jobs[0], ws);
    if (fp4_quantise_small_fits(q[0])) {
      ProfScope ps(FP8LIN_PROF_CAST_FUSED, stream);
      cudaError_t e = launch_fp4_quantise_small(q[0], stream);
      if (e != cudaSuccess) return cuda_fail(e);
      jobs[0].st->needs_init = 0;
      return FP8LIN_OK;
    }
  }
  uint32_t* partials = ws_u32(ws, kWsPartialOffset);
  int num_partials[2] = {0, 0};
  if (q[0].find_amax || (n == 2 && q[1].find_amax)) {
    // A tensor that needs no amax beside one that does is left out.
    const int first = q[0].find_amax ? 0 : 1;
    const int count = n == 2 && q[0].find_amax && q[1].find_amax ? 2 : 1;
    ProfScope ps(FP8LIN_PROF_AMAX, stream);
    cudaError_t e = launch_fp4_amax(q + first, count, partials + first * (kMaxPartials / 2),
                                    num_partials + first, dev, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  ProfScope ps(FP8LIN_PROF_CAST, stream);
  cudaError_t e = launch_fp4_quantise(q, n, partials, num_partials, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  for (int i = 0; i < n; ++i)
    if (jobs[i].st != nullptr) jobs[i].st->needs_init = 0;
  return FP8LIN_OK;
}

fp8lin_status check_fp4_gemm(const fp8lin_fp4_tensor* a, const fp8lin_fp4_tensor* b, const void* d,
                             int64_t ldd, const void* ws, size_t ws_bytes) {
  fp8lin_status s;
  if ((s = check_fp4(a)) != FP8LIN_OK) return s;
  if ((s = check_fp4(b)) != FP8LIN_OK) return s;
  if (a->cols != b->cols || a->fmt != b->fmt) return FP8LIN_EINVAL;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  if (a->rows > 0 && b->rows > 0 &&
      (d == nullptr || (reinterpret_cast<uintptr_t>(d) & 1u) != 0 || ldd < b->rows))
    return FP8LIN_EINVAL;
  return FP8LIN_OK;
}

Fp4GemmArgs fp4_gemm_args(const fp8lin_fp4_tensor* a, const fp8lin_fp4_tensor* b, void* d,
                          int64_t ldd, void* ws, size_t ws_bytes) {
  Fp4GemmArgs g;
  g.a = fp4_view(a);
  g.b = fp4_view(b);
  g.fmt = a->fmt;
  g.M = a->rows;
  g.N = b->rows;
  g.K = a->cols;
  g.inv_a = inv_of(a);
  g.inv_b = inv_of(b);
  g.d = d;
  g.ldd = ldd;
  g.ws_error = ws_error(ws);
  if (ws_bytes > kWsSplitOffset) {
    g.ws_tickets = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsTicketOffset);
    g.ws_begun = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kWsSlicesOffset);
    g.ws_split = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsSplitOffset);
    g.ws_split_bytes = ws_bytes - kWsSplitOffset;
  }
  return g;
}

fp8lin_status run_fp4_gemm(const fp8lin_fp4_tensor* a, const fp8lin_fp4_tensor* b, void* d,
                           int64_t ldd, void* ws, size_t ws_bytes, const DeviceInfo& dev,
                           cudaStream_t stream) {
  if (a->rows == 0 || b->rows == 0) return FP8LIN_OK;
  if (a->cols == 0) {
    cudaError_t e = cudaMemset2DAsync(d, static_cast<size_t>(ldd) * 2, 0,
                                      static_cast<size_t>(b->rows) * 2,
                                      static_cast<size_t>(a->rows), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  Fp4GemmArgs g = fp4_gemm_args(a, b, d, ldd, ws, ws_bytes);
  ProfScope ps(FP8LIN_PROF_GEMM, stream);
  cudaError_t e = launch_fp4_gemm(g, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

// y = x . w4^T with x quantised into x4: one launch for a few tokens, else the
// quantisation and the product.
fp8lin_status run_fp4_linear(const QuantJob& job, const fp8lin_fp4_tensor* w4, void* y, int64_t ldy,
                             void* ws, size_t ws_bytes, const DeviceInfo& dev,
                             cudaStream_t stream) {
  const bool empty = empty_job(job);
  if (!empty && w4->rows > 0) {
    const Fp4GemmArgs g = fp4_gemm_args(job.out, w4, y, ldy, ws, ws_bytes);
    if (fp4_fused_fits(g, dev)) {
      ProfScope ps(FP8LIN_PROF_SMALL_M, stream);
      cudaError_t e = launch_fp4_fused(g, quant_args(job, ws), dev, stream);
      if (e != cudaSuccess) return cuda_fail(e);
      if (job.st != nullptr) job.st->needs_init = 0;
      return FP8LIN_OK;
    }
  }
  fp8lin_status s;
  if ((s = run_quantise(&job, 1, ws, dev, stream)) != FP8LIN_OK) return s;
  return run_fp4_gemm(job.out, w4, y, ldy, ws, ws_bytes, dev, stream);
}

// Whether two 4-bit tensors are one tensor and its transpose, by their sizes.
bool fp4_transposed(const fp8lin_fp4_tensor* t, const fp8lin_fp4_tensor* tt) {
  return t->rows == tt->cols && t->cols == tt->rows && t->fmt == tt->fmt;
}

}  // namespace

size_t fp8lin_fp4_scale_bytes(int64_t rows, int64_t cols, int32_t fmt) {
  if (rows < 0 || cols < 0 || !valid_fp4(fmt)) return 0;
  return static_cast<size_t>((rows + 127) / 128) *
         static_cast<size_t>(fp4_scale_ktiles(cols, fmt)) * 512;
}

fp8lin_status fp8lin_fp4_quantise(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                  fp8lin_scaling_state* st, const fp8lin_fp4_tensor* out,
                                  const fp8lin_fp4_tensor* out_t, void* ws, cudaStream_t stream) {
  fp8lin_status s = check_quantise(x, rows, cols, ld, st, out, out_t, ws);
  if (s != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  const QuantJob job = {x, rows, cols, ld, st, out, out_t};
  return run_quantise(&job, 1, ws, dev, stream);
}

fp8lin_status fp8lin_fp4_dequantise(const fp8lin_fp4_tensor* t, void* out, int64_t ldo, int32_t f32,
                                    cudaStream_t stream) {
  fp8lin_status s = check_fp4(t);
  if (s != FP8LIN_OK) return s;
  if (t->rows == 0 || t->cols == 0) return FP8LIN_OK;
  if (out == nullptr || (reinterpret_cast<uintptr_t>(out) & (f32 ? 3u : 1u)) != 0 || ldo < t->cols)
    return FP8LIN_EINVAL;
  if (((t->rows + 31) / 32) > kFp4MaxDim / ((t->cols + 127) / 128)) return FP8LIN_EUNSUPPORTED;
  ProfScope ps(FP8LIN_PROF_CAST, stream);
  cudaError_t e = launch_fp4_dequantise(fp4_view(t), t->fmt, inv_of(t), t->rows, t->cols, out,
                                        ldo, f32 != 0, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_fp4_gemm(const fp8lin_fp4_tensor* a, const fp8lin_fp4_tensor* b, void* d,
                              int64_t ldd, void* ws, size_t ws_bytes, cudaStream_t stream) {
  fp8lin_status s = check_fp4_gemm(a, b, d, ldd, ws, ws_bytes);
  if (s != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return run_fp4_gemm(a, b, d, ldd, ws, ws_bytes, dev, stream);
}

fp8lin_status fp8lin_fp4_linear(const void* x, int64_t ldx, fp8lin_scaling_state* sx,
                                const fp8lin_fp4_tensor* x4, const fp8lin_fp4_tensor* w4, void* y,
                                int64_t ldy, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (x4 == nullptr) return FP8LIN_EINVAL;
  fp8lin_status s = check_quantise(x, x4->rows, x4->cols, ldx, sx, x4, nullptr, ws);
  if (s != FP8LIN_OK) return s;
  if ((s = check_fp4_gemm(x4, w4, y, ldy, ws, ws_bytes)) != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  const QuantJob job = {x, x4->rows, x4->cols, ldx, sx, x4, nullptr};
  return run_fp4_linear(job, w4, y, ldy, ws, ws_bytes, dev, stream);
}

fp8lin_status fp8lin_fp4_forward(const void* x, const void* w, fp8lin_scaling_state* sx,
                                 fp8lin_scaling_state* sw, const fp8lin_fp4_tensor* x4,
                                 const fp8lin_fp4_tensor* x4t, const fp8lin_fp4_tensor* w4,
                                 const fp8lin_fp4_tensor* w4t, void* y, void* ws, size_t ws_bytes,
                                 cudaStream_t stream) {
  if (x4 == nullptr || w4 == nullptr) return FP8LIN_EINVAL;
  const int64_t M = x4->rows, K = x4->cols, N = w4->rows;
  fp8lin_status s = check_quantise(x, M, K, K, sx, x4, x4t, ws);
  if (s != FP8LIN_OK) return s;
  const bool given = w != nullptr || N == 0 || K == 0;  // an empty W has no address
  if (given && (s = check_quantise(w, N, K, K, sw, w4, w4t, ws)) != FP8LIN_OK) return s;
  if (!given && sw != nullptr && sw->kind == FP8LIN_DELAYED && sw->needs_init)
    return FP8LIN_EINVAL;
  if ((s = check_fp4_gemm(x4, w4, y, N, ws, ws_bytes)) != FP8LIN_OK) return s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  const QuantJob jobs[2] = {{x, M, K, K, sx, x4, x4t}, {w, N, K, K, sw, w4, w4t}};
  if ((s = run_quantise(jobs, given ? 2 : 1, ws, dev, stream)) != FP8LIN_OK) return s;
  return run_fp4_gemm(x4, w4, y, N, ws, ws_bytes, dev, stream);
}

fp8lin_status fp8lin_fp4_backward(const void* dy, fp8lin_scaling_state* sdy,
                                  const fp8lin_fp4_tensor* dy4, const fp8lin_fp4_tensor* dy4t,
                                  const fp8lin_fp4_tensor* w4t, const fp8lin_fp4_tensor* x4t,
                                  void* dx, void* dw, void* ws, size_t ws_bytes,
                                  cudaStream_t stream) {
  if (dx == nullptr && dw == nullptr) return FP8LIN_OK;
  if ((dx != nullptr && dy4 == nullptr) || (dw != nullptr && dy4t == nullptr)) return FP8LIN_EINVAL;
  if (dx == nullptr) dy4 = nullptr;    // a copy that no product reads is not made
  if (dw == nullptr) dy4t = nullptr;
  const int64_t M = dy4 != nullptr ? dy4->rows : dy4t->cols;
  const int64_t N = dy4 != nullptr ? dy4->cols : dy4t->rows;
  if (dy4 != nullptr && dy4t != nullptr && !fp4_transposed(dy4, dy4t)) return FP8LIN_EINVAL;
  fp8lin_status s = check_quantise(dy, M, N, N, sdy, dy4, dy4t, ws);
  if (s != FP8LIN_OK) return s;
  if (dx != nullptr &&
      (w4t == nullptr || (s = check_fp4_gemm(dy4, w4t, dx, w4t->rows, ws, ws_bytes)) != FP8LIN_OK))
    return w4t == nullptr ? FP8LIN_EINVAL : s;
  if (dw != nullptr &&
      (x4t == nullptr || (s = check_fp4_gemm(dy4t, x4t, dw, x4t->rows, ws, ws_bytes)) != FP8LIN_OK))
    return x4t == nullptr ? FP8LIN_EINVAL : s;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  const QuantJob job = {dy, M, N, N, sdy, dy4, dy4t};
  if ((s = run_quantise(&job, 1, ws, dev, stream)) != FP8LIN_OK) return s;
  if (dx != nullptr &&
      (s = run_fp4_gemm(dy4, w4t, dx, w4t->rows, ws, ws_bytes, dev, stream)) != FP8LIN_OK)
    return s;
  if (dw != nullptr) return run_fp4_gemm(dy4t, x4t, dw, x4t->rows, ws, ws_bytes, dev, stream);
  return FP8LIN_OK;
}

// ---- gradient norm and clipping

namespace {

fp8lin_status check_grads(const fp8lin_grad* grads, int32_t count, bool outs) {
  if (count < 0 || (count > 0 && grads == nullptr)) return FP8LIN_EINVAL;
  for (int32_t i = 0; i < count; ++i) {
    const fp8lin_grad& t = grads[i];
    if (t.n < 0) return FP8LIN_EINVAL;
    if (t.n == 0) continue;
    if (t.g == nullptr || (reinterpret_cast<uintptr_t>(t.g) & (t.g_f32 ? 3u : 1u)) != 0)
      return FP8LIN_EINVAL;
    if (!outs) continue;
    if (t.out == nullptr || (reinterpret_cast<uintptr_t>(t.out) & (t.out_f32 ? 3u : 1u)) != 0)
      return FP8LIN_EINVAL;
    if (t.out == t.g && (t.out_f32 != 0) != (t.g_f32 != 0)) return FP8LIN_EINVAL;
  }
  return FP8LIN_OK;
}

double* norm_partials(void* ws) {
  return reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kWsPartialOffset);
}

// left: null, or where a single launch may leave its partial sums for the
// scaling; then their number, else 0.
fp8lin_status run_grad_norm(const fp8lin_grad* grads, int32_t count, float* norm, void* ws,
                            const DeviceInfo& dev, cudaStream_t stream, int* left) {
  GradNormArgs a;
  a.partials = norm_partials(ws);
  a.total = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kWsNormTotalOffset);
  a.ticket = ws_u32(ws, kWsAtomicTicketOffset);
  a.norm = norm;
  int64_t of[2] = {0, 0};
  for (int32_t i = 0; i < count; ++i)
    if (grads[i].n > 0) ++of[grads[i].g_f32 != 0];
  int64_t launches = 0;
  for (int64_t n : of) launches += (n + kClipMaxTensors - 1) / kClipMaxTensors;
  if (left != nullptr) *left = 0;
  if (launches == 0) {
    cudaError_t e = cudaMemsetAsync(norm, 0, sizeof(float), stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  a.leave = left != nullptr && launches == 1;
  int64_t k = 0;
  for (int f32 = 0; f32 < 2; ++f32) {
    a.bf16 = f32 == 0;
    fp8lin_status s = for_lists(
        grads, count, [&](const fp8lin_grad& t) { return (t.g_f32 != 0) == (f32 != 0); },
        [&](const GradTensor* list, int n) {
          ProfScope ps(FP8LIN_PROF_AMAX, stream);
          a.first = k == 0;
          a.last = ++k == launches;
          int grid = 0;
          cudaError_t e = launch_grad_norm(list, n, a, dev, stream, &grid);
          if (a.leave) *left = grid;
          return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
        });
    if (s != FP8LIN_OK) return s;
  }
  return FP8LIN_OK;
}

fp8lin_status run_grad_clip(const fp8lin_grad* grads, int32_t count, GradScaleArgs a,
                            const DeviceInfo& dev, cudaStream_t stream) {
  for (int kind = 0; kind < 4; ++kind) {
    const bool f32 = (kind & 1) != 0, out_f32 = (kind & 2) != 0;
    a.bf16 = !f32;
    a.out_bf16 = !out_f32;
    fp8lin_status s = for_lists(
        grads, count,
        [&](const fp8lin_grad& t) { return (t.g_f32 != 0) == f32 && (t.out_f32 != 0) == out_f32; },
        [&](const GradTensor* list, int n) {
          ProfScope ps(FP8LIN_PROF_SCALE, stream);
          cudaError_t e = launch_grad_scale(list, n, a, dev, stream);
          return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
        });
    if (s != FP8LIN_OK) return s;
  }
  return FP8LIN_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

fp8lin_status fp8lin_grad_norm(const fp8lin_grad* grads, int32_t count, float* norm, void* ws,
                               size_t ws_bytes, cudaStream_t stream) {
  fp8lin_status s = check_grads(grads, count, false);
  if (s != FP8LIN_OK) return s;
  if (norm == nullptr || !aligned4(norm) || !ws_ok(ws) || ws_bytes < kWsFixedBytes)
    return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  return run_grad_norm(grads, count, norm, ws, dev, stream, nullptr);
}

fp8lin_status fp8lin_grad_clip(const fp8lin_grad* grads, int32_t count, const float* norm,
                               float max_norm, float eps, cudaStream_t stream) {
  fp8lin_status s = check_grads(grads, count, true);
  if (s != FP8LIN_OK) return s;
  if (norm == nullptr || !aligned4(norm) || !(max_norm >= 0.0f) || !(eps >= 0.0f))
    return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  GradScaleArgs a = {};
  a.norm = const_cast<float*>(norm);  // only read: count is 0
  a.max_norm = max_norm;
  a.eps = eps;
  return run_grad_clip(grads, count, a, dev, stream);
}

fp8lin_status fp8lin_grad_clip_norm(const fp8lin_grad* grads, int32_t count, float max_norm,
                                    float eps, float* norm, void* ws, size_t ws_bytes,
                                    cudaStream_t stream) {
  fp8lin_status s = check_grads(grads, count, true);
  if (s != FP8LIN_OK) return s;
  if (norm == nullptr || !aligned4(norm) || !ws_ok(ws) || ws_bytes < kWsFixedBytes ||
      !(max_norm >= 0.0f) || !(eps >= 0.0f))
    return FP8LIN_EINVAL;
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  GradScaleArgs a = {};
  a.norm = norm;
  a.max_norm = max_norm;
  a.eps = eps;
  a.partials = norm_partials(ws);
  if ((s = run_grad_norm(grads, count, norm, ws, dev, stream, &a.count)) != FP8LIN_OK) return s;
  return run_grad_clip(grads, count, a, dev, stream);
}

// ---- layer norm

namespace {

// A bf16 [rows, cols] tensor of any stride and alignment that a call needs.
bool bf16_rows_ok(const void* p, int64_t cols, int64_t ld) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 1u) == 0 && ld >= cols;
}

// Of an output that may be an input too: it then has the same rows.
bool same_rows(const void* out, int64_t ldout, const void* in, int64_t ldin, int64_t rows) {
  return out == nullptr || out != in || ldout == ldin || rows <= 1;
}

// Whether two buffers of `bytes` each have any in common.
bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q ? q - p < bytes : p - q < bytes;
}

bool param_ok(const void* p, int32_t f32) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (f32 ? 3u : 1u)) == 0;
}

fp8lin_status zero_async(void* p, size_t bytes, cudaStream_t stream) {
  if (p == nullptr) return FP8LIN_OK;
  cudaError_t e = cudaMemsetAsync(p, 0, bytes, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

}  // namespace

fp8lin_status fp8lin_layer_norm(const void* x, int64_t ldx, const void* r, int64_t ldr, void* h,
                                int64_t ldh, const void* w, const void* b, int32_t param_f32,
                                int64_t rows, int64_t cols, float eps, void* y, int64_t ldy,
                                float* stats, float* y_amax, void* ws, cudaStream_t stream) {
  if (rows < 0 || cols < 0 || !(eps >= 0.0f)) return FP8LIN_EINVAL;
  if (cols < 1 || cols > kNormMaxCols) return FP8LIN_EUNSUPPORTED;
  if (!aligned4(stats) || !aligned4(y_amax) || (y_amax != nullptr && !ws_ok(ws)))
    return FP8LIN_EINVAL;
  if ((r == nullptr) != (h == nullptr)) return FP8LIN_EINVAL;
  if (!param_ok(w, param_f32) || (b != nullptr && !param_ok(b, param_f32))) return FP8LIN_EINVAL;
  if (rows > 0) {
    if (!bf16_rows_ok(x, cols, ldx) || !bf16_rows_ok(y, cols, ldy)) return FP8LIN_EINVAL;
    if (r != nullptr && (!bf16_rows_ok(r, cols, ldr) || !bf16_rows_ok(h, cols, ldh)))
      return FP8LIN_EINVAL;
    if (!same_rows(h, ldh, x, ldx, rows) || !same_rows(h, ldh, r, ldr, rows) ||
        !same_rows(y, ldy, x, ldx, rows) || !same_rows(y, ldy, r, ldr, rows) ||
        !same_rows(y, ldy, h, ldh, rows))
      return FP8LIN_EINVAL;
  }
  DeviceInfo dev;
  fp8lin_status s = get_dev(&dev);
  if (s != FP8LIN_OK) return s;
  if (rows == 0) return zero_async(y_amax, sizeof(float), stream);
  LayerNormArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.r = static_cast<const uint16_t*>(r);
  a.ldr = ldr;
  a.h = static_cast<uint16_t*>(h);
  a.ldh = ldh;
  a.w = w;
  a.b = b;
  a.param_f32 = param_f32 != 0;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.y = static_cast<uint16_t*>(y);
  a.ldy = ldy;
  a.stats = stats;
  if (y_amax != nullptr) {
    a.amax = reinterpret_cast<uint32_t*>(y_amax);
    a.acc = ws_u32(ws, kWsAtomicAccOffset);
    a.ticket = ws_u32(ws, kWsAtomicTicketOffset);
  }
  ProfScope ps(FP8LIN_PROF_CAST, stream);
  cudaError_t e = launch_layer_norm(a, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                         const void* w, int32_t param_f32, const float* stats,
                                         int64_t rows, int64_t cols, const void* dres,
                                         int64_t lddres, void* dx, int64_t lddx, void* dw, void* db,
                                         float* dx_amax, void* ws, size_t ws_bytes,
                                         cudaStream_t stream) {
  if (rows < 0 || cols < 0) return FP8LIN_EINVAL;
  if (cols < 1 || cols > kNormMaxCols) return FP8LIN_EUNSUPPORTED;
  if (!param_ok(w, param_f32) || (dw != nullptr && !param_ok(dw, param_f32)) ||
      (db != nullptr && !param_ok(db, param_f32)))
    return FP8LIN_EINVAL;
  if (!aligned4(dx_amax) || (dx_amax != nullptr && dx == nullptr && rows > 0)) return FP8LIN_EINVAL;
  // Partial column sums: room for those of one CTA at least.
  const size_t room = sizeof(float) * 2 * static_cast<size_t>(cols + 7);
  if (!ws_ok(ws) || ws_bytes < kWsSplitOffset + room) return FP8LIN_EINVAL;
  if (rows > 0) {
    if (!bf16_rows_ok(dy, cols, lddy) || !bf16_rows_ok(x, cols, ldx)) return FP8LIN_EINVAL;
    if (dres != nullptr && !bf16_rows_ok(dres, cols, lddres)) return FP8LIN_EINVAL;
    if (dx != nullptr && !bf16_rows_ok(dx, cols, lddx)) return FP8LIN_EINVAL;
    if (!same_rows(dx, lddx, dy, lddy, rows) || !same_rows(dx, lddx, dres, lddres, rows)) return FP8LIN_EINVAL;
    if (stats == nullptr || !aligned4(stats)) return FP8LIN_EINVAL;
  }
  DeviceInfo dev;
  fp8lin_status s = get_dev(&dev);
  if (s != FP8LIN_OK) return s;
  if (rows == 0) {
    const size_t bytes = static_cast<size_t>(cols) * (param_f32 ? 4 : 2);
    if ((s = zero_async(dw, bytes, stream)) != FP8LIN_OK) return s;
    if ((s = zero_async(db, bytes, stream)) != FP8LIN_OK) return s;
    return zero_async(dx_amax, sizeof(float), stream);
  }
  if (dx == nullptr && dw == nullptr && db == nullptr) return FP8LIN_OK;
  LayerNormBackwardArgs a = {};
  a.dy = static_cast<const uint16_t*>(dy);
  a.lddy = lddy;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.w = w;
  a.param_f32 = param_f32 != 0;
  a.stats = stats;
  a.rows = rows;
  a.cols = cols;
  a.dres = static_cast<const uint16_t*>(dres);
  a.lddres = lddres;
  a.dx = static_cast<uint16_t*>(dx);
  a.lddx = lddx;
  a.dw = dw;
  a.db = db;
  if (dx_amax != nullptr) {
    a.amax = reinterpret_cast<uint32_t*>(dx_amax);
    a.acc = ws_u32(ws, kWsAtomicAccOffset);
    a.ticket = ws_u32(ws, kWsAtomicTicketOffset);
  }
  a.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsSplitOffset);
  a.ws_bytes = ws_bytes - kWsSplitOffset;
  int launches = 0;
  cudaError_t e;
  {
    ProfScope ps(FP8LIN_PROF_CAST, stream);
    e = launch_layer_norm_backward(a, dev, stream, &launches);
  }
  if (launches > 1) g_launches.fetch_add(1, std::memory_order_relaxed);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

// ---- low-rank adapters

namespace {

// The bank and its rows' adapters.
fp8lin_status check_adapters(const fp8lin_adapters* ad, int64_t rows, const int32_t* index,
                             const void* route) {
  if (ad == nullptr || ad->count < 1 || ad->k < 1 || ad->n < 1 || ad->rank < 1 || rows < 0)
    return FP8LIN_EINVAL;
  if (ad->count > kAdapterMaxCount || ad->rank > kAdapterMaxRank || ad->k > kAdapterMaxDim ||
      ad->n > kAdapterMaxDim || rows > kAdapterMaxRows)
    return FP8LIN_EUNSUPPORTED;
  for (const void* p : {ad->a, ad->b})
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 1u) != 0) return FP8LIN_EINVAL;
  if (ad->scale == nullptr || !aligned4(ad->scale)) return FP8LIN_EINVAL;
  if (!aligned4(index) || !aligned4(route)) return FP8LIN_EINVAL;
  if (rows > 0 && index == nullptr && route == nullptr) return FP8LIN_EINVAL;
  return FP8LIN_OK;
}

AdapterArgs adapter_args(const fp8lin_adapters* ad, int64_t rows) {
  AdapterArgs a = {};
  a.a = static_cast<const uint16_t*>(ad->a);
  a.b = static_cast<const uint16_t*>(ad->b);
  a.scale = ad->scale;
  a.count = ad->count;
  a.k = ad->k;
  a.n = ad->n;
  a.rank = ad->rank;
  a.rows = rows;
  return a;
}

// The caller's route, or one made at the start of the workspace's room, which
// then begins behind it.
fp8lin_status route_rows(AdapterArgs& a, const int32_t* index, const void* route, uint8_t*& room,
                         size_t& room_bytes, const DeviceInfo& dev, cudaStream_t stream) {
  a.route = static_cast<const int32_t*>(route);
  if (route != nullptr) return FP8LIN_OK;
  const size_t bytes = adapter_route_bytes(a.rows, a.count);
  if (bytes > room_bytes) return FP8LIN_EUNSUPPORTED;
  ProfScope ps(FP8LIN_PROF_SCALE, stream);
  int32_t* made = reinterpret_cast<int32_t*>(room);
  cudaError_t e = launch_adapter_route(index, a.rows, a.count, made, dev, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  a.route = made;
  room += bytes;
  room_bytes -= bytes;
  return FP8LIN_OK;
}

}  // namespace

size_t fp8lin_adapter_route_bytes(int64_t rows, int64_t count) {
  if (rows < 0 || rows > kAdapterMaxRows || count < 1 || count > kAdapterMaxCount) return 0;
  return adapter_route_bytes(rows, count);
}

fp8lin_status fp8lin_adapter_route(const int32_t* index, int64_t rows, int64_t count, void* route,
                                   cudaStream_t stream) {
  if (rows < 0 || count < 1) return FP8LIN_EINVAL;
  if (rows > kAdapterMaxRows || count > kAdapterMaxCount) return FP8LIN_EUNSUPPORTED;
  if (!aligned4(index) || (rows > 0 && index == nullptr) || route == nullptr || !aligned4(route))
    return FP8LIN_EINVAL;
  DeviceInfo dev;
  fp8lin_status s = get_dev(&dev);
  if (s != FP8LIN_OK) return s;
  ProfScope ps(FP8LIN_PROF_SCALE, stream);
  cudaError_t e = launch_adapter_route(index, rows, count, static_cast<int32_t*>(route), dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_adapter_linear(const fp8lin_adapters* ad, const void* x, int64_t ldx,
                                    const int32_t* index, const void* route, int64_t rows,
                                    const void* base, int64_t ldbase, void* y, int64_t ldy, float* h,
                                    void* ws, size_t ws_bytes, cudaStream_t stream) {
  fp8lin_status s = check_adapters(ad, rows, index, route);
  if (s != FP8LIN_OK) return s;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  if (rows > 0) {
    if (!bf16_rows_ok(x, ad->k, ldx) || !bf16_rows_ok(y, ad->n, ldy)) return FP8LIN_EINVAL;
    if (base != nullptr && !bf16_rows_ok(base, ad->n, ldbase)) return FP8LIN_EINVAL;
    if (!same_rows(y, ldy, base, ldbase, rows) || y == x) return FP8LIN_EINVAL;
    if (h == nullptr || !aligned4(h)) return FP8LIN_EINVAL;
  }
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  if (rows == 0) return FP8LIN_OK;
  AdapterArgs a = adapter_args(ad, rows);
  const uint16_t* xs = static_cast<const uint16_t*>(x);
  const uint16_t* bases = static_cast<const uint16_t*>(base);
  uint16_t* ys = static_cast<uint16_t*>(y);
  if (index != nullptr && adapter_few_fits(a)) {
    ProfScope ps(FP8LIN_PROF_SMALL_M, stream);
    cudaError_t e = launch_adapter_few(a, index, xs, ldx, bases, ldbase, ys, ldy, h, stream);
    return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
  }
  uint8_t* room = static_cast<uint8_t*>(ws) + kWsSplitOffset;
  size_t room_bytes = ws_bytes > kWsSplitOffset ? ws_bytes - kWsSplitOffset : 0;
  if ((s = route_rows(a, index, route, room, room_bytes, dev, stream)) != FP8LIN_OK) return s;
  {
    ProfScope ps(FP8LIN_PROF_GEMM, stream);
    cudaError_t e = launch_adapter_low(a, false, xs, ldx, h, dev, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  ProfScope ps(FP8LIN_PROF_GEMM, stream);
  cudaError_t e = launch_adapter_high(a, false, h, bases, ldbase, ys, ldy, dev, stream);
  return e == cudaSuccess ? FP8LIN_OK : cuda_fail(e);
}

fp8lin_status fp8lin_adapter_backward(const fp8lin_adapters* ad, const void* dy, int64_t lddy,
                                      const void* x, int64_t ldx, const float* h,
                                      const int32_t* index, const void* route, int64_t rows,
                                      const void* base, int64_t ldbase, void* dx, int64_t lddx,
                                      float* dh, void* da, void* db, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  fp8lin_status s = check_adapters(ad, rows, index, route);
  if (s != FP8LIN_OK) return s;
  if (!ws_ok(ws) || ws_bytes < kWsFixedBytes) return FP8LIN_EINVAL;
  for (const void* p : {static_cast<const void*>(da), static_cast<const void*>(db)})
    if ((reinterpret_cast<uintptr_t>(p) & 1u) != 0) return FP8LIN_EINVAL;
  if (rows > 0) {
    if (!bf16_rows_ok(dy, ad->n, lddy)) return FP8LIN_EINVAL;
    if (da != nullptr && !bf16_rows_ok(x, ad->k, ldx)) return FP8LIN_EINVAL;
    if (db != nullptr && (h == nullptr || !aligned4(h))) return FP8LIN_EINVAL;
    if (base != nullptr && !bf16_rows_ok(base, ad->k, ldbase)) return FP8LIN_EINVAL;
    if (dx != nullptr && !bf16_rows_ok(dx, ad->k, lddx)) return FP8LIN_EINVAL;
    if (!same_rows(dx, lddx, base, ldbase, rows)) return FP8LIN_EINVAL;
    if (dx != nullptr && (dx == dy || (da != nullptr && dx == x))) return FP8LIN_EINVAL;
    if (dh == nullptr || !aligned4(dh)) return FP8LIN_EINVAL;
    // dh is written before dB reads h.
    if (db != nullptr && overlap(dh, h, static_cast<size_t>(rows) * ad->rank * sizeof(float))) return FP8LIN_EINVAL;
  }
  DeviceInfo dev;
  if ((s = get_dev(&dev)) != FP8LIN_OK) return s;
  const size_t da_bytes = static_cast<size_t>(ad->count) * ad->rank * ad->k * 2;
  const size_t db_bytes = static_cast<size_t>(ad->count) * ad->rank * ad->n * 2;
  if (rows == 0) {
    if ((s = zero_async(da, da_bytes, stream)) != FP8LIN_OK) return s;
    return zero_async(db, db_bytes, stream);
  }
  AdapterArgs a = adapter_args(ad, rows);
  const uint16_t* dys = static_cast<const uint16_t*>(dy);
  uint8_t* room = static_cast<uint8_t*>(ws) + kWsSplitOffset;
  size_t room_bytes = ws_bytes > kWsSplitOffset ? ws_bytes - kWsSplitOffset : 0;
  if ((s = route_rows(a, index, route, room, room_bytes, dev, stream)) != FP8LIN_OK) return s;
  cudaError_t e;
  {
    ProfScope ps(FP8LIN_PROF_GEMM, stream);
    e = launch_adapter_low(a, true, dys, lddy, dh, dev, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  // The weight gradients' operands from h and dh, laid out once where the rows pay for
  // that launch (16384 x 4096 x 14336 with rank 16: 264 us with it, 386 without; 1024 x
  // 4096 x 4096: 31 and 32; with rank 32, 318 x 5954 x 1857 of three adapters: 38.5 and
  // 40.2) and the workspace has room.  Below that it is one launch less for the same time
  // (256 rows of one adapter 18.9 and 19.1; with rank 64, 201 x 5550 x 185 of six 34.9 and
  // 35.4).
  AdapterWeight wa, wb;
  if (da != nullptr) {
    wa.dw = static_cast<uint16_t*>(da);
    wa.x = static_cast<const uint16_t*>(x);
    wa.ldx = ldx;
    wa.low = dh;
  }
  if (db != nullptr) {
    wb.dw = static_cast<uint16_t*>(db);
    wb.x = dys;
    wb.ldx = lddy;
    wb.low = h;
  }
  const int64_t pays = ad->rank > 16 && 64 * ad->count < 512 ? 64 * ad->count : 512;
  const size_t packed = (adapter_packed_bytes(a) + 255) / 256 * 256;
  for (AdapterWeight* w : {&wa, &wb}) {
    if (w->dw == nullptr || rows < pays || packed > room_bytes) continue;
    w->packed = room;
    room += packed;
    room_bytes -= packed;
  }
  if (wa.packed != nullptr || wb.packed != nullptr) {
    ProfScope ps(FP8LIN_PROF_GEMM, stream);
    e = launch_adapter_pack(a, wb, wa, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  if (da != nullptr || db != nullptr) {
    ProfScope ps(FP8LIN_PROF_GEMM, stream);
    e = launch_adapter_weight(a, wb, wa, dev, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  if (dx != nullptr) {
    ProfScope ps(FP8LIN_PROF_GEMM, stream);
    e = launch_adapter_high(a, true, dh, static_cast<const uint16_t*>(base), ldbase,
                            static_cast<uint16_t*>(dx), lddx, dev, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return FP8LIN_OK;
}

uint64_t fp8lin_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

void fp8lin_profile_enable(int on) {
  g_prof_on = on != 0;
  if (g_prof_on) g_prof_used = 0;
}

int64_t fp8lin_profile_launches(double* ms, int32_t* kind, int64_t capacity) {
  if (ms == nullptr || kind == nullptr || capacity < 0) return -static_cast<int64_t>(FP8LIN_EINVAL);
  const int64_t n = g_prof_used < capacity ? g_prof_used : capacity;
  for (int64_t i = 0; i < n; ++i) {
    cudaError_t e = cudaEventSynchronize(g_prof[i].stop);
    if (e != cudaSuccess) return -static_cast<int64_t>(cuda_fail(e));
    float t = 0.0f;
    e = cudaEventElapsedTime(&t, g_prof[i].start, g_prof[i].stop);
    if (e != cudaSuccess) return -static_cast<int64_t>(cuda_fail(e));
    ms[i] = t;
    kind[i] = g_prof[i].kind;
  }
  g_prof_used = 0;
  return n;
}

fp8lin_status fp8lin_profile_collect(double* ms, int64_t* count) {
  if (ms == nullptr || count == nullptr) return FP8LIN_EINVAL;
  for (int k = 0; k < FP8LIN_PROF_KINDS; ++k) {
    ms[k] = 0.0;
    count[k] = 0;
  }
  for (int i = 0; i < g_prof_used; ++i) {
    cudaError_t e = cudaEventSynchronize(g_prof[i].stop);
    if (e != cudaSuccess) return cuda_fail(e);
    float t = 0.0f;
    e = cudaEventElapsedTime(&t, g_prof[i].start, g_prof[i].stop);
    if (e != cudaSuccess) return cuda_fail(e);
    ms[g_prof[i].kind] += t;
    count[g_prof[i].kind] += 1;
  }
  g_prof_used = 0;
  return FP8LIN_OK;
}

}  // extern "C"
