// Entry points of the 8-bit operators: argument checks (all of them before
// any HIP call) and launches.
#include <algorithm>
#include <atomic>
#include <map>
#include <tuple>

#include "fp8_checks.hpp"

namespace {

// ------------------------------------------------------------- workspace
// The split products' sums and the column sums of gradients, one buffer per (device,
// stream). Every split plan fits kOwnBytes (at most 512 tiles of 128 x 128 fp32 sums);
// what needs more has a second buffer of kOwnWideBytes (the widest norm's gradients take
// 101 MB), and what needs more than that is refused without a caller's. So a buffer
// never grows and nothing waits for the stream. It needs no clearing. A split product
// is two launches: whoever enqueues them holds the buffer's lock over both, so
// that host threads that share a stream do not put one product's sums between
// the other's sums and their joining. The per-thread default stream is a stream
// of each thread under one handle: there the thread is part of the key.
constexpr size_t kOwnBytes = (size_t)512 * 128 * 128 * 4, kOwnWideBytes = (size_t)128 << 20;
struct OwnWorkspace {
  std::mutex mu;
  void* ptr = nullptr;
};
struct OwnKey {
  int dev;
  void* stream;
  uint64_t thread;   // 0 but for hipStreamPerThread
  bool wide;         // the buffer of kOwnWideBytes
  bool operator<(const OwnKey& o) const {
    return std::tie(dev, stream, thread, wide) < std::tie(o.dev, o.stream, o.thread, o.wide);
  }
};
std::mutex g_mu;   // of the map; its entries stay
std::map<OwnKey, OwnWorkspace> g_own;

// a number of this thread that no other thread has or will have
uint64_t thread_number() {
  static std::atomic<uint64_t> count{0};
  thread_local const uint64_t mine = ++count;
  return mine;
}

}  // namespace

namespace iris {
int fp8_own_workspace(int dev, void* stream, size_t need, void** out, std::unique_lock<std::mutex>* hold) {
  if (need > kOwnWideBytes)
    return fail(IRIS_ERR_WORKSPACE, "a workspace of %zu bytes has to be passed (the library's own holds %zu)", need, kOwnWideBytes);
  const bool wide = need > kOwnBytes;
  const size_t bytes = wide ? kOwnWideBytes : kOwnBytes;
  try {
    OwnWorkspace* w;
    {
      std::lock_guard<std::mutex> lk(g_mu);
      w = &g_own[{dev, stream, stream == (void*)hipStreamPerThread ? thread_number() : 0, wide}];
    }
    *hold = std::unique_lock<std::mutex>(w->mu);
    if (!w->ptr) {
      // allocating is no stream operation: allowed while a stream captures
      hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
      (void)hipThreadExchangeStreamCaptureMode(&mode);
      const hipError_t e = hipMalloc(&w->ptr, bytes);
      (void)hipThreadExchangeStreamCaptureMode(&mode);
      if (e != hipSuccess) {
        w->ptr = nullptr;
        return fail(IRIS_ERR_NO_MEMORY, "hipMalloc of a %zu-byte workspace failed: %s", bytes, hipGetErrorString(e));
      }
    }
    *out = w->ptr;
    return IRIS_OK;
  } catch (const std::exception& e) {
    return fail(IRIS_ERR_NO_MEMORY, "workspace: %s", e.what());
  }
}

// iris_finalize's share: frees the workspaces above once their streams are done
int fp8_finalize() {
  std::lock_guard<std::mutex> lk(g_mu);
  int status = IRIS_OK;
  for (auto& kv : g_own) {
    std::lock_guard<std::mutex> hold(kv.second.mu);
    if (!kv.second.ptr) continue;
    (void)hipSetDevice(kv.first.dev);
    // another thread's default stream cannot be named here
    if (kv.first.thread)
      (void)hipDeviceSynchronize();
    else
      (void)hipStreamSynchronize((hipStream_t)kv.first.stream);
    if (hipFree(kv.second.ptr) != hipSuccess) status = IRIS_ERR_HIP;
    kv.second.ptr = nullptr;
  }
  return status;
}
}  // namespace iris

extern "C" {

int iris_fp8_quantize(const iris_fp8_t* q, const iris_fp8_t* q_t, const void* x, int32_t x_type, int64_t ldx,
                      const iris_fp8_t* x8, int64_t rows, int64_t cols, void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  if ((st = check_dims(rows, cols)) || (st = check_dims(cols, rows))) return st;
  if (!q && !q_t) return fail(IRIS_ERR_INVALID_ARG, "q and q_t are both NULL");
  if (q && (st = check_fp8(q, rows, cols, "q"))) return st;
  if (q_t && (st = check_fp8(q_t, cols, rows, "q_t"))) return st;
  if (q && q_t && q->block != q_t->block)
    return fail(IRIS_ERR_INVALID_ARG, "q and q_t have different blocks (%d, %d)", q->block, q_t->block);
  iris::Fp8QuantArgs a{};
  a.block = q ? q->block : q_t->block;
  if ((q_t || a.block != 1) && (st = check_tiles(rows, cols))) return st;
  if (x8) {
    if (x) return fail(IRIS_ERR_INVALID_ARG, "x and x8 are both given");
    if (q || a.block != 1)
      return fail(IRIS_ERR_UNSUPPORTED, "an 8-bit matrix is only turned around: q must be NULL and q_t's block 1");
    if ((st = check_blocks1(x8, rows, cols, "x8"))) return st;
    a.x8 = mat(x8);
    a.x_type = iris::T_FP8;
  } else {
    if ((st = check_plain(x, x_type, true, ldx, rows, cols, "x"))) return st;
    a.x = x;
    a.ldx = (int32_t)ldx;
    a.x_type = x_type;
    a.vec = rows16(x, ldx, x_type);
  }
  if (rows == 0 || cols == 0) return IRIS_OK;
  if ((st = check_distinct({{q, "q", true}, {q_t, "q_t", true}, {x, "x", false}, {x8, "x8", false}}))) return st;
  if ((st = ready())) return st;
  a.q = mat(q);
  a.qt = mat(q_t);
  a.rows = (int)rows;
  a.cols = (int)cols;
  return launched(iris::launch_fp8_quantize(a, (hipStream_t)stream), "iris_fp8_quantize");
} catch (const std::exception& e) {
  return caught(e);
}

size_t iris_fp8_mm_workspace_size(int64_t M, int64_t N, int64_t K) try {
  if (check_mm_dims(M, N, K) || M == 0 || N == 0) return 0;
  return std::max(iris::fp8_mm_plan(M, N, K, false).ws_bytes, iris::fp8_mm_plan(M, N, K, true).ws_bytes);
} catch (const std::exception&) {
  return 0;
}

int iris_fp8_mm(void* C, int32_t c_type, int64_t ldc, const iris_fp8_t* A, const iris_fp8_t* B, const void* bias,
                int64_t M, int64_t N, int64_t K, int32_t flags, void* workspace, size_t workspace_bytes,
                void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st = check_mm_dims(M, N, K);
  if (st) return st;
  if (flags & ~(IRIS_FLAG_BIAS_ALONG_M | IRIS_FLAG_ACCUMULATE))
    return fail(IRIS_ERR_CONFIG, "unknown flag bits 0x%x", flags);
  if ((st = check_plain(C, c_type, true, ldc, M, N, "C")) || (st = check_blocks1(A, M, K, "A")) ||
      (st = check_fp8(B, N, K, "B")))
    return st;
  if ((st = check_scale_words(A, M, K, "A")) || (st = check_scale_words(B, N, K, "B"))) return st;
  if (bias && (uintptr_t)bias % type_bytes(c_type) != 0) return fail(IRIS_ERR_ALIGNMENT, "bias is not aligned to its type");
  if (M == 0 || N == 0) return IRIS_OK;
  const iris::Fp8MmPlan plan = iris::fp8_mm_plan(M, N, K, c_type == IRIS_TYPE_FP32);
  if (workspace && workspace_bytes < plan.ws_bytes)
    return fail(IRIS_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, plan.ws_bytes);
  if (workspace && (uintptr_t)workspace % 256 != 0) return fail(IRIS_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if ((st = check_distinct({{C, "C", true}, {A, "A", false}, {B, "B", false}, {bias, "bias", false},
                            {workspace, "workspace", true}})))
    return st;
  int dev = 0, cus = 0;
  if ((st = iris::use_device(&dev, &cus))) return st;
  std::unique_lock<std::mutex> hold;   // over both launches of a split product
  if (plan.ws_bytes > 0 && !workspace && (st = iris::fp8_own_workspace(dev, stream, plan.ws_bytes, &workspace, &hold))) return st;
  iris::Fp8MmArgs a{};
  a.A = mat(A);
  a.B = mat(B);
  a.b_block = (uint8_t)B->block;
  a.bias = bias;
  a.bias_along_m = (flags & IRIS_FLAG_BIAS_ALONG_M) ? 1 : 0;
  a.accumulate = (flags & IRIS_FLAG_ACCUMULATE) ? 1 : 0;
  a.C = C;
  a.c_type = (uint8_t)c_type;
  a.ldc = (int32_t)ldc;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  const hipError_t e = plan.bm == 0 ? iris::launch_fp8_mm_few(a, (hipStream_t)stream)
                                              : iris::launch_fp8_mm(a, plan, workspace, (hipStream_t)stream);
  return launched(e, "iris_fp8_mm");
} catch (const std::exception& e) {
  return caught(e);
}

int iris_fp8_swiglu(const iris_fp8_t* h, const iris_fp8_t* gate_kept, const iris_fp8_t* up_kept, const void* gate,
                    const void* up, int32_t type, int64_t ld_gate, int64_t ld_up, int64_t rows, int64_t cols,
                    void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  if ((st = check_dims(rows, cols)) || (st = check_blocks1(h, rows, cols, "h"))) return st;
  if (!gate_kept != !up_kept) return fail(IRIS_ERR_INVALID_ARG, "gate_kept and up_kept go together");
  if (gate_kept && ((st = check_blocks1(gate_kept, rows, cols, "gate_kept")) ||
                    (st = check_blocks1(up_kept, rows, cols, "up_kept"))))
    return st;
  if ((st = check_plain(gate, type, false, ld_gate, rows, cols, "gate")) ||
      (st = check_plain(up, type, false, ld_up, rows, cols, "up")))
    return st;
  if (rows == 0 || cols == 0) return IRIS_OK;
  if ((st = check_distinct({{h, "h", true}, {gate_kept, "gate_kept", true}, {up_kept, "up_kept", true},
                            {gate, "gate", false}, {up, "up", false}})))
    return st;
  if ((st = ready())) return st;
  iris::Fp8SwigluArgs a{};
  a.gate = gate;
  a.up = up;
  a.ld_gate = (int32_t)ld_gate;
  a.ld_up = (int32_t)ld_up;
  a.type = type;
  a.vec = rows16(gate, ld_gate, type) && rows16(up, ld_up, type);
  a.h = mat(h);
  a.gate8 = mat(gate_kept);
  a.up8 = mat(up_kept);
  a.rows = (int)rows;
  a.cols = (int)cols;
  return launched(iris::launch_fp8_swiglu(a, (hipStream_t)stream), "iris_fp8_swiglu");
} catch (const std::exception& e) {
  return caught(e);
}

int iris_fp8_swiglu_bwd(const iris_fp8_t* dgate, const iris_fp8_t* dup, const iris_fp8_t* dgate_t,
                        const iris_fp8_t* dup_t, const iris_fp8_t* h_t, const void* dh, int32_t type, int64_t ld_dh,
                        const iris_fp8_t* gate_kept, const iris_fp8_t* up_kept, int64_t rows, int64_t cols,
                        void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  if ((st = check_dims(rows, cols)) || (st = check_dims(cols, rows))) return st;
  if ((st = check_tiles(rows, cols))) return st;
  const struct {
    const iris_fp8_t* q;
    const char* name;
    bool turned, required;
  } mats[] = {{dgate, "dgate", false, true},          {dup, "dup", false, true},
              {gate_kept, "gate_kept", false, true},  {up_kept, "up_kept", false, true},
              {dgate_t, "dgate_t", true, false},      {dup_t, "dup_t", true, false},
              {h_t, "h_t", true, false}};
  for (const auto& m : mats)
    if ((m.required || m.q) &&
        (st = check_blocks1(m.q, m.turned ? cols : rows, m.turned ? rows : cols, m.name)))
      return st;
  if ((st = check_plain(dh, type, false, ld_dh, rows, cols, "dh"))) return st;
  if (rows == 0 || cols == 0) return IRIS_OK;
  if ((st = check_distinct({{dgate, "dgate", true}, {dup, "dup", true}, {dgate_t, "dgate_t", true}, {dup_t, "dup_t", true},
                            {h_t, "h_t", true}, {gate_kept, "gate_kept", false}, {up_kept, "up_kept", false},
                            {dh, "dh", false}})))
    return st;
  if ((st = ready())) return st;
  iris::Fp8SwigluBwdArgs a{};
  a.dh = dh;
  a.ld_dh = (int32_t)ld_dh;
  a.type = type;
  a.vec = rows16(dh, ld_dh, type);
  a.gate8 = mat(gate_kept);
  a.up8 = mat(up_kept);
  a.dgate = mat(dgate);
  a.dup = mat(dup);
  a.dgate_t = mat(dgate_t);
  a.dup_t = mat(dup_t);
  a.h_t = mat(h_t);
  a.rows = (int)rows;
  a.cols = (int)cols;
  return launched(iris::launch_fp8_swiglu_bwd(a, (hipStream_t)stream), "iris_fp8_swiglu_bwd");
} catch (const std::exception& e) {
  return caught(e);
}

}  // extern "C"
