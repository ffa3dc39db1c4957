// Entry points of the 8-bit operators: argument checks (all of them before
// any HIP call) and launches.
#include "../../include/iris_local.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <map>
#include <mutex>
#include <tuple>

#include "fp8.hpp"

namespace iris {
// beside the other entry points
int set_error(int status, const char* msg);
int use_device(int* dev, int* cus);
}  // namespace iris

namespace {

using iris::Fp8Mat;

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return iris::set_error(status, buf);
}

int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return IRIS_OK;
  return fail(IRIS_ERR_HIP, "%s launch: %s (%d)", what, hipGetErrorString(e), (int)e);
}

constexpr int64_t kBlk = iris::kFp8Block;
// the kernels address a tile's rows with 32-bit offsets
constexpr int64_t kMaxPitch = 1 << 22;
int64_t blocks(int64_t n) { return (n + kBlk - 1) / kBlk; }

// rows and columns of a memory-bound operator: its grid numbers 128-wide
// blocks of rows (or tiles) in 31 bits
int check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0)
    return fail(IRIS_ERR_INVALID_ARG, "rows and cols must not be negative (got %lld, %lld)", (long long)rows,
                (long long)cols);
  if (rows > (1 << 30) || cols > (1 << 30) || (rows > 0 && blocks(cols) > (((int64_t)1 << 31) - 1) / rows))
    return fail(IRIS_ERR_UNSUPPORTED, "matrix too large (limits: rows and cols <= 2^30, rows * ceil(cols / 128) < 2^31)");
  return IRIS_OK;
}

// of the operators that work on tiles of 128 x 128, one launch for all
int check_tiles(int64_t rows, int64_t cols) {
  if (blocks(rows) * blocks(cols) > iris::kMaxTiles)
    return fail(IRIS_ERR_UNSUPPORTED, "matrix too large (limit: fewer than 2^23 tiles of 128 x 128)");
  return IRIS_OK;
}

int check_fp8(const iris_fp8_t* q, int64_t rows, int64_t cols, const char* name) {
  if (!q) return fail(IRIS_ERR_INVALID_ARG, "%s is NULL", name);
  if (q->block != 1 && q->block != kBlk)
    return fail(IRIS_ERR_INVALID_ARG, "%s: block must be 1 or 128 (got %d)", name, q->block);
  if (rows == 0 || cols == 0) return IRIS_OK;
  if (!q->codes || !q->scales) return fail(IRIS_ERR_INVALID_ARG, "%s: codes and scales must not be NULL", name);
  if ((uintptr_t)q->codes % 16 != 0 || q->ld % 16 != 0)
    return fail(IRIS_ERR_ALIGNMENT, "%s: codes must be 16-byte aligned and ld a multiple of 16 (ld %lld)", name,
                (long long)q->ld);
  if (q->ld > kMaxPitch || q->ld_scales > kMaxPitch)
    return fail(IRIS_ERR_UNSUPPORTED, "%s: row pitch too large (limit 2^22)", name);
  if (q->ld < cols)
    return fail(IRIS_ERR_INVALID_ARG, "%s: ld %lld is shorter than the %lld columns", name, (long long)q->ld, (long long)cols);
  if (q->ld_scales < blocks(cols))
    return fail(IRIS_ERR_INVALID_ARG, "%s: ld_scales %lld is shorter than the %lld blocks of a row", name,
                (long long)q->ld_scales, (long long)blocks(cols));
  return IRIS_OK;
}

int check_blocks1(const iris_fp8_t* q, int64_t rows, int64_t cols, const char* name) {
  const int st = check_fp8(q, rows, cols, name);
  if (st) return st;
  if (q->block != 1) return fail(IRIS_ERR_UNSUPPORTED, "%s: block must be 1 here (got %d)", name, q->block);
  return IRIS_OK;
}

int type_bytes(int32_t type) { return type == IRIS_TYPE_FP32 ? 4 : 2; }

int check_plain(const void* x, int32_t type, bool fp32_too, int64_t ld, int64_t rows, int64_t cols, const char* name) {
  if (type != IRIS_TYPE_FP16 && type != IRIS_TYPE_BF16 && !(fp32_too && type == IRIS_TYPE_FP32))
    return fail(IRIS_ERR_INVALID_ARG, "%s: type %d is not served here", name, type);
  if (rows == 0 || cols == 0) return IRIS_OK;
  if (!x) return fail(IRIS_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)x % type_bytes(type) != 0) return fail(IRIS_ERR_ALIGNMENT, "%s is not aligned to its type", name);
  if (ld > kMaxPitch) return fail(IRIS_ERR_UNSUPPORTED, "%s: row pitch too large (limit 2^22)", name);
  if (ld < cols)
    return fail(IRIS_ERR_INVALID_ARG, "%s: row pitch %lld is shorter than the %lld columns", name, (long long)ld, (long long)cols);
  return IRIS_OK;
}

// What a call reads and writes, by address. An output that is also another operand
// would be read before or after it is written as the kernel for its size happens to.
struct Memory {
  const void* at[2];   // codes and scales, or a plain matrix
  const char* name;
  bool output;
  Memory(const iris_fp8_t* q, const char* name, bool output)
      : at{q ? q->codes : nullptr, q ? q->scales : nullptr}, name(name), output(output) {}
  Memory(const void* x, const char* name, bool output) : at{x, nullptr}, name(name), output(output) {}
};
template <size_t N>
int check_distinct(const Memory (&m)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = 0; j < i; ++j) {
      if (!m[i].output && !m[j].output) continue;
      for (const void* p : m[i].at)
        if (p && (p == m[j].at[0] || p == m[j].at[1]))
          return fail(IRIS_ERR_INVALID_ARG, "%s and %s share memory", m[j].name, m[i].name);
    }
  return IRIS_OK;
}

// every row of a plain matrix starts at a multiple of 16 bytes
bool rows16(const void* x, int64_t ld, int32_t type) {
  return (uintptr_t)x % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

Fp8Mat mat(const iris_fp8_t* q) {
  if (!q) return Fp8Mat{};
  return Fp8Mat{(uint8_t*)q->codes, (uint8_t*)q->scales, (int32_t)q->ld, (int32_t)q->ld_scales};
}

// No exception leaves a C entry: what can throw here is memory for a message or
// for a device's record, or a lock.
int caught(const std::exception& e) { return iris::set_error(IRIS_ERR_NO_MEMORY, e.what()); }

int ready() {
  int dev = 0, cus = 0;
  return iris::use_device(&dev, &cus);
}

// ------------------------------------------------------------- workspace
// The split products' sums, one buffer per (device, stream). Every split plan
// fits kOwnBytes (at most 512 tiles of 128 x 128 fp32 sums), so a buffer never
// grows and nothing waits for the stream. It needs no clearing. A split product
// is two launches: whoever enqueues them holds the buffer's lock over both, so
// that host threads that share a stream do not put one product's sums between
// the other's sums and their joining. The per-thread default stream is a stream
// of each thread under one handle: there the thread is part of the key.
constexpr size_t kOwnBytes = (size_t)512 * 128 * 128 * 4;
struct OwnWorkspace {
  std::mutex mu;
  void* ptr = nullptr;
};
struct OwnKey {
  int dev;
  void* stream;
  uint64_t thread;   // 0 but for hipStreamPerThread
  bool operator<(const OwnKey& o) const { return std::tie(dev, stream, thread) < std::tie(o.dev, o.stream, o.thread); }
};
std::mutex g_mu;   // of the map; its entries stay
std::map<OwnKey, OwnWorkspace> g_own;

// a number of this thread that no other thread has or will have
uint64_t thread_number() {
  static std::atomic<uint64_t> count{0};
  thread_local const uint64_t mine = ++count;
  return mine;
}

// The buffer, locked by `hold` until the caller has enqueued all its launches.
int own_workspace(int dev, void* stream, size_t need, void** out, std::unique_lock<std::mutex>* hold) {
  try {
    OwnWorkspace* w;
    {
      std::lock_guard<std::mutex> lk(g_mu);
      w = &g_own[{dev, stream, stream == (void*)hipStreamPerThread ? thread_number() : 0}];
    }
    *hold = std::unique_lock<std::mutex>(w->mu);
    if (!w->ptr) {
      // allocating is no stream operation: allowed while a stream captures
      hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
      (void)hipThreadExchangeStreamCaptureMode(&mode);
      const hipError_t e = hipMalloc(&w->ptr, std::max(need, kOwnBytes));
      (void)hipThreadExchangeStreamCaptureMode(&mode);
      if (e != hipSuccess) {
        w->ptr = nullptr;
        return fail(IRIS_ERR_NO_MEMORY, "hipMalloc of a %zu-byte workspace failed: %s", kOwnBytes, hipGetErrorString(e));
      }
    }
    *out = w->ptr;
    return IRIS_OK;
  } catch (const std::exception& e) {
    return fail(IRIS_ERR_NO_MEMORY, "workspace: %s", e.what());
  }
}

int check_mm_dims(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0)
    return fail(IRIS_ERR_INVALID_ARG, "M, N, K must not be negative (got %lld, %lld, %lld)", (long long)M, (long long)N,
                (long long)K);
  // the largest tile, 256 x 256, has to fit one launch
  if (M > (1 << 30) || N > (1 << 30) || K > (1 << 21) || (M + 255) / 256 * ((N + 255) / 256) > iris::kMaxMmTiles)
    return fail(IRIS_ERR_UNSUPPORTED, "shape too large (limits: M, N <= 2^30, K <= 2^21, fewer than 2^24 output tiles of 256 x 256)");
  return IRIS_OK;
}

}  // namespace

namespace iris {
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
  if (M > 0 && K > 0 && ((uintptr_t)A->scales % 4 != 0 || A->ld_scales % 4 != 0))
    return fail(IRIS_ERR_ALIGNMENT, "A: scales must be 4-byte aligned and ld_scales a multiple of 4");
  if (N > 0 && K > 0 && ((uintptr_t)B->scales % 4 != 0 || B->ld_scales % 4 != 0))
    return fail(IRIS_ERR_ALIGNMENT, "B: scales must be 4-byte aligned and ld_scales a multiple of 4");
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
  if (plan.ws_bytes > 0 && !workspace && (st = own_workspace(dev, stream, plan.ws_bytes, &workspace, &hold))) return st;
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
