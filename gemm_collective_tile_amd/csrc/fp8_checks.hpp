// Argument checks that the entry points beside iris_local.cpp's share: all of them run
// before any HIP call.
#pragma once

#include "../../include/iris_local.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <exception>
#include <mutex>

#include "fp8.hpp"

namespace iris {
// beside the other entry points
int set_error(int status, const char* msg);
int use_device(int* dev, int* cus);
// The library's own workspace of (device, stream) for work that needs `need` bytes, locked
// by `hold` until the caller has enqueued all its launches.
int fp8_own_workspace(int dev, void* stream, size_t need, void** out, std::unique_lock<std::mutex>* hold);
}  // namespace iris

namespace {

using iris::Fp8Mat;

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
[[maybe_unused]] int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return iris::set_error(status, buf);
}

[[maybe_unused]] int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return IRIS_OK;
  return fail(IRIS_ERR_HIP, "%s launch: %s (%d)", what, hipGetErrorString(e), (int)e);
}

constexpr int64_t kBlk = iris::kFp8Block;
// the kernels address a tile's rows with 32-bit offsets
constexpr int64_t kMaxPitch = 1 << 22;
[[maybe_unused]] int64_t blocks(int64_t n) { return (n + kBlk - 1) / kBlk; }

// rows and columns of a memory-bound operator: its grid numbers 128-wide
// blocks of rows (or tiles) in 31 bits
[[maybe_unused]] int check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0)
    return fail(IRIS_ERR_INVALID_ARG, "rows and cols must not be negative (got %lld, %lld)", (long long)rows,
                (long long)cols);
  if (rows > (1 << 30) || cols > (1 << 30) || (rows > 0 && blocks(cols) > (((int64_t)1 << 31) - 1) / rows))
    return fail(IRIS_ERR_UNSUPPORTED, "matrix too large (limits: rows and cols <= 2^30, rows * ceil(cols / 128) < 2^31)");
  return IRIS_OK;
}

// of the operators that work on tiles of 128 x 128, one launch for all
[[maybe_unused]] int check_tiles(int64_t rows, int64_t cols) {
  if (blocks(rows) * blocks(cols) > iris::kMaxTiles)
    return fail(IRIS_ERR_UNSUPPORTED, "matrix too large (limit: fewer than 2^23 tiles of 128 x 128)");
  return IRIS_OK;
}

[[maybe_unused]] int check_fp8(const iris_fp8_t* q, int64_t rows, int64_t cols, const char* name) {
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

[[maybe_unused]] int check_blocks1(const iris_fp8_t* q, int64_t rows, int64_t cols, const char* name) {
  const int st = check_fp8(q, rows, cols, name);
  if (st) return st;
  if (q->block != 1) return fail(IRIS_ERR_UNSUPPORTED, "%s: block must be 1 here (got %d)", name, q->block);
  return IRIS_OK;
}

[[maybe_unused]] int type_bytes(int32_t type) { return type == IRIS_TYPE_FP32 ? 4 : 2; }

[[maybe_unused]] int check_plain(const void* x, int32_t type, bool fp32_too, int64_t ld, int64_t rows, int64_t cols, const char* name) {
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

// an operand of a product: its scales are read four at a time
[[maybe_unused]] int check_scale_words(const iris_fp8_t* q, int64_t rows, int64_t K, const char* name) {
  if (rows > 0 && K > 0 && ((uintptr_t)q->scales % 4 != 0 || q->ld_scales % 4 != 0))
    return fail(IRIS_ERR_ALIGNMENT, "%s: scales must be 4-byte aligned and ld_scales a multiple of 4", name);
  return IRIS_OK;
}

// every row of a plain matrix starts at a multiple of 16 bytes
[[maybe_unused]] bool rows16(const void* x, int64_t ld, int32_t type) {
  return (uintptr_t)x % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

[[maybe_unused]] Fp8Mat mat(const iris_fp8_t* q) {
  if (!q) return Fp8Mat{};
  return Fp8Mat{(uint8_t*)q->codes, (uint8_t*)q->scales, (int32_t)q->ld, (int32_t)q->ld_scales};
}

// No exception leaves a C entry: what can throw here is memory for a message or
// for a device's record, or a lock.
[[maybe_unused]] int caught(const std::exception& e) { return iris::set_error(IRIS_ERR_NO_MEMORY, e.what()); }

[[maybe_unused]] int check_mm_dims(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0)
    return fail(IRIS_ERR_INVALID_ARG, "M, N, K must not be negative (got %lld, %lld, %lld)", (long long)M, (long long)N,
                (long long)K);
  // the largest tile, 256 x 256, has to fit one launch
  if (M > (1 << 30) || N > (1 << 30) || K > (1 << 21) || (M + 255) / 256 * ((N + 255) / 256) > iris::kMaxMmTiles)
    return fail(IRIS_ERR_UNSUPPORTED, "shape too large (limits: M, N <= 2^30, K <= 2^21, fewer than 2^24 output tiles of 256 x 256)");
  return IRIS_OK;
}

[[maybe_unused]] int ready() {
  int dev = 0, cus = 0;
  return iris::use_device(&dev, &cus);
}

}  // namespace
