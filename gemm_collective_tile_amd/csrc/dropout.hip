// out = residual + alpha m x, the mask computed on the way (dropout.hpp).
#include <algorithm>

#include "column_sums.hpp"
#include "dropout.hpp"
#include "fp8.hpp"

namespace iris {
namespace {

// A thread takes 8 columns of a row: one call of the generator (10 rounds of two 32-bit
// products, some 70 instructions), 16 bytes a load. Bound by memory: 8192 x 11008 in
// bf16 with a residual, 541 MB, 91 us (5.9 TB/s, part of it the cache's; a plain copy
// of 1 GiB reaches 5.2); 1001 x 1376 in fp16 2.9 us, of which 2.2 are the launch's.
template <class T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a, FastDiv pieces) {
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x, row = pieces.div(id);
  if ((int)row >= a.rows) return;
  const int col = 8 * (int)(id - row * pieces.d);
  float v[8], r[8];
  load8<WHOLE>((const T*)a.x + (int64_t)row * a.ldx, col, a.cols, v);
  if (a.residual) load8<WHOLE>((const T*)a.residual + (int64_t)row * a.ldr, col, a.cols, r);
  Drop(a.drop).apply(a.first_row + row, (uint32_t)col >> 3, v);
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  store8<WHOLE>((T*)a.out + (int64_t)row * a.ldo, col, a.cols, v);
}

// The same with the sums of out over its rows, before its rounding: a workgroup takes 128
// columns of a share of the rows, 16 rows at a time, and leaves a row of partial sums
// (no atomics: the order of the sums is always the same), which join_columns adds.
template <class T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void dropout_sums_kernel(DropoutArgs a, int share, float* part, int64_t ldp) {
  __shared__ float red[4][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 128 + 8 * (lane & 15), from = blockIdx.y * share, to = min(from + share, a.rows);
  const Drop drop(a.drop);
  float sums[8] = {};
  for (int base = from; base < to; base += 16) {
    const int at = base + (threadIdx.x >> 4), row = min(at, to - 1);
    const bool on = at < to;
    float v[8], r[8];
    load8<WHOLE>((const T*)a.x + (int64_t)row * a.ldx, col, a.cols, v);
    if (a.residual) load8<WHOLE>((const T*)a.residual + (int64_t)row * a.ldr, col, a.cols, r);
    drop.apply((uint32_t)row, (uint32_t)col >> 3, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.residual) v[i] += r[i];
      sums[i] += on ? v[i] : 0.0f;
    }
    if (on) store8<WHOLE>((T*)a.out + (int64_t)row * a.ldo, col, a.cols, v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[i] = same_columns_sum<16>(sums[i]);
  if (lane < 16) __builtin_memcpy(&red[wave][8 * lane], sums, sizeof sums);
  __syncthreads();
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && c < a.cols) {
    const int t = threadIdx.x;
    part[(int64_t)blockIdx.y * ldp + c] = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
  }
}

template <class T, bool WHOLE>
hipError_t dropout_sums(const DropoutArgs& a, const DropoutPlan& plan, void* sums, void* ws, hipStream_t s) {
  if (a.rows > 0) {
    hipLaunchKernelGGL((dropout_sums_kernel<T, WHOLE>), dim3((a.cols + 127) / 128, plan.parts), dim3(kThreads), 0, s, a, plan.share,
                       (float*)ws, (int64_t)plan.pitch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return join_columns((const float*)ws, plan.parts, (int64_t)plan.pitch, a.cols, (T*)sums, s);
}

template <class T, bool WHOLE>
hipError_t dropout(const DropoutArgs& args, hipStream_t s) {
  const uint32_t pieces = (uint32_t)((args.cols + 7) / 8);
  const FastDiv d = FastDiv::make(pieces);
  // rows of a launch: its threads are counted in 32 bits
  const int part = (int)std::min<int64_t>(((int64_t)1 << 31) / pieces, 1 << 30);
  for (int r = 0; r < args.rows;) {
    DropoutArgs a = args;
    a.rows = std::min(part, args.rows - r);
    a.first_row = (uint32_t)r;
    a.x = (const T*)args.x + (int64_t)r * a.ldx;
    if (a.residual) a.residual = (const T*)args.residual + (int64_t)r * a.ldr;
    a.out = (T*)args.out + (int64_t)r * a.ldo;
    const uint32_t grid = (uint32_t)(((uint64_t)a.rows * pieces + kThreads - 1) / kThreads);
    hipLaunchKernelGGL((dropout_kernel<T, WHOLE>), dim3(grid), dim3(kThreads), 0, s, a, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    r += a.rows;
  }
  return hipSuccess;
}

template <class T>
hipError_t of_type(const DropoutArgs& a, const DropoutPlan& plan, void* sums, void* ws, hipStream_t s) {
  const bool whole = a.vec && a.cols % 8 == 0;
  if (sums) return whole ? dropout_sums<T, true>(a, plan, sums, ws, s) : dropout_sums<T, false>(a, plan, sums, ws, s);
  return whole ? dropout<T, true>(a, s) : dropout<T, false>(a, s);
}

}  // namespace

// Workgroups for eight a compute unit, shares of whole steps of 16 rows: fewer leave loads that
// are not under way, more leave more partial sums to write and join. bf16 without a residual,
// with 2, 4, 8 and 16 a unit: 8192 x 11008 119, 78.3, 77.9 and 75.4 us; 8192 x 4096 30.4, 26.2,
// 25.7 and 26.6; 4096 x 4096 18.5, 16.4, 15.2 and 16.5; 32768 x 512 19.4, 18.5, 19.9 and 25.4. Small
// calls (333 x 1376) take the host's 8.5 to 9.7 us with any.
DropoutPlan dropout_plan(int64_t rows, int64_t cols) {
  const int64_t blocks = (cols + 127) / 128, most = std::max<int64_t>(1, 8 * kFp8Cus / blocks);
  DropoutPlan p{};
  p.share = (int32_t)(((rows + most - 1) / most + 15) / 16 * 16);
  p.parts = rows > 0 ? (int32_t)((rows + p.share - 1) / p.share) : 0;
  p.pitch = (int32_t)((cols + 3) / 4 * 4);
  p.ws_bytes = (size_t)p.parts * p.pitch * 4;
  return p;
}

hipError_t launch_dropout(const DropoutArgs& a, const DropoutPlan& plan, void* sums, void* ws, hipStream_t s) {
  switch (a.type) {
    case T_FP16: return of_type<f16>(a, plan, sums, ws, s);
    case T_BF16: return of_type<bf16>(a, plan, sums, ws, s);
    default: return of_type<float>(a, plan, sums, ws, s);
  }
}

}  // namespace iris
