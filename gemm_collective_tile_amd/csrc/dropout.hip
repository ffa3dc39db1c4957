// out = residual + alpha m x, the mask computed on the way (dropout.hpp).
#include <algorithm>

#include "dropout.hpp"
#include "fp8.hpp"

namespace iris {
namespace {

// A thread takes 8 columns of a row: one call of the generator.
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
hipError_t of_type(const DropoutArgs& a, hipStream_t s) {
  return a.vec && a.cols % 8 == 0 ? dropout<T, true>(a, s) : dropout<T, false>(a, s);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  switch (a.type) {
    case T_FP16: return of_type<f16>(a, s);
    case T_BF16: return of_type<bf16>(a, s);
    default: return of_type<float>(a, s);
  }
}

}  // namespace iris
