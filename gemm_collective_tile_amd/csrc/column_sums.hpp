// Sums over the rows of a matrix, for gradients of biases: the last steps. Workgroups leave
// partial sums, a row for every share of the matrix's rows, and these are added in order:
// no atomics, the same bits every time.
#pragma once

#include "fp8_common.hpp"

namespace iris {
namespace {

// the sum over the lanes that hold the same columns, `lanes` of them side by side to a row
template <int LANES>
__device__ __forceinline__ float same_columns_sum(float v) {
  static_assert(LANES == 8 || LANES == 16, "");
  if constexpr (LANES == 8) v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
  const uint32_t t = __builtin_bit_cast(uint32_t, v);
  const auto y = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  return __builtin_bit_cast(float, (uint32_t)y[0]) + __builtin_bit_cast(float, (uint32_t)y[1]);
}

// out = the partial sums, added in order: a wave a quarter of them, 16 loads under way.
// Bound by latency: 16 rows of 11008 4.1 us.
template <class OUT>
__global__ __launch_bounds__(256) void join_columns_kernel(const float* part, int parts, int64_t ldp, int N, OUT* out) {
  __shared__ float red[4][64];
  const int l = threadIdx.x & 63, c = blockIdx.x * 64 + l, g = threadIdx.x >> 6;
  float v = 0.0f;
  for (int i = g; i < parts; i += 64) {
    float x[16];   // a row past the end reads the last one and drops it: no branch between the loads
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = part[min(i + 4 * k, parts - 1) * ldp + min(c, N - 1)];
#pragma unroll
    for (int k = 0; k < 16; ++k) v += i + 4 * k < parts ? x[k] : 0.0f;
  }
  red[g][l] = v;
  __syncthreads();
  if (g == 0 && c < N) narrow((red[0][l] + red[1][l]) + (red[2][l] + red[3][l]), out[c]);
}

template <class OUT>
hipError_t join_columns(const float* part, int parts, int64_t ldp, int N, OUT* out, hipStream_t s) {
  hipLaunchKernelGGL((join_columns_kernel<OUT>), dim3((N + 63) / 64), dim3(256), 0, s, part, parts, ldp, N, out);
  return hipGetLastError();
}

}  // namespace
}  // namespace iris
