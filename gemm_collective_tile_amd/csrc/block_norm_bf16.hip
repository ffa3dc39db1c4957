// The block norms of bf16 activations, and the joining of the column sums.
#include "block_norm_kernels.hpp"

namespace iris {

template hipError_t launch_norm<bf16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<bf16>(const NormBwdArgs&, bool, bool, hipStream_t);

namespace {

constexpr int kJoinGates = 16;

// Adds the workgroups' sums, 16 of every 64 columns at a time. blockIdx.y: 0 to 3 the
// parameters' gradients; from 4 on the gates' whose rows several workgroups share, each
// by the workgroup that has its first row.
__global__ __launch_bounds__(1024) void block_norm_join_kernel(NormBwdArgs a) {
  __shared__ float sums[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const int64_t pitch = (a.cols + 7) & ~7;
  // rows [from, to) of `first` on, every step-th
  const auto join = [&](const float* first, int n, int64_t step, float* out) {
    float v = 0.0f;
    if (c < a.cols) {
#pragma unroll 4
      for (int i = part; i < n; i += 16) v += first[i * step + c];
    }
    sums[part][threadIdx.x & 63] = v;
    __syncthreads();
    if (part == 0 && c < a.cols) {
      v = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) v += sums[i][threadIdx.x & 63];
      out[c] = v;
    }
    __syncthreads();
  };
  if (blockIdx.y < 4) {
    float* const outs[4] = {a.dpre_w, a.dpre_b, a.dpost_w, a.dpost_b};
    float* out = nullptr;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k == (int)blockIdx.y) out = outs[k];
    if (out && a.wgs > 1) join(a.part + (int64_t)blockIdx.y * a.wgs * pitch, a.wgs, pitch, out);
    return;
  }
  const int64_t every = a.p.rows_per_gate;
  for (int w = blockIdx.y - 4; w < a.wgs - 1; w += kJoinGates) {
    const int64_t next = (int64_t)(w + 1) * a.wg_rows;       // the first row of the next workgroup
    const int64_t g = (next - 1) / every, g0 = g * every, g1 = min(g0 + every, (int64_t)a.rows);
    if (g1 <= next || g0 < next - a.wg_rows) continue;       // ends here, or began before
    const int n = (int)((g1 - 1) / a.wg_rows) - w;           // further workgroups: their first share each
    const float* const own = a.part + ((int64_t)4 * a.wgs + 2 * w + (g0 == next - a.wg_rows ? 0 : 1)) * pitch;
    float v = 0.0f;
    if (c < a.cols) {
#pragma unroll 4
      for (int i = part; i < n; i += 16) v += a.part[((int64_t)4 * a.wgs + 2 * (w + 1 + i)) * pitch + c];
    }
    sums[part][threadIdx.x & 63] = v;
    __syncthreads();
    if (part == 0 && c < a.cols) {
      v = own[c];
#pragma unroll
      for (int i = 0; i < 16; ++i) v += sums[i][threadIdx.x & 63];
      a.dgate[g * a.cols + c] = v;
    }
    __syncthreads();
  }
}

}  // namespace

NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols) {
  int waves = 1;
  while (waves < 16 && 512 * waves < cols) waves *= 2;
  if (rows == 0) return {1, 0, 0};    // the parameters' gradients alone: zeros
  const int64_t step = 16 / waves;    // rows that a workgroup works on at a time
  const int64_t share = ((rows + kNormWgs - 1) / kNormWgs + step - 1) / step * step;
  NormBwdPlan p{};
  p.wg_rows = (int)share;
  p.wgs = (int)((rows + share - 1) / share);
  p.ws_bytes = p.wgs > 1 ? (size_t)6 * p.wgs * ((cols + 7) / 8 * 8) * 4 : 0;
  return p;
}

hipError_t launch_norm_join(const NormBwdArgs& a, hipStream_t s) {
  if (a.wgs <= 1) return hipSuccess;
  const dim3 grid((a.cols + 63) / 64, a.dgate ? 4 + kJoinGates : 4);
  hipLaunchKernelGGL(block_norm_join_kernel, grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace iris
