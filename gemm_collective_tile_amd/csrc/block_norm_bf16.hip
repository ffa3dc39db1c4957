// The block norms of bf16 activations, and the joining of the column sums.
#include "block_norm_kernels.hpp"

namespace iris {

template hipError_t launch_norm<bf16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<bf16>(const NormBwdArgs&, bool, bool, hipStream_t);

namespace {

constexpr int kJoinGates = 16;

// Adds the workgroups' sums, 64 columns at a time, 16 waves a sixteenth of the workgroups
// each with up to 16 loads under way. blockIdx.y: 0 to 3 the parameters' gradients; from
// 4 on the gates' whose rows several workgroups share, each by the workgroup that has
// its first row.
__global__ __launch_bounds__(1024) void block_norm_join_kernel(NormBwdArgs a, FastDiv gate_rows) {
  __shared__ float sums[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const int64_t pitch = (a.cols + 7) & ~7;
  // out = own + rows 0 .. n - 1 of `first` on, each step floats after the one before
  const auto join = [&](const float* own, const float* first, int n, int64_t step, float* out) {
    const int cc = min(c, a.cols - 1);
    const float before = own ? own[cc] : 0.0f;
    float v = 0.0f;
    for (int i = part; i < n; i += 256) {
      float x[16];   // a row past the end reads the last one and drops it: no branch between the loads
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = first[min(i + 16 * k, n - 1) * step + cc];
#pragma unroll
      for (int k = 0; k < 16; ++k) v += i + 16 * k < n ? x[k] : 0.0f;
    }
    sums[part][threadIdx.x & 63] = v;
    __syncthreads();
    if (part == 0 && c < a.cols) {
      v = before;
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
    if (out) join(nullptr, a.part + (int64_t)blockIdx.y * a.wgs * pitch, a.wgs, pitch, out);
    return;
  }
  const float* const gates = a.part + (int64_t)4 * a.wgs * pitch;
  for (int w = blockIdx.y - 4; w < a.wgs - 1; w += kJoinGates) {
    const int next = (w + 1) * a.wg_rows;                    // the first row of the next workgroup
    const uint32_t g = gate_rows.div(next - 1);
    const int64_t g0 = (int64_t)g * a.p.rows_per_gate;
    const int g1 = (int)min(g0 + a.p.rows_per_gate, (int64_t)a.rows);
    if (g1 > next && g0 >= next - a.wg_rows) {               // goes on there, and begins here
      const int n = (g1 - 1) / a.wg_rows - w;                // further workgroups: their first share each
      join(gates + (2 * w + (g0 == next - a.wg_rows ? 0 : 1)) * pitch, gates + 2 * (w + 1) * pitch, n, 2 * pitch,
           a.dgate + (int64_t)g * a.cols);
    }
    if (a.p.rows_per_gate >= a.rows) break;                  // one gate: the first workgroup's
  }
}

}  // namespace

NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols) {
  int waves = 1;
  while (waves < 16 && 512 * waves < cols) waves *= 2;
  if (rows == 0) return {1, 0, 0};    // the parameters' gradients alone: zeros
  const int64_t step = norm_bwd_waves(waves) / waves;    // rows that a workgroup works on at a time
  const int64_t most = kFp8Cus * (16 / norm_bwd_waves(waves));
  const int64_t share = ((rows + most - 1) / most + step - 1) / step * step;
  NormBwdPlan p{};
  p.wg_rows = (int)share;
  p.wgs = (int)((rows + share - 1) / share);
  p.ws_bytes = p.wgs > 1 ? (size_t)6 * p.wgs * ((cols + 7) / 8 * 8) * 4 : 0;
  return p;
}

hipError_t launch_norm_join(const NormBwdArgs& a, hipStream_t s) {
  if (a.wgs <= 1) return hipSuccess;
  const int gates = !a.dgate ? 0 : a.p.rows_per_gate >= a.rows ? 1 : kJoinGates;
  hipLaunchKernelGGL(block_norm_join_kernel, dim3((a.cols + 63) / 64, 4 + gates), dim3(1024), 0, s, a,
                     FastDiv::make((uint32_t)a.p.rows_per_gate));
  return hipGetLastError();
}

}  // namespace iris
