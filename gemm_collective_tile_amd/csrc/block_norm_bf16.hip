// The block norms of bf16 activations, and the joining of the column sums.
#include <algorithm>

#include "block_norm_kernels.hpp"
#include "column_sums.hpp"

namespace iris {

template hipError_t launch_norm<bf16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<bf16>(const NormBwdArgs&, bool, bool, hipStream_t);

namespace {

constexpr int kJoinGates = 16;

struct JoinArgs {   // short: the host writes a kernel's arguments for every launch
  float *dpre_w, *dpre_b, *dpost_w, *dpost_b, *dgate;
  const float* part;
  int32_t rows, cols, rows_per_gate, wgs, wg_rows, groups;
};

// Adds the workgroups' sums, 64 columns at a time, 16 waves a sixteenth of the workgroups
// each with up to 16 loads under way. blockIdx.y: 0 to 3 the parameters' gradients; from
// 4 on the gates' whose rows several workgroups share. Bound by latency, so many loads at
// a time: four gradients of 4096 columns from 512 workgroups 6.4 us (with one load at a
// time 23.7), from 256 4.0.
__global__ __launch_bounds__(1024) void block_norm_join_kernel(JoinArgs a, FastDiv gate_rows, FastDiv wg_rows) {
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
  // by group where there are fewer groups than workgroups, else by the workgroup a group begins in
  const float* const gates = a.part + (int64_t)4 * a.wgs * pitch;
  const int64_t every = a.rows_per_gate;
  const bool by_group = a.groups < a.wgs;
  for (int k = blockIdx.y - 4; k < (by_group ? a.groups : a.wgs - 1); k += gridDim.y - 4) {
    const int64_t g = by_group ? k : gate_rows.div((k + 1) * a.wg_rows - 1);
    const int64_t g0 = g * every, g1 = min(g0 + every, (int64_t)a.rows);
    const int w = by_group ? (int)wg_rows.div((uint32_t)g0) : k, next = min((w + 1) * a.wg_rows, a.rows);
    if (g1 <= next || g0 < (int64_t)w * a.wg_rows) continue;   // ends here, or began before
    const int n = (int)wg_rows.div((uint32_t)(g1 - 1)) - w;    // further workgroups: their first share each
    join(gates + (2 * w + (g0 == (int64_t)w * a.wg_rows ? 0 : 1)) * pitch, gates + 2 * (w + 1) * pitch, n, 2 * pitch,
         a.dgate + g * a.cols);
  }
}

}  // namespace

NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols, bool whole) {
  int waves = 1;
  while (waves < 16 && 512 * waves < cols) waves *= 2;
  if (rows == 0) return {1, 0, 0};    // the parameters' gradients alone: zeros
  const int64_t step = norm_bwd_waves(waves) / waves;    // rows that a workgroup works on at a time
  NormBwdPlan p{};
  const auto share = [&](bool ahead) {   // of the rows, for as many workgroups as the chip holds
    const int64_t most = kFp8Cus * (ahead ? 1 : 16 / norm_bwd_waves(waves)), n = ((rows + most - 1) / most + step - 1) / step * step;
    p.wg_rows = (int)n;
    p.wgs = (int)((rows + n - 1) / n);
  };
  share(false);   // the larger number: the workspace's
  p.ws_bytes = p.wgs > 1 ? (size_t)6 * p.wgs * ((cols + 7) / 8 * 8) * 4 : 0;
  if (norm_bwd_ahead(waves, whole)) share(true);
  return p;
}

hipError_t launch_norm_join(const NormBwdArgs& a, hipStream_t s) {
  if (a.rows == 0 && a.dgate) return join_columns(nullptr, 0, 0, a.cols, a.dgate, s);   // zeros, as the kernel gives the others
  if (a.wgs <= 1) return hipSuccess;
  const JoinArgs j{a.dpre_w, a.dpre_b, a.dpost_w, a.dpost_b, a.dgate, a.part, a.rows, a.cols, a.p.rows_per_gate, a.wgs, a.wg_rows,
                   a.dgate ? (a.rows + a.p.rows_per_gate - 1) / a.p.rows_per_gate : 0};
  hipLaunchKernelGGL(block_norm_join_kernel, dim3((a.cols + 63) / 64, 4 + std::min(j.groups, kJoinGates)), dim3(1024), 0, s, j,
                     FastDiv::make((uint32_t)j.rows_per_gate), FastDiv::make((uint32_t)j.wg_rows));
  return hipGetLastError();
}

}  // namespace iris
