// C = A B^T + bias for block-scaled 8-bit operands.
//
// A (M x K) and B (N x K) hold their rows along the contraction, with a
// power-of-two scale for every 128 values of it; each output is rounded once,
// after bias and old value. Two ways to multiply, by C's type:
//
// 16-bit C: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 64 codes of a row at a
// time, applies both scales inside and adds to a 32-bit accumulator. Inside,
// it lines up the products of 8 neighbouring k with the largest of them and
// keeps 2^-13 of it and up (measured; sums of such groups, and what is carried
// from one instruction to the next, keep 24 bits and more). Against 64 bits
// that is 1.4e-5 of the result on normally distributed operands: a fifteenth
// of what rounding to fp16 adds, a hundredth of bf16's.
//
// fp32 C (weight gradients to be summed up) asks for more: the codes become
// bf16 values with their scales applied (v_cvt_scalef32_pk_bf16_fp8, exact)
// and v_mfma_f32_32x32x16_bf16, at half the rate, multiplies them exactly and
// sums in 32 bits (4e-8 of the result, measured).
//
// Any order of k inside an instruction's slice gives the same sum as long as
// both operands use it, and a block's scale is the same for all its slices, so
// a lane takes the 16-byte pieces that are cheapest to read.
//
// One workgroup of 4 waves takes a 128 x 128 tile, a wave 64 x 64 of it. A K
// step of 128 bytes goes through registers into LDS, rows of 128 bytes whose
// 16-byte pieces are permuted by the row.
#include "fp8.hpp"
#include "fp8_mma.hpp"

namespace iris {
namespace {

constexpr int kBK = 128;
constexpr int kTM = 128, kTN = 128;

__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row >> 1) & 7u; }

template <class OUT>
__global__ __launch_bounds__(256) void fp8_mm_kernel(Fp8MmArgs g) {
  __shared__ char lds[(kTM + kTN) * kBK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n_pn = (g.N + kTN - 1) / kTN;
  const int m0 = (int)(blockIdx.x / n_pn) * kTM, n0 = (int)(blockIdx.x % n_pn) * kTN;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int ch = tid & 7;

  f32x16 acc[2][2] = {};
  const int nk = (g.K + kBK - 1) / kBK;
  for (int t = 0; t < nk; ++t) {
    u32x4 r[8];
    const int valid = min(16, g.K - (t * kBK + 16 * ch));
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int row = tid / 8 + 32 * (n & 3);
      // rows past the end repeat the last one: their outputs are not stored
      const uint8_t* p = n < 4 ? g.A.codes + (int64_t)min(m0 + row, g.M - 1) * g.A.ld
                               : g.B.codes + (int64_t)min(n0 + row, g.N - 1) * g.B.ld;
      r[n] = u32x4{};
      if (valid > 0) r[n] = keep_bytes(ld16(p + t * kBK + 16 * ch), valid);
    }
    int sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sa[i] = g.A.scales[(int64_t)min(m0 + wm + 32 * i + (lane & 31), g.M - 1) * g.A.lds + t];
      sb[i] = g.B.scales[(int64_t)(min(n0 + wn + 32 * i + (lane & 31), g.N - 1) / g.b_block) * g.B.lds + t];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int row = tid / 8 + 32 * n;
      *(u32x4*)(lds + row * kBK + ((ch ^ swz(row)) << 4)) = r[n];
    }
    __syncthreads();
    // lane (r, h) of a 32-row block takes pieces h, 2 + h, 4 + h, 6 + h of row r
    u32x4 a[2][4], b[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t c = 2 * p + (lane >> 5);
        const uint32_t ra = wm + 32 * i + (lane & 31), rb = kTM + wn + 32 * i + (lane & 31);
        a[i][p] = *(const u32x4*)(lds + ra * kBK + ((c ^ swz(ra)) << 4));
        b[i][p] = *(const u32x4*)(lds + rb * kBK + ((c ^ swz(rb)) << 4));
      }
    if constexpr (sizeof(OUT) == 4) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        bf16x8 x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = to_bf16x8(a[i][s / 2][2 * (s & 1)], a[i][s / 2][2 * (s & 1) + 1], __builtin_bit_cast(float, sa[i] << 23));
          y[i] = to_bf16x8(b[i][s / 2][2 * (s & 1)], b[i][s / 2][2 * (s & 1) + 1], __builtin_bit_cast(float, sb[i] << 23));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[j], x[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                pair(b[j][2 * s], b[j][2 * s + 1]), pair(a[i][2 * s], a[i][2 * s + 1]), acc[i][j], 0, 0, 0, sb[j], 0, sa[i]);
    }
  }

  // B is the first operand, so a lane holds row lane % 32 of each block and,
  // for q = 0..3, its columns 8 q + 4 (lane / 32) .. + 3
  const OUT* bias = (const OUT*)g.bias;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = m0 + wm + 32 * i + (lane & 31);
    if (m >= g.M) continue;
    OUT* crow = (OUT*)g.C + (int64_t)m * g.ldc;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int n = n0 + wn + 32 * j + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (n >= g.N) continue;
        put_output(crow + n, acc[i][j][e], bias, g.bias_along_m ? m : n, g.accumulate);
      }
  }
}

}  // namespace

hipError_t launch_fp8_mm(const Fp8MmArgs& a, hipStream_t s) {
  if (a.M <= kFp8FewRows) return launch_fp8_mm_few(a, s);
  const uint32_t grid = (uint32_t)(((int64_t)a.M + kTM - 1) / kTM * (((int64_t)a.N + kTN - 1) / kTN));
  switch (a.c_type) {
    case T_FP16: hipLaunchKernelGGL((fp8_mm_kernel<f16>), dim3(grid), dim3(256), 0, s, a); break;
    case T_BF16: hipLaunchKernelGGL((fp8_mm_kernel<bf16>), dim3(grid), dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((fp8_mm_kernel<float>), dim3(grid), dim3(256), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace iris
