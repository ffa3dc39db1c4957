// C = A B^T + bias for few rows of A (serving: one token, a small batch).
//
// Bound by the bytes of B, each of which meets at most 64 rows: 45 MB for a
// 4096 x 11008 projection against 0.4 us of matrix work at one row. So B goes
// from memory straight into the registers of the lane that multiplies it, once,
// and as many of its bytes as possible are under way at a time.
//
// A workgroup of 8 waves takes 16 rows of B; its waves split the contraction,
// in units of 512 (one 32-bit word of scale bytes per row), and sum through LDS
// in a fixed order. All loads of a wave's next unit (8 KB of B) are issued
// before it multiplies the present one. v_mfma_scale_f32_16x16x128 takes row
// l % 16 from lane l, 32 of its 128 bytes: pieces l / 16 and 4 + l / 16.
#include "fp8.hpp"
#include "fp8_mma.hpp"

namespace iris {
namespace {

constexpr int kWaves = 8;
constexpr int kRows = 16;      // rows of B per workgroup, and of A per block
constexpr int kUnit = 4;       // steps of 128 per unit

struct Side {
  const uint8_t* codes;   // this lane's row, at its first piece
  const uint8_t* scales;
};

struct Unit {
  u32x4 v[kUnit][2];
  uint32_t s;             // scale bytes of the unit's steps
};

__device__ __forceinline__ void load_unit(const Side& p, int u, Unit& x) {
  const uint8_t* c = p.codes + (int64_t)u * (kUnit * kFp8Block);
  x.s = *(const uint32_t*)(p.scales + kUnit * u);
#pragma unroll
  for (int t = 0; t < kUnit; ++t) {
    x.v[t][0] = ld16(c + t * kFp8Block);
    x.v[t][1] = ld16(c + t * kFp8Block + 64);
  }
}

// the ragged end of the contraction: bytes past K are zeros, blocks past it have scale 1
__device__ __forceinline__ void load_last_unit(const Side& p, int u, int K, int piece, Unit& x) {
  const uint8_t* c = p.codes + (int64_t)u * (kUnit * kFp8Block);
  x.s = *(const uint32_t*)(p.scales + kUnit * u);
#pragma unroll
  for (int t = 0; t < kUnit; ++t) {
    const int k = (u * kUnit + t) * kFp8Block;
    if (k >= K) x.s = (x.s & ~(0xffu << (8 * t))) | (127u << (8 * t));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int valid = K - (k + 64 * h + piece);
      x.v[t][h] = u32x4{};
      if (valid > 0) x.v[t][h] = keep_bytes(ld16(c + t * kFp8Block + 64 * h), min(16, valid));
    }
  }
}

template <bool EXACT, int T>
__device__ __forceinline__ void multiply(const Unit& a, const Unit& b, f32x4& acc) {
  if constexpr (EXACT) {
    const float sa = __builtin_bit_cast(float, ((a.s >> (8 * T)) & 0xff) << 23);
    const float sb = __builtin_bit_cast(float, ((b.s >> (8 * T)) & 0xff) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x8 x = to_bf16x8(a.v[T][q / 2][2 * (q & 1)], a.v[T][q / 2][2 * (q & 1) + 1], sa);
      const bf16x8 y = to_bf16x8(b.v[T][q / 2][2 * (q & 1)], b.v[T][q / 2][2 * (q & 1) + 1], sb);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x, acc, 0, 0, 0);
    }
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pair(b.v[T][0], b.v[T][1]), pair(a.v[T][0], a.v[T][1]), acc,
                                                           0, 0, T, (int)b.s, T, (int)a.s);
  }
}

template <bool EXACT>
__device__ __forceinline__ void multiply_unit(const Unit& a, const Unit& b, f32x4& acc) {
  multiply<EXACT, 0>(a, b, acc);
  multiply<EXACT, 1>(a, b, acc);
  multiply<EXACT, 2>(a, b, acc);
  multiply<EXACT, 3>(a, b, acc);
}

template <class OUT, int MB>
__global__ __launch_bounds__(kWaves * 64) void fp8_mm_few_kernel(Fp8MmArgs g) {
  constexpr bool EXACT = sizeof(OUT) == 4;
  __shared__ f32x4 part[kWaves][MB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kRows, r = lane & 15, piece = 16 * (lane >> 4);
  // rows past the end repeat the last one: their outputs are not stored
  const int n = min(n0 + r, g.N - 1);
  const Side b{g.B.codes + (int64_t)n * g.B.ld + piece, g.B.scales + (int64_t)(n / g.b_block) * g.B.lds};
  Side a[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = min(16 * i + r, g.M - 1);
    a[i] = Side{g.A.codes + (int64_t)m * g.A.ld + piece, g.A.scales + (int64_t)m * g.A.lds};
  }
  f32x4 acc[MB] = {};
  const int nu = g.K / (kUnit * kFp8Block);
  const int u0 = (int)((int64_t)nu * wave / kWaves), u1 = (int)((int64_t)nu * (wave + 1) / kWaves);
  if (u0 < u1) {
    Unit bc, bn;
    load_unit(b, u0, bc);
    for (int u = u0; u < u1; ++u) {
      // A's before the next of B: loads return in order
      Unit au[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) load_unit(a[i], u, au[i]);
      if (u + 1 < u1) load_unit(b, u + 1, bn);
#pragma unroll
      for (int i = 0; i < MB; ++i) multiply_unit<EXACT>(au[i], bc, acc[i]);
      bc = bn;
    }
  }
  // the first wave has no more whole units than the others
  if (wave == 0 && nu * (kUnit * kFp8Block) < g.K) {
    Unit bc, ac;
    load_last_unit(b, nu, g.K, piece, bc);
    for (int i = 0; i < MB; ++i) {
      load_last_unit(a[i], nu, g.K, piece, ac);
      multiply_unit<EXACT>(ac, bc, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // B is the first operand: lane l of a block holds row l % 16, columns 4 (l / 16) .. + 3
  for (int e = threadIdx.x; e < MB * 256; e += kWaves * 64) {
    const int i = e >> 8, m = 16 * i + ((e >> 4) & 15), nn = n0 + (e & 15);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += ((const float*)&part[w][i][((e >> 4) & 15) + 16 * ((e & 15) >> 2)])[e & 3];
    if (m < g.M && nn < g.N)
      put_output((OUT*)g.C + (int64_t)m * g.ldc + nn, v, (const OUT*)g.bias, g.bias_along_m ? m : nn, g.accumulate);
  }
}

template <class OUT>
hipError_t launch(const Fp8MmArgs& a, hipStream_t s) {
  const dim3 grid((a.N + kRows - 1) / kRows), block(kWaves * 64);
  switch ((a.M + 15) / 16) {
    case 1: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 3>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 4>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_mm_few(const Fp8MmArgs& a, hipStream_t s) {
  switch (a.c_type) {
    case T_FP16: return launch<f16>(a, s);
    case T_BF16: return launch<bf16>(a, s);
    default: return launch<float>(a, s);
  }
}

}  // namespace iris
