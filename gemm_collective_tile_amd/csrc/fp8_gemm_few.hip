// C = A B^T + bias for few rows of A (serving: one token, a small batch).
//
// Bound by the bytes of B, each of which meets at most 64 rows: 45 MB for a
// 4096 x 11008 projection against 0.4 us of matrix work at one row. So all of B
// is under way as early as possible and is touched once.
//
// A workgroup takes 16 rows of B; its waves split the contraction in steps of
// 128 and sum through LDS in a fixed order. Nothing is shared in between, so
// there is no barrier: a wave loads a step's rows (16 of B and up to 16 MB of
// A, 128 bytes each) straight into its own piece of LDS, waits for them, and
// multiplies; other waves' loads are under way meanwhile. The detour over LDS
// is for the loads' sake: 8 neighbouring lanes read one row's 128 bytes, while
// the matrix instruction wants neighbouring lanes to hold different rows.
// v_mfma_scale_f32_16x16x128 takes row l % 16 from lane l, 32 of its 128 bytes:
// pieces l / 16 and 4 + l / 16 of 16 bytes. The pieces of a row are permuted in
// LDS by the row, so that 16 rows' same pieces lie in different banks.
#include "fp8.hpp"
#include "fp8_mma.hpp"

namespace iris {
namespace {

constexpr int kRows = 16;      // rows of B per workgroup, and of A per block
constexpr int kBlockBytes = kRows * kFp8Block;

// one wave's copy of 16 rows x 128 bytes: rows that lanes l and l + 64 fetch
struct Rows16 {
  const uint8_t* lo;   // this lane's piece of row lane / 8
  const uint8_t* hi;   // of row 8 + lane / 8
  bool lo_on, hi_on;
  __device__ __forceinline__ Rows16(const Fp8Mat& x, int first, int rows, int lane, bool clamp) {
    const int r = lane >> 3;
    const int a = first + r, b = a + 8;
    lo_on = clamp || a < rows;
    hi_on = clamp || b < rows;
    lo = x.codes + (int64_t)min(a, rows - 1) * x.ld + 16 * ((lane & 7) ^ (r >> 1));
    hi = x.codes + (int64_t)min(b, rows - 1) * x.ld + 16 * ((lane & 7) ^ (4 + (r >> 1)));
  }
  __device__ __forceinline__ void fetch(int k, char* lds) const {
    if (lo_on) load_to_lds(lo + k, lds);
    if (hi_on) load_to_lds(hi + k, lds + 1024);
  }
};

// a lane's operand of one step: two pieces of its row
struct Operand {
  u32x4 v[2];
};
__device__ __forceinline__ Operand read_operand(const char* lds, int lane) {
  const int r = lane & 15, g = lane >> 4;
  Operand o;
  o.v[0] = *(const u32x4*)(lds + r * kFp8Block + ((g ^ (r >> 1)) << 4));
  o.v[1] = *(const u32x4*)(lds + r * kFp8Block + (((4 + g) ^ (r >> 1)) << 4));
  return o;
}

template <bool EXACT>
__device__ __forceinline__ void multiply(const Operand& a, const Operand& b, uint32_t sa, uint32_t sb, f32x4& acc) {
  if constexpr (EXACT) {
    const float fa = __builtin_bit_cast(float, (sa & 0xff) << 23), fb = __builtin_bit_cast(float, (sb & 0xff) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x8 x = to_bf16x8(a.v[q / 2][2 * (q & 1)], a.v[q / 2][2 * (q & 1) + 1], fa);
      const bf16x8 y = to_bf16x8(b.v[q / 2][2 * (q & 1)], b.v[q / 2][2 * (q & 1) + 1], fb);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x, acc, 0, 0, 0);
    }
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pair(b.v[0], b.v[1]), pair(a.v[0], a.v[1]), acc, 0, 0, 0,
                                                           (int)sb, 0, (int)sa);
  }
}

// the ragged last step of the contraction: bytes past K are zeros
__device__ __forceinline__ Operand last_operand(const uint8_t* row, int k, int K, int lane) {
  Operand o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = k + 64 * h + 16 * (lane >> 4), valid = K - at;
    o.v[h] = u32x4{};
    if (valid > 0) o.v[h] = keep_bytes(ld16(row + at), min(16, valid));
  }
  return o;
}

template <class OUT, int MB, int NW>
__global__ __launch_bounds__(NW * 64) void fp8_mm_few_kernel(Fp8MmArgs g) {
  constexpr bool EXACT = sizeof(OUT) == 4;
  __shared__ __align__(16) char lds[NW * (1 + MB) * kBlockBytes];
  static_assert(sizeof(lds) >= NW * MB * 64 * 16, "the partial sums reuse the rows' memory");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kRows, r = lane & 15;
  char* const own = lds + wave * (1 + MB) * kBlockBytes;

  // rows of B past the end repeat the last one, rows of A past it are not
  // fetched: their outputs are not stored
  const Rows16 b(g.B, n0, g.N, lane, true);
  const int n = min(n0 + r, g.N - 1);
  const uint8_t* const bs = g.B.scales + (int64_t)(n / g.b_block) * g.B.lds;
  f32x4 acc[MB] = {};
  const int nk = g.K / kFp8Block;
  const int k0 = (int)((int64_t)nk * wave / NW), k1 = (int)((int64_t)nk * (wave + 1) / NW);
  uint32_t sb = 0, sa[MB];
  for (int k = k0; k < k1; ++k) {
    b.fetch(k * kFp8Block, own);
#pragma unroll
    for (int i = 0; i < MB; ++i)
      Rows16(g.A, 16 * i, g.M, lane, false).fetch(k * kFp8Block, own + (1 + i) * kBlockBytes);
    if (k == k0 || (k & 3) == 0) {
      // four steps' scale bytes
      sb = *(const uint32_t*)(bs + (k & ~3)) >> (8 * (k & 3));
#pragma unroll
      for (int i = 0; i < MB; ++i)
        sa[i] = *(const uint32_t*)(g.A.scales + (int64_t)min(16 * i + r, g.M - 1) * g.A.lds + (k & ~3)) >> (8 * (k & 3));
    }
    wait_loads<0>();
    const Operand y = read_operand(own, lane);
    Operand x[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) x[i] = read_operand(own + (1 + i) * kBlockBytes, lane);
    wait_lds();   // before the next step's loads overwrite them
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      multiply<EXACT>(x[i], y, sa[i], sb, acc[i]);
      sa[i] >>= 8;
    }
    sb >>= 8;
  }
  // the first wave has no more whole steps than the others
  if (wave == 0 && nk * kFp8Block < g.K) {
    const Operand y = last_operand(g.B.codes + (int64_t)n * g.B.ld, nk * kFp8Block, g.K, lane);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = min(16 * i + r, g.M - 1);
      const Operand x = last_operand(g.A.codes + m * g.A.ld, nk * kFp8Block, g.K, lane);
      multiply<EXACT>(x, y, g.A.scales[m * g.A.lds + nk], bs[nk], acc[i]);
    }
  }
  __syncthreads();
  f32x4(*const part)[MB][64] = (f32x4(*)[MB][64])lds;
#pragma unroll
  for (int i = 0; i < MB; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // B is the first operand: lane l of a block holds row l % 16, columns 4 (l / 16) .. + 3
  for (int e = threadIdx.x; e < MB * 256; e += NW * 64) {
    const int i = e >> 8, m = 16 * i + ((e >> 4) & 15), nn = n0 + (e & 15);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += ((const float*)&part[w][i][((e >> 4) & 15) + 16 * ((e & 15) >> 2)])[e & 3];
    if (m < g.M && nn < g.N)
      put_output((OUT*)g.C + (int64_t)m * g.ldc + nn, v, (const OUT*)g.bias, g.bias_along_m ? m : nn, g.accumulate);
  }
}

template <class OUT>
hipError_t launch(const Fp8MmArgs& a, hipStream_t s) {
  const dim3 grid((a.N + kRows - 1) / kRows);
  switch ((a.M + 15) / 16) {
    case 1: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 1, 8>), grid, dim3(512), 0, s, a); break;
    case 2: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 2, 16>), grid, dim3(1024), 0, s, a); break;
    case 3: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 3, 16>), grid, dim3(1024), 0, s, a); break;
    default: hipLaunchKernelGGL((fp8_mm_few_kernel<OUT, 4, 16>), grid, dim3(1024), 0, s, a); break;
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
