// Products A B^T for few rows of A (serving: one token, a small batch).
//
// Bound by the bytes of B, each of which meets at most 96 rows: 45 MB for a
// 4096 x 11008 projection against 0.4 us of matrix work at one row. So all of B
// is under way as early as possible and is touched once.
//
// A workgroup takes 16 NB rows of B; its waves split the contraction in steps of
// 128 and sum through LDS in a fixed order. Nothing is shared in between, so
// there is no barrier: a wave loads a step's rows (16 NB of B and up to
// 16 MB of A, 128 bytes each) straight into its own piece of LDS, waits for them, and
// multiplies; other waves' loads are under way meanwhile. The detour over LDS
// is for the loads' sake: 8 neighbouring lanes read one row's 128 bytes, while
// the matrix instruction wants neighbouring lanes to hold different rows.
// v_mfma_scale_f32_16x16x128 takes row l % 16 from lane l, 32 of its 128 bytes:
// pieces l / 16 and 4 + l / 16 of 16 bytes. The pieces of a row are permuted in
// LDS by the row, so that 16 rows' same pieces lie in different banks.
//
// Beyond 16 rows of A the CU's load path (about 60 GB/s) is the limit: every
// workgroup reads all of A again. NB = 2 or 3 share that reading among more rows of
// B, if the CUs stay occupied (fp8_few_blocks). 11008 x 4096 in bf16: 33 rows 10.7
// us against 17.2 with NB = 1, 64 rows 12.7 against 23.3, 17 rows 9.7 against 13.0.
// At one row it is B's bytes: 11008 x 4096 in 8.4 us out of the last-level cache (5.3
// TB/s with the launch; 6.6 TB/s between 16 and 45 MB), 10.0 out of HBM (ten such
// matrices in turn, 4.5 TB/s). Two steps under way per wave gained nothing there and
// cost a tenth at 33 rows. NB = 4 gained 8 % at 64 rows of 32000 x 4096 and took
// more than the register file with 32-bit sums kept in two parts.
#pragma once

#include <algorithm>

#include "fp8.hpp"
#include "fp8_mma.hpp"

namespace iris {
namespace {

constexpr int kRows = 16;      // of a block of A or B
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

// The contraction is cut in SHARES, which NW waves work on and whose sums are
// added in pairs, if there are 16, and then in order, whatever NW is: a
// column's result does not depend on how many columns there are (NB).
// END takes each output (m, n) from its sum.
template <class END, bool EXACT, int MB, int NB, int NW, int SHARES>
__global__ __launch_bounds__(NW * 64) void fp8_mm_few_kernel(Fp8MmArgs g, END end) {
  constexpr int kPerWave = SHARES / NW, kAtOnce = SHARES == 16 && NW == 16 ? 2 : 1;
  static_assert(kPerWave * NW == SHARES && (SHARES == 8 || SHARES == 16) && (NW == 8 || NW == 16), "pairs of shares");
  constexpr int kWaveBytes = (NB + MB) * kBlockBytes;
  // the rows' memory, reused by the waves' sums
  __shared__ __align__(16) char lds[NW * std::max(kWaveBytes, MB * NB * 64 * (int)sizeof(f32x4))];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * (NB * kRows), r = lane & 15;
  char* const own = lds + wave * kWaveBytes;

  // rows of B past the end repeat the last one, rows of A past it are not
  // fetched: their outputs are not stored
  int n[NB];
  const uint8_t* bs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    n[j] = min(n0 + kRows * j + r, g.N - 1);
    bs[j] = g.B.scales + (int64_t)(n[j] / g.b_block) * g.B.lds;
  }
  f32x4 acc[MB][NB] = {}, sum[MB][NB] = {};
  const int nk = g.K / kFp8Block;
  // the first share has no more whole steps than the others: it takes the ragged one
  if (wave == 0 && nk * kFp8Block < g.K) {
    Operand y[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) y[j] = last_operand(g.B.codes + (int64_t)n[j] * g.B.ld, nk * kFp8Block, g.K, lane);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = min(kRows * i + r, g.M - 1);
      const Operand x = last_operand(g.A.codes + m * g.A.ld, nk * kFp8Block, g.K, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j) multiply<EXACT>(x, y[j], g.A.scales[m * g.A.lds + nk], bs[j][nk], acc[i][j]);
    }
  }
  for (int share = wave * kPerWave; share < (wave + 1) * kPerWave; ++share) {
    const int k0 = (int)((int64_t)nk * share / SHARES), k1 = (int)((int64_t)nk * (share + 1) / SHARES);
    uint32_t sb[NB], sa[MB];
    for (int k = k0; k < k1; ++k) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
        Rows16(g.B, n0 + kRows * j, g.N, lane, true).fetch(k * kFp8Block, own + j * kBlockBytes);
#pragma unroll
      for (int i = 0; i < MB; ++i)
        Rows16(g.A, kRows * i, g.M, lane, false).fetch(k * kFp8Block, own + (NB + i) * kBlockBytes);
      if (k == k0 || (k & 3) == 0) {
        // four steps' scale bytes
#pragma unroll
        for (int j = 0; j < NB; ++j) sb[j] = *(const uint32_t*)(bs[j] + (k & ~3)) >> (8 * (k & 3));
#pragma unroll
        for (int i = 0; i < MB; ++i)
          sa[i] = *(const uint32_t*)(g.A.scales + (int64_t)min(kRows * i + r, g.M - 1) * g.A.lds + (k & ~3)) >> (8 * (k & 3));
      }
      wait_loads<0>();
      Operand x[MB], y[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) y[j] = read_operand(own + j * kBlockBytes, lane);
#pragma unroll
      for (int i = 0; i < MB; ++i) x[i] = read_operand(own + (NB + i) * kBlockBytes, lane);
      wait_lds();   // before the next step's loads overwrite them
#pragma unroll
      for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int j = 0; j < NB; ++j) multiply<EXACT>(x[i], y[j], sa[i], sb[j], acc[i][j]);
        sa[i] >>= 8;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) sb[j] >>= 8;
    }
    if constexpr (kPerWave > 1)
#pragma unroll
      for (int ij = 0; ij < MB * NB; ++ij) sum[ij / NB][ij % NB] += acc[ij / NB][ij % NB], acc[ij / NB][ij % NB] = f32x4{};
  }
  __syncthreads();
  f32x4(*const part)[MB * NB][64] = (f32x4(*)[MB * NB][64])lds;
#pragma unroll
  for (int ij = 0; ij < MB * NB; ++ij)
    part[wave][ij][lane] = kPerWave > 1 ? sum[ij / NB][ij % NB] : acc[ij / NB][ij % NB];
  __syncthreads();
  // B is the first operand: lane l of a block holds row l % 16, columns 4 (l / 16) .. + 3
  for (int e = threadIdx.x; e < MB * NB * 256; e += NW * 64) {
    const int ij = e >> 8, m = kRows * (ij / NB) + ((e >> 4) & 15), nn = n0 + kRows * (ij % NB) + (e & 15);
    const auto of = [&](int w) { return ((const float*)&part[w][ij][((e >> 4) & 15) + 16 * ((e & 15) >> 2)])[e & 3]; };
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w += kAtOnce) v += kAtOnce == 2 ? of(w) + of(w + 1) : of(w);
    if (m < g.M && nn < g.N) end.put(g, m, nn, v);
  }
}

template <class END, bool EXACT, int MB, int NB, int NW, int SHARES>
void launch_few_one(const Fp8MmArgs& a, const END& end, hipStream_t s) {
  const dim3 grid((a.N + NB * kRows - 1) / (NB * kRows));
  hipLaunchKernelGGL((fp8_mm_few_kernel<END, EXACT, MB, NB, NW, SHARES>), grid, dim3(NW * 64), 0, s, a, end);
}

template <class END, bool EXACT, int MB>
void launch_few_wide(const Fp8MmArgs& a, const END& end, hipStream_t s) {
  switch (fp8_few_blocks(a.M, a.N)) {
    case 1: launch_few_one<END, EXACT, MB, 1, MB <= 4 ? 16 : 8, MB <= 4 ? 16 : 8>(a, end, s); break;
    case 2: launch_few_one<END, EXACT, MB, 2, 8, MB <= 4 ? 16 : 8>(a, end, s); break;
    default: launch_few_one<END, EXACT, MB, 3, 8, MB <= 4 ? 16 : 8>(a, end, s); break;
  }
}

template <class END, bool EXACT>
hipError_t launch_few(const Fp8MmArgs& a, const END& end, hipStream_t s) {
  switch ((a.M + kRows - 1) / kRows) {
    case 1: launch_few_one<END, EXACT, 1, 1, 8, 8>(a, end, s); break;
    case 2: launch_few_wide<END, EXACT, 2>(a, end, s); break;
    case 3: launch_few_wide<END, EXACT, 3>(a, end, s); break;
    case 4: launch_few_wide<END, EXACT, 4>(a, end, s); break;
    default: launch_few_wide<END, EXACT, 6>(a, end, s); break;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace iris
