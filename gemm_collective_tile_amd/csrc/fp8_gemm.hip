// C = A B^T + bias for block-scaled 8-bit operands: the plain product, and which tile
// and split a product takes. How a tile is multiplied is in fp8_gemm_tile.hpp.
#include <algorithm>

#include "fp8_gemm_tile.hpp"

namespace iris {
namespace {

// One tile of C, or, with g.splits > 1, of one split's sum over its share of k
// (OUT is float then, C a workspace of g.splits matrices).
template <class OUT, bool EXACT, int BM, int BN>
__global__ __launch_bounds__(256) void fp8_mm_kernel(Fp8MmArgs g) {
  using T = Tile<BM, BN>;
  __shared__ __align__(16) char lds[T::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int pm, pn;
  if (!pick_tile<OUT, T>(g, pm, pn)) return;
  const int m0 = pm * BM, n0 = pn * BN;
  const int wm = (wave >> 1) * T::WM, wn = (wave & 1) * T::WN;
  const int r32 = lane & 31;
  // the tile's bias: a value per thread, parked until the end
  float bias_v = 0.0f;
  f32x16 acc[T::FM][T::FN];
  tile_sums<EXACT, T>(g, lds, pm, pn, acc, [&] {
    if (g.bias) {
      const int e = tid + (g.bias_along_m ? m0 : n0);
      if (tid < (g.bias_along_m ? BM : BN) && e < (g.bias_along_m ? g.M : g.N)) bias_v = widen(((const OUT*)g.bias)[e]);
    }
  });

  // Epilogue, 32 rows of a wave at a time: the accumulators turn around in LDS
  // (B is the first operand, so a lane holds row lane % 32 of each block and, for
  // q = 0..3, its columns 8 q + 4 (lane / 32) .. + 3) and leave in whole lines,
  // with the bias and the old values added before the one rounding.
  constexpr int V = 16 / (int)sizeof(OUT);            // columns a lane writes at once
  constexpr int PITCH = T::WN + 4;                    // floats; keeps rows on different banks
  constexpr int RPI = 64 * V / T::WN;                 // rows a wave writes at once
  static_assert(4 * 32 * PITCH * 4 + 1024 <= T::LDS, "the turn does not fit");
  float* const bl = (float*)lds;
  float* const strip = (float*)(lds + 1024) + wave * 32 * PITCH;
  bl[tid] = bias_v;
  __syncthreads();
  const int c = V * (lane % (T::WN / V)), n = n0 + wn + c;
  float bn[V];
#pragma unroll
  for (int e = 0; e < V; ++e) bn[e] = g.bias_along_m ? 0.0f : bl[wn + c + e];
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(strip + r32 * PITCH + 32 * j + 8 * q + 4 * (lane >> 5)) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
    wait_lds();
#pragma unroll 2
    for (int r = 0; r < 32; r += RPI) {
      const int row = r + lane / (T::WN / V), tm = wm + 32 * i + row, m = m0 + tm;
      float v[V];
      __builtin_memcpy(v, strip + row * PITCH + c, sizeof v);
      if (m < g.M && n < g.N) put_row_piece((OUT*)g.C + (int64_t)m * g.ldc + n, g.N - n, g.accumulate,
                                            g.bias_along_m ? bl[tm] : 0.0f, bn, v);
    }
    wait_lds();
    __builtin_amdgcn_wave_barrier();
  }
}

// C = the sum of the splits' matrices, in order, + bias (+ C)
template <class OUT>
__global__ __launch_bounds__(256) void fp8_mm_join_kernel(Fp8MmArgs g, const float* part, int64_t ldp, FastDiv pieces) {
  constexpr int V = 4;
  const uint32_t id = blockIdx.x * 256 + threadIdx.x, m = pieces.div(id);
  const int n = V * (int)(id - m * pieces.d);
  if ((int)m >= g.M) return;
  const float* p = part + (int64_t)m * ldp + n;
  float v[V] = {}, bn[V];
#pragma unroll 4
  for (int s = 0; s < g.splits; ++s) {
    const f32x4 x = *(const f32x4*)(p + (int64_t)s * g.M * ldp);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += x[e];
  }
  const OUT* const bias = (const OUT*)g.bias;
#pragma unroll
  for (int e = 0; e < V; ++e) bn[e] = bias && !g.bias_along_m && n + e < g.N ? widen(bias[n + e]) : 0.0f;
  put_row_piece((OUT*)g.C + (int64_t)m * g.ldc + n, g.N - n, g.accumulate,
                bias && g.bias_along_m ? widen(bias[m]) : 0.0f, bn, v);
}

template <class OUT, bool EXACT, int BM, int BN>
hipError_t launch(const Fp8MmArgs& a, hipStream_t s) {
  const int64_t tiles = ((int64_t)a.M + BM - 1) / BM * (((int64_t)a.N + BN - 1) / BN) * a.splits;
  const int64_t round = kPatch * kXcds;
  const uint32_t grid = (uint32_t)((tiles + round - 1) / round * round);
  hipLaunchKernelGGL((fp8_mm_kernel<OUT, EXACT, BM, BN>), dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class OUT, bool EXACT>
hipError_t small_tile(const Fp8MmArgs& a, const Fp8MmPlan& plan, hipStream_t s) {
  return plan.bn == 128   ? launch<OUT, EXACT, 128, 128>(a, s)
         : plan.bm == 128 ? launch<OUT, EXACT, 128, 64>(a, s)
                          : launch<OUT, EXACT, 64, 64>(a, s);
}

template <class OUT>
hipError_t run(const Fp8MmArgs& a, const Fp8MmPlan& plan, void* ws, hipStream_t s) {
  constexpr bool EXACT = sizeof(OUT) == 4;
  Fp8MmArgs g = a;
  g.splits = plan.splits;
  g.split_steps = plan.split_steps;
  if (plan.splits == 1)
    return plan.bm == 256 ? launch<OUT, EXACT, 256, 256>(g, s) : small_tile<OUT, EXACT>(g, plan, s);
  const hipError_t e = launch_fp8_mm_splits(a, plan, EXACT, ws, s);
  if (e != hipSuccess) return e;
  const int64_t ldp = fp8_sums_pitch(a.N);
  const uint32_t pieces = (uint32_t)(ldp / 4);
  const uint32_t grid = (uint32_t)(((int64_t)a.M * pieces + 255) / 256);
  hipLaunchKernelGGL((fp8_mm_join_kernel<OUT>), dim3(grid), dim3(256), 0, s, g, (const float*)ws, ldp,
                     FastDiv::make(pieces));
  return hipGetLastError();
}

}  // namespace

// The plan with the least predicted time, in us, from times measured on MI355X: a
// step of k on a tile that has a CU to itself, with 2 and with 4 (64 x 64 only, by
// their LDS) on each CU, and a workgroup's start and epilogue. Workgroups beyond
// what the chip holds make further rounds; the last, partial one starts as CUs
// fall free, so half its ends are hidden. Between 1 and 2 (2 and 4) a CU a step's
// time rises at once by 0.4 of the way, then evenly. Splitting the contraction
// costs a launch (2.5) and each split's sums written and read (5 TB/s at these sizes,
// in the last-level cache). What it decides, kernel times, bf16 unless named:
//                              256     128 x 128   128 x 64   64 x 64
//   128 x 1024 x 1024          18.0        8.2        6.6       5.7
//   2048 x 1024 x 4096         54.8       27.1       22.4      21.2
//   2176 x 2048 x 4096         55.2       35.6       44.8      45.8
//   2048 x 4096 x 2048         36.6       23.5       29.2      33.3
//   2176 x 4096 x 2048 fp32    63.5       50.3       52.4      52.7
//   4096 x 2048 x 4096         61.9       40.9       53.3      59.4
//   5328 x 5536 x 416          35.9       36.9       47.5      45.6
// and splits of 64 x 64 tiles:   1      2      4
//   256 x 1024 x 4096           16.9   12.7   10.9
//   784 x 389 x 5242            23.9   18.6   14.5
//   182 x 4704 x 9980           37.3   29.5   28.9
//   2048 x 1024 x 4096          21.2   26.5   33.5
// Over 42 sizes drawn at random (97 to 4096 rows, 97 to 8192 columns, 256 to 8192
// deep) its choice is 1.2 % slower than the best tile and split (geometric mean; the
// worst, 948 x 207 x 3204 in 7 splits where 4 are best, 15 %). Its predicted times are
// looser than its choice: 1360 x 3015 x 5344 is predicted at 40.6 and took 38.9 and 50.2
// on two cards. More LDS stages (five of each operand) leave all of these as they are.
// Up to 96 rows of A the kernel for few rows competes, by what a CU loads at 66 GB/s:
//   65 x 4096 x 4096     few 8.6, tiles 12.5      96 x 11008 x 4096 (fp32)   16.2, 26.8
//   65 x 800 x 11008         14.0       11.9      96 x 2048 x 8192           14.5, 13.4
// From 97 rows on its gain is gone (128 x 8192 x 8192: 23.8, 24.2; 128 x 4096 x 11008:
// 24.9, 22.5). Up to 64 rows of A it runs without a comparison, so that a column's bits
// do not depend on N (a token's logits not on the vocabulary's shard). Where B has few
// rows and K is long that costs time: 64 x 512 x 11008 takes 13.7 us on 32 workgroups,
// split tiles of 65 rows 10.3; 64 x 1024 x 11008 14.3 and 12.1; at 2048 rows of B they
// are even (14.4, 15.4).
namespace {
struct TileTimes {
  int bm, bn, levels;       // levels: 1, 2, 4 tiles on a CU
  double step[2][3], ends[2];   // of 16-bit and of fp32 C
};
constexpr TileTimes kTileTimes[] = {
    {256, 256, 1, {{1.55}, {2.92}}, {11.0, 16.0}},
    {128, 128, 2, {{0.66, 1.08}, {1.00, 1.90}}, {5.5, 6.5}},
    {128, 64, 2, {{0.57, 0.75}, {0.80, 1.16}}, {3.6, 4.4}},
    {64, 64, 3, {{0.43, 0.56, 0.815}, {0.61, 0.80, 1.26}}, {3.2, 4.0}},
};

// workgroups of `share` steps each
double predicted(const TileTimes& t, int64_t wgs, int64_t share, bool fp32) {
  const double* const step = t.step[fp32];
  const double ends = t.ends[fp32];
  const int64_t held = (int64_t)kFp8Cus << (t.levels - 1), rest = wgs % held;
  double us = (double)(wgs / held) * (share * step[t.levels - 1] + ends);
  if (rest > 0) {
    int level = 0;
    while (rest > (int64_t)kFp8Cus << level) ++level;
    const double half = (double)((int64_t)kFp8Cus << level) / 2;
    const double s = level == 0 ? step[0] : step[level - 1] + (step[level] - step[level - 1]) * (0.4 + 0.6 * (rest - half) / half);
    us += share * s + (wgs > held && t.levels > 1 ? ends / 2 : ends);
  }
  return us;
}
}  // namespace

hipError_t launch_fp8_mm_splits(const Fp8MmArgs& a, const Fp8MmPlan& plan, bool exact, void* ws, hipStream_t s) {
  Fp8MmArgs g = a;
  g.splits = plan.splits;
  g.split_steps = plan.split_steps;
  g.C = ws;
  g.ldc = (int32_t)fp8_sums_pitch(a.N);
  g.bias = nullptr;
  g.accumulate = 0;
  return exact ? small_tile<float, true>(g, plan, s) : small_tile<float, false>(g, plan, s);
}

Fp8MmPlan fp8_mm_plan(int64_t M, int64_t N, int64_t K, bool fp32) { return fp8_mm_plan_wide(M, N, K, fp32, 0); }

Fp8MmPlan fp8_mm_plan_wide(int64_t M, int64_t N, int64_t K, bool fp32, int least_bn) {
  Fp8MmPlan best;
  if (M <= kFp8AlwaysFew) {
    best.bm = 0;
    return best;
  }
  const int64_t steps = (K + kBK - 1) / kBK;
  double least = 0;
  for (const TileTimes& tile : kTileTimes) {
    const int64_t n_tiles = (M + tile.bm - 1) / tile.bm * ((N + tile.bn - 1) / tile.bn);
    const int64_t held = (int64_t)kFp8Cus << (tile.levels - 1);
    if (n_tiles > kMaxMmTiles) continue;
    // 256 x 256 tiles are for large products and never split
    for (int64_t want = 1; want == 1 || (want <= 16 && tile.levels > 1 && n_tiles * want <= held); ++want) {
      // shares are whole words of scale bytes
      const int64_t share = want == 1 ? steps : ((steps + want - 1) / want + 3) & ~(int64_t)3;
      const int64_t n = share > 0 ? (steps + share - 1) / share : 1;   // splits
      if (n != want || (n == 1 && tile.bn < least_bn)) continue;
      double us = predicted(tile, n_tiles * n, share, fp32);
      if (n > 1) us += 2.5 + (double)n * M * N * 8 / 5e6;
      if (least > 0 && us >= least) continue;
      least = us;
      best.bm = tile.bm;
      best.bn = tile.bn;
      best.splits = (int)n;
      best.split_steps = (int)share;
      best.ws_bytes = n > 1 ? (size_t)n * M * fp8_sums_pitch(N) * 4 : 0;
    }
  }
  if (M <= kFp8FewRows && fp8_few_loads(M, N, fp8_few_blocks(M, N)) * K / 66e3 + 2.5 < least) {
    best = {};
    best.bm = 0;
  }
  return best;
}

hipError_t launch_fp8_mm(const Fp8MmArgs& a, const Fp8MmPlan& plan, void* ws, hipStream_t s) {
  switch (a.c_type) {
    case T_FP16: return run<f16>(a, plan, ws, s);
    case T_BF16: return run<bf16>(a, plan, ws, s);
    default: return run<float>(a, plan, ws, s);
  }
}

}  // namespace iris
