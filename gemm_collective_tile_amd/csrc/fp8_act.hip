// Products A B^T of block-scaled 8-bit operands with bias, activation, dropout and
// residual in their epilogue, into 16 or 32 bits and / or 8, and the backward pass of
// such an epilogue. The sums are those of the plain product (fp8_gemm_tile.hpp,
// fp8_gemm_few.hpp); what follows here happens in 32 bits, with one rounding of each
// output. A tile's sums turn around in LDS, 32 rows at a time, so that a lane gets 8
// columns of a row: a call of the dropout's generator, 16 bytes of a 16-bit matrix; 16
// lanes hold a block of 128 of an 8-bit output and agree on its scale among themselves.
#include <algorithm>

#include "fp8_act_math.hpp"
#include "fp8_gemm_few.hpp"
#include "fp8_gemm_tile.hpp"

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

// 8 sums of row m, columns n .. n + 7, through the epilogue; on: they lie inside C. All
// 16 lanes of a block of 128 columns call it together where q is wanted.
template <class OUT>
__device__ __forceinline__ void finish8(const Fp8ActArgs& a, const Drop& drop, int m, int n, bool on, const float (&bias)[8],
                                        float (&v)[8], float (&sums)[8]) {
  const int N = a.g.N;
  if (on) {
    if (a.backward) {
      float z[8];
      load8((const OUT*)a.z + (int64_t)m * a.ldz, n, N, z);
      times_slope(a.act, z, v);
      drop.apply((uint32_t)m, (uint32_t)n >> 3, v);
      if (a.dbias_part) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[i] += v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += bias[i];
      if (a.z) store8<false>((OUT*)a.z + (int64_t)m * a.ldz, n, N, v);
      activate(a.act, v);
      drop.apply((uint32_t)m, (uint32_t)n >> 3, v);
      if (a.residual) {
        float r[8];
        load8((const OUT*)a.residual + (int64_t)m * a.ldr, n, N, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
    }
    if (a.g.C) store8<false>((OUT*)a.g.C + (int64_t)m * a.g.ldc, n, N, v);
  }
  if (a.q.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = on && n + i < N ? __builtin_canonicalizef(v[i]) : 0.0f;
    const uint32_t s = scale_byte(group_max<16>(piece_amax(v)));
    uint32_t w[2];
    encode_piece(v, scale_value(s), w);
    if (on) {
      store_codes<false, 8>(a.q.codes + (int64_t)m * a.q.ld, 0, n, N, w);
      if (n % kFp8Block == 0) a.q.scales[(int64_t)m * a.q.lds + n / kFp8Block] = (uint8_t)s;
    }
  }
}

template <class OUT>
__device__ __forceinline__ void load_bias8(const Fp8ActArgs& a, int n, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  if (a.g.bias && n < a.g.N) load8((const OUT*)a.g.bias, n, a.g.N, b);
}

template <class OUT, int BM, int BN>
__global__ __launch_bounds__(256) void fp8_mm_act_kernel(Fp8ActArgs a) {
  using T = Tile<BM, BN>;
  constexpr bool EXACT = sizeof(OUT) == 4;
  __shared__ __align__(16) char lds[T::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int pm, pn;
  if (!pick_tile<OUT, T>(a.g, pm, pn)) return;
  const int m0 = pm * BM, n0 = pn * BN, r32 = lane & 31;
  f32x16 acc[T::FM][T::FN];
  tile_sums<EXACT, T>(a.g, lds, pm, pn, acc, [] {});

  // A strip of 32 rows is as wide as a block of 128 (64 where the tile is): a wave's own
  // at 256 columns, else what two waves side by side hold, who then take 16 of its rows each.
  constexpr bool SHARED = BN <= 128;
  constexpr int SW = BN < 128 ? BN : 128, PITCH = SW + 4, LPR = SW / 8, RPI = 64 / LPR;
  constexpr int STRIP = 32 * PITCH, STRIPS = SHARED ? 2 : 4, ROWS = SHARED ? 16 : 32;
  static_assert(STRIPS * STRIP * 4 <= T::LDS && 4 * SW * 4 <= T::LDS, "the turn does not fit");
  const int right = wave & 1, half = wave >> 1;
  float* const strip = (float*)lds + (SHARED ? half : wave) * STRIP;
  const int c = 8 * (lane % LPR), n = n0 + (SHARED ? 0 : right * T::WN) + c;
  const Drop drop(a.drop);
  float bias[8], sums[8] = {};
  load_bias8<OUT>(a, n, bias);
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    float* const to = strip + r32 * PITCH + (SHARED ? right * T::WN : 0) + 4 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(to + 32 * j + 8 * q) = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < ROWS; r += RPI) {
      const int row = (SHARED ? right * 16 : 0) + r + lane / LPR, m = m0 + half * T::WM + 32 * i + row;
      float v[8];
      __builtin_memcpy(v, strip + row * PITCH + c, sizeof v);
      finish8<OUT>(a, drop, m, n, m < a.g.M && n < a.g.N, bias, v, sums);
    }
    __syncthreads();
  }
  if (!a.dbias_part) return;
  // the tile's column sums: over the lanes, then over the waves, in order
  float* const red = (float*)lds;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[e] = same_columns_sum<LPR>(sums[e]);
  if (lane < LPR) __builtin_memcpy(red + wave * SW + c, sums, sizeof sums);
  __syncthreads();
  if (tid < BN && n0 + tid < a.g.N) {
    const float* const of = red + (SHARED ? tid : (tid / SW) * SW + tid % SW);
    a.dbias_part[(int64_t)pm * a.ldp + n0 + tid] = SHARED ? (of[0] + of[SW]) + (of[2 * SW] + of[3 * SW]) : of[0] + of[2 * SW];
  }
}

// Few rows of A: an output a thread.
template <class OUT>
struct PutAct {
  void *z, *c;
  const void *bias, *residual;
  int32_t ldz, ldc, ldr;
  uint8_t act, backward;
  DropArgs drop;
  __device__ __forceinline__ void put(const Fp8MmArgs&, int m, int n, float s) const {
    float v[1] = {s};
    const Drop d(drop);
    OUT* const at = z ? (OUT*)z + (int64_t)m * ldz + n : nullptr;
    if (backward) {
      const float y[1] = {widen(*at)};
      times_slope(act, y, v);
      v[0] = d.apply((uint32_t)m, (uint32_t)n, v[0]);
    } else {
      if (bias) v[0] += widen(((const OUT*)bias)[n]);
      if (at) narrow(v[0], *at);
      activate(act, v);
      v[0] = d.apply((uint32_t)m, (uint32_t)n, v[0]);
      if (residual) v[0] += widen(((const OUT*)residual)[(int64_t)m * ldr + n]);
    }
    narrow(v[0], ((OUT*)c)[(int64_t)m * ldc + n]);
  }
};
// its sums alone
struct PutSum {
  float* sums;
  int64_t pitch;
  __device__ __forceinline__ void put(const Fp8MmArgs&, int m, int n, float s) const { sums[m * pitch + n] = s; }
};

// Sums in the workspace (those of a.g.splits splits, added in order) through the epilogue.
// A workgroup takes a block of 128 columns, `rows` rows of it, 16 at a time.
template <class OUT>
__global__ __launch_bounds__(256) void fp8_mm_act_join_kernel(Fp8ActArgs a, const float* part, int64_t ldp, int rows) {
  __shared__ float red[4][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = blockIdx.x * 128 + 8 * (lane & 15), from = blockIdx.y * rows, to = min(from + rows, a.g.M);
  const Drop drop(a.drop);
  float bias[8], sums[8] = {};
  load_bias8<OUT>(a, n, bias);
  for (int base = from; base < to; base += 16) {
    const int m = base + (threadIdx.x >> 4);
    const bool on = m < to && n < a.g.N;
    float v[8] = {};
    if (on) {
      const float* p = part + (int64_t)m * ldp + n;
      for (int s = 0; s < a.g.splits; ++s, p += (int64_t)a.g.M * ldp) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (n + 4 * h >= a.g.N) continue;   // the pitch is a multiple of 4
          const f32x4 x = *(const f32x4*)(p + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * h + e] += x[e];
        }
      }
    }
    finish8<OUT>(a, drop, m, n, on, bias, v, sums);
  }
  if (!a.dbias_part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[e] = same_columns_sum<16>(sums[e]);
  if (lane < 16) __builtin_memcpy(&red[wave][8 * lane], sums, sizeof sums);
  __syncthreads();
  const int col = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && col < a.g.N) {
    const int t = threadIdx.x;
    a.dbias_part[(int64_t)blockIdx.y * a.ldp + col] = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
  }
}

// dbias = the partial sums, 16 of every 64 columns at a time
template <class OUT>
__global__ __launch_bounds__(1024) void fp8_dbias_kernel(const float* part, int parts, int64_t ldp, int N, OUT* dbias) {
  __shared__ float red[16][64];
  const int l = threadIdx.x & 63, c = blockIdx.x * 64 + l, g = threadIdx.x >> 6;
  float v = 0.0f;
  if (c < N) {
#pragma unroll 4
    for (int i = g; i < parts; i += 16) v += part[i * ldp + c];
  }
  red[g][l] = v;
  __syncthreads();
  if (g == 0 && c < N) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[i][l];
    narrow(v, dbias[c]);
  }
}

constexpr int kJoinRows = 16, kJoinRowsSummed = 64;   // without and with column sums

template <class OUT, int BM, int BN>
hipError_t launch_tiles(const Fp8ActArgs& a, hipStream_t s) {
  const int64_t tiles = ((int64_t)a.g.M + BM - 1) / BM * (((int64_t)a.g.N + BN - 1) / BN);
  const int64_t round = kPatch * kXcds;
  hipLaunchKernelGGL((fp8_mm_act_kernel<OUT, BM, BN>), dim3((uint32_t)((tiles + round - 1) / round * round)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class OUT>
hipError_t join_dbias(const float* part, int parts, int64_t ldp, int N, OUT* dbias, hipStream_t s) {
  hipLaunchKernelGGL((fp8_dbias_kernel<OUT>), dim3((N + 63) / 64), dim3(1024), 0, s, part, parts, ldp, N, dbias);
  return hipGetLastError();
}

template <class OUT>
hipError_t run(const Fp8ActArgs& args, const Fp8ActPlan& plan, OUT* dbias, void* ws, hipStream_t s) {
  Fp8ActArgs a = args;
  hipError_t e = hipSuccess;
  a.g.splits = 1;
  a.ldp = (int32_t)fp8_sums_pitch(a.g.N);
  if (a.g.M == 0) return join_dbias(nullptr, 0, 0, a.g.N, dbias, s);
  a.dbias_part = plan.parts > 0 ? (float*)((char*)ws + plan.part_at) : nullptr;
  if (plan.sums) {
    const int64_t ldp = a.ldp;
    e = plan.mm.bm == 0 ? launch_few<PutSum, sizeof(OUT) == 4>(a.g, PutSum{(float*)ws, ldp}, s)
                        : launch_fp8_mm_splits(a.g, plan.mm, sizeof(OUT) == 4, ws, s);
    if (e != hipSuccess) return e;
    a.g.splits = plan.mm.splits;
    const int rows = plan.parts > 0 ? kJoinRowsSummed : kJoinRows;
    hipLaunchKernelGGL((fp8_mm_act_join_kernel<OUT>), dim3((a.g.N + 127) / 128, (a.g.M + rows - 1) / rows), dim3(256), 0, s, a,
                       (const float*)ws, ldp, rows);
    e = hipGetLastError();
  } else if (plan.mm.bm == 0) {
    e = launch_few<PutAct<OUT>, sizeof(OUT) == 4>(a.g, PutAct<OUT>{a.z, a.g.C, a.g.bias, a.residual, a.ldz, a.g.ldc, a.ldr, a.act,
                                                                  a.backward, a.drop}, s);
  } else if (plan.mm.bm == 256) {
    e = launch_tiles<OUT, 256, 256>(a, s);
  } else if (plan.mm.bn == 128) {
    e = launch_tiles<OUT, 128, 128>(a, s);
  } else {
    e = plan.mm.bm == 128 ? launch_tiles<OUT, 128, 64>(a, s) : launch_tiles<OUT, 64, 64>(a, s);
  }
  if (e != hipSuccess || plan.parts == 0) return e;
  return join_dbias(a.dbias_part, plan.parts, a.ldp, a.g.N, dbias, s);
}

}  // namespace

// An 8-bit output needs whole blocks of 128 columns in a workgroup: unsplit tiles of 128
// columns and more, or sums that are joined (few rows, splits). So do column sums of few
// rows, whose kernel gives a workgroup 16 to 48 columns and every thread one output.
Fp8ActPlan fp8_mm_act_plan(int64_t M, int64_t N, int64_t K, bool fp32, bool to8, bool dbias) {
  Fp8ActPlan p{};
  if (M == 0) return p;   // the bias's gradient alone: zeros
  p.mm = fp8_mm_plan_wide(M, N, K, fp32, to8 ? 128 : 0);
  p.sums = p.mm.splits > 1 || (p.mm.bm == 0 && (to8 || dbias));
  const size_t pitch = (size_t)fp8_sums_pitch(N) * 4, sums = p.sums ? (size_t)p.mm.splits * M * pitch : 0;
  p.part_at = (sums + 255) / 256 * 256;
  if (dbias) p.parts = (int32_t)(p.sums ? (M + kJoinRowsSummed - 1) / kJoinRowsSummed : (M + p.mm.bm - 1) / p.mm.bm);
  p.ws_bytes = p.parts > 0 ? p.part_at + p.parts * pitch : sums;
  return p;
}

hipError_t launch_fp8_mm_act(const Fp8ActArgs& a, const Fp8ActPlan& plan, void* dbias, void* ws, hipStream_t s) {
  switch (a.g.c_type) {
    case T_FP16: return run(a, plan, (f16*)dbias, ws, s);
    case T_BF16: return run(a, plan, (bf16*)dbias, ws, s);
    default: return run(a, plan, (float*)dbias, ws, s);
  }
}

}  // namespace iris
