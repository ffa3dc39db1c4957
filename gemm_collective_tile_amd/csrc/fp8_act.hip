// Products A B^T of block-scaled 8-bit operands with bias, activation, dropout and
// residual in their epilogue, into 16 or 32 bits and / or 8, and the backward pass of
// such an epilogue. The sums are those of the plain product (fp8_gemm_tile.hpp,
// fp8_gemm_few.hpp); what follows here happens in 32 bits, with one rounding of each
// output. A tile's sums turn around in LDS, 32 rows at a time, so that a lane gets 8
// columns of a row: a call of the dropout's generator, 16 bytes of a 16-bit matrix; 16
// lanes hold a block of 128 of an 8-bit output and agree on its scale among themselves.
#include <algorithm>

#include "column_sums.hpp"
#include "fp8_act_math.hpp"
#include "fp8_gemm_few.hpp"
#include "fp8_gemm_tile.hpp"

namespace iris {
namespace {

// the matrix that an epilogue reads beside the sums: z, the residual or none
template <bool BACKWARD, class OUT>
struct Beside {
  const OUT* at;
  int ld;
  __device__ __forceinline__ explicit Beside(const Fp8ActArgs& a)
      : at((const OUT*)(BACKWARD ? a.z : a.residual)), ld(BACKWARD ? a.ldz : a.ldr) {}
  __device__ __forceinline__ void load(int m, int n, int N, bool on, Raw8<OUT>& r) const {
    if (at && on) r.template load<false>(at + (int64_t)m * ld, n, N);
  }
};

// C and z written at any pitch and alignment, by those lanes whose piece lies inside
template <class OUT>
struct PutRagged {
  static constexpr bool WHOLE = false;
  const Fp8ActArgs* a;
  int m, n;
  bool on;
  __device__ __forceinline__ void z(const float (&v)[8]) const {
    if (on) store8<false>((OUT*)a->z + (int64_t)m * a->ldz, n, a->g.N, v);
  }
  __device__ __forceinline__ void c(const float (&v)[8]) const {
    if (on) store8<false>((OUT*)a->g.C + (int64_t)m * a->g.ldc, n, a->g.N, v);
  }
};
// whole, aligned pieces through buffers, which drop a lane's that is off: no branch
// between them, so that the number of stores under way is known
template <class OUT>
struct PutWhole {
  static constexpr bool WHOLE = true;
  __amdgpu_buffer_rsrc_t c_rows, z_rows;
  uint32_t c_at, z_at;   // bytes, or kOob
  static __device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t at, const float (&v)[8]) {
    OUT t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) narrow(v[i], t[i]);
    u32x4 w[sizeof t / 16];
    __builtin_memcpy(w, t, sizeof t);
#pragma unroll
    for (int i = 0; i < (int)(sizeof t / 16); ++i) __builtin_amdgcn_raw_buffer_store_b128(w[i], r, at + 16 * i, 0, 0);
  }
  __device__ __forceinline__ void z(const float (&v)[8]) const { put(z_rows, z_at, v); }
  __device__ __forceinline__ void c(const float (&v)[8]) const { put(c_rows, c_at, v); }
};

// U times 8 sums, of rows m[u], columns n .. n + 7, through the epilogue; on: they lie
// inside C. All 16 lanes of a block of 128 columns call it together where q is wanted.
// `beside`: their values of z (backward) or of the residual, in memory's form. Each step
// is taken for all U before the next: what is not wanted is branched over once for them
// (with one wave a SIMD a branch taken costs as much as seven instructions: 8192 x 11008 x
// 4096 without an activation 356 us with U = 1, 336 with 4, as the plain product).
template <bool BACKWARD, class OUT, class PUT, int U>
__device__ __forceinline__ void finish(const Fp8ActArgs& a, const Drop& drop, const int (&m)[U], int n, const bool (&on)[U],
                                       const float (&bias)[8], const Raw8<OUT> (&beside)[U], const PUT (&put)[U],
                                       float (&v)[U][8], float (&sums)[8]) {
  const int N = a.g.N;
  if constexpr (BACKWARD) {
    float z[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) beside[u].values(z[u]);
    times_slope<sizeof(OUT) == 4>(a.act, z, v);
    drop.apply(m, (uint32_t)n >> 3, v);
    if (a.dbias_part) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (__all(on[u])) {   // all but the last tiles: no select for each value
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[i] += v[u][i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[i] += on[u] ? v[u][i] : 0.0f;
        }
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] += bias[i];
    if (a.z) {
#pragma unroll
      for (int u = 0; u < U; ++u) put[u].z(v[u]);
    }
    activate<sizeof(OUT) == 4>(a.act, v);
    drop.apply(m, (uint32_t)n >> 3, v);
    if (a.residual) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float r[8];
        beside[u].values(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] += r[i];
      }
    }
  }
  if (BACKWARD || a.g.C) {
#pragma unroll
    for (int u = 0; u < U; ++u) put[u].c(v[u]);
  }
  if (!BACKWARD && a.q.codes) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // what lies outside has no say in the scale, and its codes go nowhere
      if constexpr (!PUT::WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = n + i < N ? v[u][i] : 0.0f;
      }
      const uint32_t s = scale_byte(group_max<16>(piece_amax(v[u]) & on_mask(on[u])));
      uint32_t w[2];
      encode_piece(v[u], scale_value(s), w);
      if (on[u]) {
        store_codes<PUT::WHOLE, 8>(a.q.codes + (int64_t)m[u] * a.q.ld, 0, n, N, w);
        if (n % kFp8Block == 0) a.q.scales[(int64_t)m[u] * a.q.lds + n / kFp8Block] = (uint8_t)s;
      }
    }
  }
}

template <class OUT>
__device__ __forceinline__ void load_bias8(const Fp8ActArgs& a, int n, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  if (a.g.bias && n < a.g.N) load8<false>((const OUT*)a.g.bias, n, a.g.N, b);
}

// between the writes and the reads of a strip: of the workgroup's waves where they share
// it, else of the wave's lanes
template <bool SHARED>
__device__ __forceinline__ void strip_barrier() {
  if constexpr (SHARED) {
    __syncthreads();
  } else {
    __builtin_amdgcn_wave_barrier();
    wait_lds();
  }
}

// WHOLE: N is a multiple of 8 and all rows of C, z and the residual start at multiples of
// 16 bytes.
//
// Bound by the matrix units in the products (8192 x 11008 x 4096 324-334 us without an
// epilogue, 2250 TFLOP/s: 5.4 rounds of tiles take 6) and by the vector units behind
// them, which work while the matrix units wait: with 256 x 256 one workgroup fills a CU.
// Smaller tiles, two a CU, hide the epilogue and lose more in the products (through
// gelu_tanh with z and 8-bit codes 420 us where these took 405, 4096 x 4096 x 11008 with
// dropout and residual 184 and 153). Now 381-395 us, 152-161, and 4095 x 11008 x 4096
// backwards through gelu_tanh with dropout and the bias's gradient 209-215 (product 166-170).
//
// What is read beside the sums (z or the residual) is fetched strips ahead of its use.
// Vector memory operations are counted in their order, loads and stores alike: a load
// that is waited for without knowing the number of stores behind it waits for these too,
// a few us under load, for every strip. So with WHOLE the loads go into LDS unseen by
// the compiler, and the wait counts the stores of C that are surely behind them. Else
// they wait in registers, and are waited for as the compiler does it.
template <class OUT, int BM, int BN, bool WHOLE, bool BACKWARD>
__global__ __launch_bounds__(256, BM * BN > 128 * 128 ? 1 : 2) void fp8_mm_act_kernel(Fp8ActArgs a) {
  using T = Tile<BM, BN>;
  constexpr bool EXACT = sizeof(OUT) == 4;
  __shared__ __align__(16) char lds[T::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int pm, pn;
  if (!pick_tile<OUT, T>(a.g, pm, pn)) return;
  const int m0 = pm * BM, n0 = pn * BN, r32 = lane & 31;

  // A strip of 32 rows is as wide as a block of 128 (64 where the tile is): a wave's own
  // at 256 columns, else what two waves side by side hold, who then take 16 of its rows each.
  constexpr bool SHARED = BN <= 128;
  constexpr int SW = BN < 128 ? BN : 128, PITCH = SW + 4, LPR = SW / 8, RPI = 64 / LPR;
  constexpr int STRIP = 32 * PITCH, STRIPS = SHARED ? 2 : 4, ROWS = SHARED ? 16 : 32, PASSES = ROWS / RPI;
  constexpr int PIECES = sizeof(Raw8<OUT>) / 16, RAW_AT = STRIPS * STRIP * 4, RAW = 4 * PASSES * PIECES * 1024;
  constexpr int AHEAD = T::FM > 1 && WHOLE && RAW_AT + 2 * RAW <= T::LDS ? 2 : 1;   // strips that are fetched
  static_assert(RAW_AT + AHEAD * RAW <= T::LDS && 4 * SW * 4 <= T::LDS, "the turn does not fit");
  const int right = wave & 1, half = wave >> 1;
  const int c = 8 * (lane % LPR), nw = n0 + (SHARED ? 0 : right * T::WN), n = nw + c;
  f32x16 acc[T::FM][T::FN];
  Raw8<OUT> bias_raw = {};
  tile_sums<EXACT, T>(a.g, lds, pm, pn, acc, [&] {
    if (!BACKWARD && a.g.bias && n < a.g.N) bias_raw.template load<false>((const OUT*)a.g.bias, n, a.g.N);
  });

  float* const strip = (float*)lds + (SHARED ? half : wave) * STRIP;
  // 16-byte pieces, a lane's side by side with the other lanes'
  const int raw_wave = RAW_AT + wave * PASSES * PIECES * 1024;
  const int lane_row = (SHARED ? right * 16 : 0) + lane / LPR;   // of a strip, in the first pass
  const Drop drop(a.drop);
  const Beside<BACKWARD, OUT> beside(a);
  float bias[8], sums[8] = {};
  bias_raw.values(bias);
  const auto first_row = [&](int i) { return m0 + half * T::WM + 32 * i; };   // of strip i

  Raw8<OUT> raw[WHOLE ? 1 : PASSES];
  const uint32_t lds_raw = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + raw_wave);
  const auto fetch = [&](int i) {
    if constexpr (WHOLE) {
      // rows and columns past the end read inside again: their outputs are dropped
      const int top = min(first_row(i), a.g.M - 1);
      const i32x4 rsrc = buffer_words(beside.at + (int64_t)top * beside.ld + min(nw, a.g.N - 8));
      const uint32_t col = nw < a.g.N - 8 ? (uint32_t)min(c, a.g.N - 8 - nw) : 0;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const uint32_t row = (uint32_t)min(lane_row + RPI * p, a.g.M - 1 - top);
#pragma unroll
        for (int h = 0; h < PIECES; ++h)
          buffer_to_lds(rsrc, (row * (uint32_t)beside.ld + col) * (uint32_t)sizeof(OUT) + 16 * h, 0,
                        lds_raw + (i % AHEAD) * RAW + (p * PIECES + h) * 1024);
      }
    } else {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int m = first_row(i) + lane_row + RPI * p;
        beside.load(m, n, a.g.N, m < a.g.M && n < a.g.N, raw[p]);
      }
    }
  };
  // Until strip i has landed. Behind its loads, of this wave's, are surely the stores of C that strip
  // i - 1 sent after them (whatever else it stored) and the next strip's loads, LOADS of each.
  constexpr int LOADS = PASSES * PIECES;
  static_assert(2 * LOADS < 64, "more than a wait can count");
  const auto wait_for = [&](int i) {
    if constexpr (AHEAD == 1) {
      wait_loads<0>();
    } else {
      const bool stored = i > 0 && a.g.C, more = i + 1 < T::FM;
      if (stored && more)
        wait_loads<2 * LOADS>();
      else if (stored || more)
        wait_loads<LOADS>();
      else
        wait_loads<0>();
    }
  };
  if (beside.at) {
    fetch(0);
    if constexpr (AHEAD == 2) fetch(1);
  }
  // The passes over a strip stand in the code once: four times they exceed the instruction
  // cache (76 KB; 8192 x 11008 x 4096 through relu backwards 417 us, so 393).
#pragma unroll 1
  for (int i = 0; i < T::FM; ++i) {
    float* const to = strip + r32 * PITCH + (SHARED ? right * T::WN : 0) + 4 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < T::FM; ++k) {
      if (k != i) continue;
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(f32x4*)(to + 32 * j + 8 * q) = f32x4{acc[k][j][4 * q], acc[k][j][4 * q + 1], acc[k][j][4 * q + 2], acc[k][j][4 * q + 3]};
    }
    char* const raw_at = lds + raw_wave + (i % AHEAD) * RAW + 16 * lane;
    if (beside.at) {
      if constexpr (WHOLE) {
        wait_for(i);
      } else {
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
#pragma unroll
          for (int h = 0; h < PIECES; ++h) __builtin_memcpy(raw_at + (p * PIECES + h) * 1024, raw[p].w + 4 * h, 16);
        if (i + 1 < T::FM) fetch(i + 1);
      }
    }
    strip_barrier<SHARED>();
    const int top = first_row(i);
    const __amdgpu_buffer_rsrc_t c_rows = make_rsrc((const OUT*)a.g.C + (int64_t)top * a.g.ldc + nw, 0x7fffffffu);
    const __amdgpu_buffer_rsrc_t z_rows = make_rsrc((const OUT*)a.z + (int64_t)top * a.ldz + nw, 0x7fffffffu);
    constexpr int U = PASSES < 4 ? PASSES : 4;
#pragma unroll 1
    for (int p0 = 0; p0 < PASSES; p0 += U) {
      int m[U];
      bool on[U];
      float v[U][8];
      Raw8<OUT> here[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = lane_row + RPI * (p0 + u);
        m[u] = top + row;
        on[u] = m[u] < a.g.M && n < a.g.N;
        __builtin_memcpy(v[u], strip + row * PITCH + c, sizeof v[u]);
      }
      if (beside.at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < PIECES; ++h) __builtin_memcpy(here[u].w + 4 * h, raw_at + ((p0 + u) * PIECES + h) * 1024, 16);
      }
      if constexpr (WHOLE) {
        PutWhole<OUT> put[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t row = (uint32_t)(m[u] - top);
          put[u].c_rows = c_rows;
          put[u].z_rows = z_rows;
          put[u].c_at = on[u] ? (row * (uint32_t)a.g.ldc + c) * (uint32_t)sizeof(OUT) : kOob;
          put[u].z_at = on[u] ? (row * (uint32_t)a.ldz + c) * (uint32_t)sizeof(OUT) : kOob;
        }
        finish<BACKWARD, OUT>(a, drop, m, n, on, bias, here, put, v, sums);
      } else {
        PutRagged<OUT> put[U];
#pragma unroll
        for (int u = 0; u < U; ++u) put[u] = PutRagged<OUT>{&a, m[u], n, on[u]};
        finish<BACKWARD, OUT>(a, drop, m, n, on, bias, here, put, v, sums);
      }
    }
    strip_barrier<SHARED>();
    if (WHOLE && beside.at && i + AHEAD < T::FM) fetch(i + AHEAD);
  }
  if (!a.dbias_part) return;
  // the tile's column sums: over the lanes, then over the waves, in order
  __syncthreads();
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

// Few rows of A: an output a thread. Bound by the weights' bytes as the plain product is:
// 1 x 11008 x 4096 through gelu 7.3-9.2 us, 5.5 TB/s from the last-level cache.
template <class OUT>
struct PutAct {
  void *z, *c;
  const void *bias, *residual;
  int32_t ldz, ldc, ldr;
  uint8_t act, backward;
  DropArgs drop;
  __device__ __forceinline__ void put(const Fp8MmArgs&, int m, int n, float s) const {
    float v[1][1] = {{s}};
    const Drop d(drop);
    OUT* const at = z ? (OUT*)z + (int64_t)m * ldz + n : nullptr;
    if (backward) {
      const float y[1][1] = {{widen(*at)}};
      times_slope<sizeof(OUT) == 4>(act, y, v);
      v[0][0] = d.apply((uint32_t)m, (uint32_t)n, v[0][0]);
    } else {
      if (bias) v[0][0] += widen(((const OUT*)bias)[n]);
      if (at) narrow(v[0][0], *at);
      activate<sizeof(OUT) == 4>(act, v);
      v[0][0] = d.apply((uint32_t)m, (uint32_t)n, v[0][0]);
      if (residual) v[0][0] += widen(((const OUT*)residual)[(int64_t)m * ldr + n]);
    }
    narrow(v[0][0], ((OUT*)c)[(int64_t)m * ldc + n]);
  }
};
// its sums alone
struct PutSum {
  float* sums;
  int64_t pitch;
  __device__ __forceinline__ void put(const Fp8MmArgs&, int m, int n, float s) const { sums[m * pitch + n] = s; }
};

// Sums in the workspace (those of a.g.splits splits, added in order) through the epilogue.
// A workgroup takes a block of 128 columns, `rows` rows of it, 16 at a time. Bound by
// latency: 33 x 11008 through silu to 8 bits 2.8 us.
template <class OUT, bool BACKWARD>
__global__ __launch_bounds__(256) void fp8_mm_act_join_kernel(Fp8ActArgs a, const float* part, int64_t ldp, int rows) {
  __shared__ float red[4][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = blockIdx.x * 128 + 8 * (lane & 15), from = blockIdx.y * rows, to = min(from + rows, a.g.M);
  const Drop drop(a.drop);
  const Beside<BACKWARD, OUT> beside(a);
  float bias[8], sums[8] = {};
  load_bias8<OUT>(a, n, bias);
  for (int base = from; base < to; base += 16) {
    const int m[1] = {base + (int)(threadIdx.x >> 4)};
    const bool on[1] = {m[0] < to && n < a.g.N};
    float v[1][8] = {};
    if (on[0]) {
      const float* p = part + (int64_t)m[0] * ldp + n;
      for (int s = 0; s < a.g.splits; ++s, p += (int64_t)a.g.M * ldp) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (n + 4 * h >= a.g.N) continue;   // the pitch is a multiple of 4
          const f32x4 x = *(const f32x4*)(p + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[0][4 * h + e] += x[e];
        }
      }
    }
    Raw8<OUT> here[1];
    beside.load(m[0], n, a.g.N, on[0], here[0]);
    const PutRagged<OUT> put[1] = {{&a, m[0], n, on[0]}};
    finish<BACKWARD, OUT>(a, drop, m, n, on, bias, here, put, v, sums);
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

// Rows of a joining workgroup. Without column sums 16, a turn of its loop, so that as many
// workgroups as there are share the latency: 301 x 397 x 4111 to 8 bits 12.8 us, with 32 rows
// 16.4, with 64 23.6; 33 x 11008 x 4096 13.7, 14.6, 15.5; 517 x 2053 x 8305 27.0, 28.0, 31.0. With
// column sums 64, four turns one after the other: a quarter of the rows of partial sums, for
// which a call has to find room in the workspace (few rows of a wide B take all of the
// library's own with two such rows). That costs time: with dbias the same three take 25.7,
// 18.5 and 34.5 us, with 32 rows 18.5, 17.3 and 30.9, with 16 15.0, 16.3 and 30.0.
constexpr int kJoinRows = 16, kJoinRowsSummed = 64;

template <class OUT, int BM, int BN>
hipError_t launch_tiles(const Fp8ActArgs& a, hipStream_t s) {
  const int64_t tiles = ((int64_t)a.g.M + BM - 1) / BM * (((int64_t)a.g.N + BN - 1) / BN);
  const int64_t round = kPatch * kXcds;
  const dim3 grid((uint32_t)((tiles + round - 1) / round * round));
  const auto launch = [&](auto whole, auto backward) {
    hipLaunchKernelGGL((fp8_mm_act_kernel<OUT, BM, BN, decltype(whole)::value, decltype(backward)::value>), grid, dim3(256), 0,
                       s, a);
  };
  using std::false_type, std::true_type;
  if (a.backward)
    a.whole ? launch(true_type{}, true_type{}) : launch(false_type{}, true_type{});
  else
    a.whole ? launch(true_type{}, false_type{}) : launch(false_type{}, false_type{});
  return hipGetLastError();
}

template <class OUT>
hipError_t run(const Fp8ActArgs& args, const Fp8ActPlan& plan, OUT* dbias, void* ws, hipStream_t s) {
  Fp8ActArgs a = args;
  hipError_t e = hipSuccess;
  a.g.splits = 1;
  a.ldp = (int32_t)fp8_sums_pitch(a.g.N);
  if (a.g.M == 0) return join_columns(nullptr, 0, 0, a.g.N, dbias, s);
  a.dbias_part = plan.parts > 0 ? (float*)((char*)ws + plan.part_at) : nullptr;
  if (plan.sums) {
    const int64_t ldp = a.ldp;
    e = plan.mm.bm == 0 ? launch_few<PutSum, sizeof(OUT) == 4>(a.g, PutSum{(float*)ws, ldp}, s)
                        : launch_fp8_mm_splits(a.g, plan.mm, sizeof(OUT) == 4, ws, s);
    if (e != hipSuccess) return e;
    a.g.splits = plan.mm.splits;
    const int rows = plan.parts > 0 ? kJoinRowsSummed : kJoinRows;
    const dim3 grid((a.g.N + 127) / 128, (a.g.M + rows - 1) / rows);
    if (a.backward)
      hipLaunchKernelGGL((fp8_mm_act_join_kernel<OUT, true>), grid, dim3(256), 0, s, a, (const float*)ws, ldp, rows);
    else
      hipLaunchKernelGGL((fp8_mm_act_join_kernel<OUT, false>), grid, dim3(256), 0, s, a, (const float*)ws, ldp, rows);
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
  return join_columns(a.dbias_part, plan.parts, a.ldp, a.g.N, dbias, s);
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
