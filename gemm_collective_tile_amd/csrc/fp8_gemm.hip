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
// bf16 values with their scales applied (v_cvt_scalef32_pk_bf16_fp8, exact
// within bf16's range) and v_mfma_f32_32x32x16_bf16, at half the rate,
// multiplies them exactly and sums in 32 bits (4e-8 of the result, measured).
// The conversions run in the shadow of the matrix instructions.
//
// Any order of k inside an instruction's slice gives the same sum as long as
// both operands use it, and a block's scale is the same for all its slices, so
// a lane takes the 16-byte pieces that are cheapest to read.
//
// Design (4 waves, 2 x 2, each a (BM/2) x (BN/2) part of the tile in 32-bit
// accumulators):
//   * K is walked in steps of 128 bytes per row. Rows go from memory straight
//     into LDS (no registers in between: the accumulators and one step's
//     operands fill the file), 8 lanes to a row's 128 bytes, the 16-byte pieces
//     permuted by the row so that the operand reads of 16 rows' same pieces
//     meet 16 different bank groups.
//   * A step has two slices of 64. While slice 0 multiplies, slice 1's
//     operands are read. Then every wave has this step in registers, one
//     barrier says so, and while slice 1 multiplies, slice 0 of the next step
//     is read. No operand read is waited for.
//   * A has three LDS stages and B two (all of the 160 KB at 256 x 256), so that
//     half of a step's loads, A's for the step after the next, go out beside
//     slice 0 and the other half, B's, beside slice 1: all of them beside one
//     slice is what a CU's load path can take at most, and the waves then
//     wait to issue them. A load has half a step or more to arrive.
//   * The 32 tiles of an XCD's patch share their rows through its L2, but in
//     step they would all wait for the same lines' first fetch, and a CU's load
//     path, which returns in order, would be full of waiting loads. So within
//     every four steps of k the tiles of a row (and of a column) of the patch
//     start at different ones: each fetches a quarter first and finds the
//     others' quarters in L2. 8192^3: 505 -> 438 us on MI355X; with eight steps
//     449, with sixteen 506 (the patch's rows no longer stay in L2).
//   * Measured, by the card and its clocks: 8192^3 into fp16 421-444 us, 2.5-2.6 PFLOP/s
//     (where it took 438, its matrix instructions alone, at the power limit, 335;
//     without loads 366); 11008 x 4096 x 4095 into fp32 312-334 us, 1.1-1.2 PFLOP/s
//     (8192^3: 787-812, 1.35-1.40), 2.69 rounds of tiles in the time of three.
//   * The loads into LDS are written as assembly, because the compiler would
//     wait for all of them at the next LDS read.
#include <algorithm>

#include "fp8.hpp"
#include "fp8_mma.hpp"
#include "schedule.hpp"

namespace iris {
namespace {

constexpr int kBK = 128;
constexpr int kGroupM = 8;     // tile rows of a patch that one XCD works on
constexpr int kPatch = 32;     // tiles of a patch: the workgroups of an XCD

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from a buffer into LDS at base + 16 * lane. m0 holds the
// base for this one instruction; nothing else here keeps a value in it.
__device__ __forceinline__ void buffer_to_lds(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(base), "v"(voff),
               "s"(rsrc), "s"(soff)
               : "memory");
}

__device__ __forceinline__ i32x4 buffer_words(const void* p) {
  const uint64_t a = (uint64_t)p;
  return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)a),
               (int)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xffffu), (int)0xfffffff0u, kRsrcWord3};
}

template <int BM, int BN>
struct Tile {
  static constexpr int SA = 3, SB = 2;                 // LDS stages of A and of B
  static constexpr int WM = BM / 2, WN = BN / 2;       // a wave's part
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_STAGE = BM * kBK, B_STAGE = BN * kBK;
  static constexpr int B_AT = SA * A_STAGE;            // LDS: [A stages | B stages]
  static constexpr int LDS = B_AT + SB * B_STAGE;
  static constexpr int LA = BM / 32, LB = BN / 32;     // loads of 1 KB per wave and step
  static constexpr int NM = FM * FN;                   // 32 x 32 blocks per wave
  static constexpr int NR = 2 * (FM + FN);             // operand reads per slice
  // Beside slice 0 of step t go A's loads of step t + SA - 1, beside slice 1 B's
  // of step t + SB. Between the two, step t + 1 has to have landed: the loads
  // that were issued since its last one and may still be under way.
  static constexpr int under_way() {
    const int a = 2 * (2 - SA), b = 2 * (1 - SB) + 1;   // when A's and B's of step t + 1 went out, in half steps
    int n = 0;
    for (int h = (a > b ? a : b) + 1; h <= 0; ++h) n += h % 2 == 0 ? LA : LB;
    return n;
  }
};

// one slice's operands: two pieces per 32-row block
template <class T>
struct Slice {
  u32x4 a[T::FM][2], b[T::FN][2];
};

template <class T_>
struct Work {
  using T = T_;

  const char* lds;
  i32x4 ra, rb;                       // codes of this tile's first rows
  uint32_t va[T::LA], vb[T::LB];      // this lane's loads, from there
  uint32_t piece;                     // their offset in a row
  uint32_t lds_wave;                  // LDS address of this wave's first load of a stage
  uint32_t at[4];                     // this lane's pieces h, 2 + h, 4 + h, 6 + h in a wave's part
  uint32_t at_a, at_b;                // that part of stage 0
  uint32_t sa[T::FM], sb[T::FN];      // scale bytes of the coming steps, the present one lowest

  // Load `item` of a step's A or B rows into the stage at `to`. In a ragged last
  // step the pieces past the row's last one read that one again (`back` bytes
  // before their place).
  __device__ __forceinline__ void load_a(int item, uint32_t k, uint32_t back, uint32_t to) const {
    buffer_to_lds(ra, va[item] - back, k, lds_wave + to + item * 32 * kBK);
  }
  __device__ __forceinline__ void load_b(int item, uint32_t k, uint32_t back, uint32_t to) const {
    buffer_to_lds(rb, vb[item] - back, k, lds_wave + T::B_AT + to + item * 32 * kBK);
  }
  __device__ __forceinline__ uint32_t back(uint32_t k, int K) const {
    return (uint32_t)max(0, (int)(k + piece + 16) - ((K + 15) & ~15));
  }
  // Zeros for the bytes past K of a ragged last step that has landed in these stages
  __device__ __forceinline__ void cut(char* l, int tail, uint32_t a_at, uint32_t b_at, int tid) const {
    const int r = tid >> 3, p = tid & 7, valid = tail - 16 * p;
    if (valid < 16) {
      char* const at0 = l + r * kBK + ((p ^ ((r >> 1) & 7)) << 4);
#pragma unroll
      for (int i = 0; i < T::LA; ++i) {
        u32x4* const q = (u32x4*)(at0 + a_at + i * 32 * kBK);
        *q = keep_bytes(*q, valid);
      }
#pragma unroll
      for (int i = 0; i < T::LB; ++i) {
        u32x4* const q = (u32x4*)(at0 + T::B_AT + b_at + i * 32 * kBK);
        *q = keep_bytes(*q, valid);
      }
    }
  }

  // operand read X of slice s: a0, b0 .. b(FN-1), a1 .., the two pieces of each in turn
  __device__ __forceinline__ void read(int x, int s, uint32_t a_at, uint32_t b_at, Slice<T>& f) const {
    const int item = x / 2, h = x & 1;
    if (item == 0 || item > T::FN) {
      const int i = item == 0 ? 0 : item - T::FN;
      f.a[i][h] = *(const u32x4*)(lds + (at_a + a_at + at[2 * s + h]) + i * 32 * kBK);
    } else {
      f.b[item - 1][h] = *(const u32x4*)(lds + (at_b + b_at + at[2 * s + h]) + (item - 1) * 32 * kBK);
    }
  }
};

// multiplies one slice; `other` is what is done beside it, in n shares
template <bool EXACT, class T, class F>
__device__ __forceinline__ void multiply(Work<T>& w, const Slice<T>& f, f32x16 (&acc)[T::FM][T::FN], F other) {
  if constexpr (!EXACT) {
#pragma unroll
    for (int k = 0; k < T::NM; ++k) {
      const int i = k / T::FN, j = k % T::FN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          pair(f.b[j][0], f.b[j][1]), pair(f.a[i][0], f.a[i][1]), acc[i][j], 0, 0, 0, (int)w.sb[j], 0, (int)w.sa[i]);
      other(k, T::NM);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8 x[T::FM], y[T::FN];
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
        x[i] = to_bf16x8(f.a[i][q / 2][2 * (q & 1)], f.a[i][q / 2][2 * (q & 1) + 1],
                         __builtin_bit_cast(float, (w.sa[i] & 0xffu) << 23));
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
        y[j] = to_bf16x8(f.b[j][q / 2][2 * (q & 1)], f.b[j][q / 2][2 * (q & 1) + 1],
                         __builtin_bit_cast(float, (w.sb[j] & 0xffu) << 23));
#pragma unroll
      for (int k = 0; k < T::NM; ++k) {
        const int i = k / T::FN, j = k % T::FN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[j], x[i], acc[i][j], 0, 0, 0);
        other(q * T::NM + k, 4 * T::NM);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// in all waves: everything read is in registers, and at most the last N loads are under way
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t rotate(uint32_t word, uint32_t bits) {
  return __builtin_amdgcn_alignbit(word, word, bits);
}

// a where the mask has ones: no branch between the matrix instructions
__device__ __forceinline__ uint32_t choose(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

// shares [k n / N, (k + 1) n / N) of n things over N places
#define IRIS_SHARE(x, n, k, N) for (int x = (k) * (n) / (N); x < ((k) + 1) * (n) / (N); ++x)

// One tile of C, or, with g.splits > 1, of one split's sum over its share of k
// (OUT is float then, C a workspace of g.splits matrices).
template <class OUT, bool EXACT, int BM, int BN>
__global__ __launch_bounds__(256) void fp8_mm_kernel(Fp8MmArgs g) {
  using T = Tile<BM, BN>;
  __shared__ __align__(16) char lds[T::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_pm = (g.M + BM - 1) / BM, n_pn = (g.N + BN - 1) / BN;
  int pm, pn;
  {
    // workgroups go to the XCDs in turn: each takes whole patches of 8 x 4 tiles
    int t = xcd_tile(kPatch, blockIdx.x % kXcds, blockIdx.x / kXcds);
    const int tiles = n_pm * n_pn;
    if (t >= tiles * g.splits) return;
    if (g.splits > 1) {
      const int split = t / tiles;
      t -= split * tiles;
      const int k0 = split * g.split_steps * kBK;
      g.A.codes += k0;
      g.B.codes += k0;
      g.A.scales += split * g.split_steps;
      g.B.scales += split * g.split_steps;
      g.K = min(g.K - k0, g.split_steps * kBK);
      g.C = (OUT*)g.C + (int64_t)split * g.M * g.ldc;
    }
    grouped(t, n_pm, n_pn, kGroupM, pm, pn);
  }
  const int m0 = pm * BM, n0 = pn * BN;
  const int wm = (wave >> 1) * T::WM, wn = (wave & 1) * T::WN;
  const int r32 = lane & 31;

  Work<T> w;
  w.lds = lds;
  w.ra = buffer_words(g.A.codes + (int64_t)m0 * g.A.ld);
  w.rb = buffer_words(g.B.codes + (int64_t)n0 * g.B.ld);
  {
    const int r = wave * 8 + (lane >> 3);
    w.piece = 16 * ((lane & 7) ^ ((r >> 1) & 7));
    // rows past the end repeat the last one: their outputs are not stored
#pragma unroll
    for (int i = 0; i < T::LA; ++i) w.va[i] = (uint32_t)(min(32 * i + r, g.M - 1 - m0) * (int)g.A.ld) + w.piece;
#pragma unroll
    for (int i = 0; i < T::LB; ++i) w.vb[i] = (uint32_t)(min(32 * i + r, g.N - 1 - n0) * (int)g.B.ld) + w.piece;
  }
  w.lds_wave = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 1024);
#pragma unroll
  for (int p = 0; p < 4; ++p) w.at[p] = r32 * kBK + (((2 * p + (lane >> 5)) ^ ((r32 >> 1) & 7)) << 4);
  w.at_a = wm * kBK;
  w.at_b = T::B_AT + wn * kBK;

  // scales: 4 steps' bytes per word
  const int nk = (g.K + kBK - 1) / kBK;
  const uint8_t *psa[T::FM], *psb[T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i) psa[i] = g.A.scales + (int64_t)min(m0 + wm + 32 * i + r32, g.M - 1) * g.A.lds;
#pragma unroll
  for (int j = 0; j < T::FN; ++j)
    psb[j] = g.B.scales + (int64_t)(min(n0 + wn + 32 * j + r32, g.N - 1) / g.b_block) * g.B.lds;

  f32x16 acc[T::FM][T::FN] = {};
  Slice<T> f0, f1;
  // the tile's bias: a value per thread, parked until the end
  float bias_v = 0.0f;
  if (g.bias) {
    const int e = tid + (g.bias_along_m ? m0 : n0);
    if (tid < (g.bias_along_m ? BM : BN) && e < (g.bias_along_m ? g.M : g.N)) bias_v = widen(((const OUT*)g.bias)[e]);
  }

  const int tail = g.K % kBK;
  // Where step t stands in the row: within each four whole steps, tiles that
  // share rows start at different ones. Steps past the last load the last one
  // again, so that the count of loads under way is the same in every step.
  const int turn = (pm + pn) & 3, nkf = g.K / kBK;
  const auto at_k = [&](int t) {
    t = min(t, nk - 1);
    return (uint32_t)((t | 3) < nkf ? (t & ~3) | ((t + turn) & 3) : t) * kBK;
  };
  // the scale bytes of the four steps from t on, in that order
  const auto turn_bits = [&](int t) { return (t | 3) < nkf ? 8 * turn : 0; };
  if (nk > 0) {
#pragma unroll
    for (int i = 0; i < T::FM; ++i) w.sa[i] = rotate(*(const uint32_t*)psa[i], turn_bits(0));
#pragma unroll
    for (int j = 0; j < T::FN; ++j) w.sb[j] = rotate(*(const uint32_t*)psb[j], turn_bits(0));
#pragma unroll
    for (int t = 0; t < T::SB || t < T::SA - 1; ++t) {
      const uint32_t k = at_k(t), back = w.back(k, g.K);
      if (t < T::SA - 1) {
#pragma unroll
        for (int i = 0; i < T::LA; ++i) w.load_a(i, k, back, t * T::A_STAGE);
      }
      if (t < T::SB) {
#pragma unroll
        for (int i = 0; i < T::LB; ++i) w.load_b(i, k, back, t * T::B_STAGE);
      }
    }
    step_barrier<(T::SA - 2) * T::LA + (T::SB - 1) * T::LB>();
    if (tail && nk == 1) {
      w.cut(lds, tail, 0, 0, tid);
      __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < T::NR; ++x) w.read(x, 0, 0, 0, f0);
  }
  uint32_t na[T::FM] = {}, nb[T::FN] = {};
  uint32_t a_free = (T::SA - 1) * T::A_STAGE, a_this = 0, a_next = T::A_STAGE, b_this = 0, b_next = T::B_STAGE;
  for (int t = 0; t < nk; ++t) {
    const uint32_t ka = at_k(t + T::SA - 1), kb = at_k(t + T::SB), back_a = w.back(ka, g.K), back_b = w.back(kb, g.K);
    const uint32_t new_word = (t & 3) == 3 ? ~0u : 0u;
    const uint32_t bits = turn_bits(t + 1);
    __builtin_amdgcn_sched_barrier(0);
    if ((t & 3) == 0 && t + 4 < nk) {
#pragma unroll
      for (int i = 0; i < T::FM; ++i) na[i] = *(const uint32_t*)(psa[i] + t + 4);
#pragma unroll
      for (int j = 0; j < T::FN; ++j) nb[j] = *(const uint32_t*)(psb[j] + t + 4);
    }
    multiply<EXACT>(w, f0, acc, [&](int k, int N) {
      IRIS_SHARE(i, T::LA, k, N) w.load_a(i, ka, back_a, a_free);
      IRIS_SHARE(x, T::NR, k, N) w.read(x, 1, a_this, b_this, f1);
    });
    // the matrix instructions above stay above (the compiler would move them
    // behind the branch, and leave the unit idle here)
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) asm volatile("" : "+a"(acc[i][j]));
    step_barrier<T::under_way()>();
    if (tail && t + 2 == nk) {
      w.cut(lds, tail, a_next, b_next, tid);
      __syncthreads();
    }
    // the scales that were loaded above are there: say so here, where it costs nothing
#pragma unroll
    for (int i = 0; i < T::FM; ++i) asm volatile("" : "+v"(na[i]));
#pragma unroll
    for (int j = 0; j < T::FN; ++j) asm volatile("" : "+v"(nb[j]));
    __builtin_amdgcn_sched_barrier(0);
    multiply<EXACT>(w, f1, acc, [&](int k, int N) {
      IRIS_SHARE(i, T::LB, k, N) w.load_b(i, kb, back_b, b_this);
      IRIS_SHARE(x, T::NR, k, N) w.read(x, 0, a_next, b_next, f0);
      // the next step's scale bytes, each behind its last use
      const int last = k - (N - T::NM);
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
        if (last == (i + 1) * T::FN - 1) w.sa[i] = choose(new_word, rotate(na[i], bits), w.sa[i] >> 8);
#pragma unroll
      for (int j = 0; j < T::FN; ++j)
        if (last == T::NM - 1) w.sb[j] = choose(new_word, rotate(nb[j], bits), w.sb[j] >> 8);
    });
    a_free = a_this;
    a_this = a_next;
    a_next = a_next == (T::SA - 1) * T::A_STAGE ? 0 : a_next + T::A_STAGE;
    b_this = b_next;
    b_next = b_next == (T::SB - 1) * T::B_STAGE ? 0 : b_next + T::B_STAGE;
  }

  // Epilogue, 32 rows of a wave at a time: the accumulators turn around in LDS
  // (B is the first operand, so a lane holds row lane % 32 of each block and, for
  // q = 0..3, its columns 8 q + 4 (lane / 32) .. + 3) and leave in whole lines,
  // with the bias and the old values added before the one rounding. The last
  // loads have to land before the LDS is used again.
  step_barrier<0>();
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
  const int64_t ldp = ((int64_t)a.N + 3) / 4 * 4;
  g.C = ws;
  g.ldc = (int32_t)ldp;
  g.bias = nullptr;
  g.accumulate = 0;
  hipError_t e = small_tile<float, EXACT>(g, plan, s);
  if (e != hipSuccess) return e;
  g = a;
  g.splits = plan.splits;
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

Fp8MmPlan fp8_mm_plan(int64_t M, int64_t N, int64_t K, bool fp32) {
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
      if (n != want) continue;
      double us = predicted(tile, n_tiles * n, share, fp32);
      if (n > 1) us += 2.5 + (double)n * M * N * 8 / 5e6;
      if (least > 0 && us >= least) continue;
      least = us;
      best.bm = tile.bm;
      best.bn = tile.bn;
      best.splits = (int)n;
      best.split_steps = (int)share;
      best.ws_bytes = n > 1 ? (size_t)n * M * ((N + 3) / 4 * 4) * 4 : 0;
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
