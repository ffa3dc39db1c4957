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
#pragma once

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

template <int BM_, int BN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_;
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

// The tile that this workgroup makes, or false: none. With g.splits > 1 g becomes the
// product of one split's share of k (OUT is float then, C a workspace of g.splits matrices).
template <class OUT, class T>
__device__ __forceinline__ bool pick_tile(Fp8MmArgs& g, int& pm, int& pn) {
  const int n_pm = (g.M + T::BM - 1) / T::BM, n_pn = (g.N + T::BN - 1) / T::BN;
  {
    // workgroups go to the XCDs in turn: each takes whole patches of 8 x 4 tiles
    int t = xcd_tile(kPatch, blockIdx.x % kXcds, blockIdx.x / kXcds);
    const int tiles = n_pm * n_pn;
    if (t >= tiles * g.splits) return false;
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
  return true;
}

// The sums of a tile's products over g.K, in the waves' accumulators. No
// load is under way and no wave reads the LDS any more when it returns. `first` is
// called ahead of the loop, for loads of what the caller needs at the end.
template <bool EXACT, class T, class F>
__device__ __forceinline__ void tile_sums(const Fp8MmArgs& g, char* lds, int pm, int pn, f32x16 (&acc)[T::FM][T::FN], F first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = pm * T::BM, n0 = pn * T::BN;
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

#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = f32x16{};
  Slice<T> f0, f1;
  first();

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

  step_barrier<0>();
}

}  // namespace
}  // namespace iris
