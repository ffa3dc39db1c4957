// The 8-bit operators that are bound by memory: the block quantiser, the
// gated activation and its backward pass.
//
// Each is one pass: every value is read once, the block's largest magnitude
// is found while the block lies in registers, and the codes are written once.
// Two shapes of kernel:
//   rows   blocks along the rows only. A thread takes 16 values of a row, the
//          8 lanes of a block agree on its scale by exchanging lanes.
//   tiles  blocks along the columns too (a transposed output, or 128 x 128
//          blocks). A workgroup takes a 128 x 128 tile, so that every block of
//          either direction lies in it. A thread holds 4 rows x 8 columns (with
//          16 columns and half the threads 4096 x 4096 of 8 bits takes 8.5 us
//          instead of 8.2, 1 x 4096 3.6 instead of 3.3); codes of 4 rows of
//          one column are one 32-bit word of the transposed tile, which turns
//          around in LDS and leaves in rows of 128 bytes.
#include <algorithm>

#include "fp8.hpp"

namespace iris {
namespace {

constexpr int kTile = 128;

// ------------------------------------------------------------------- rows

// blocks (row, kb) are numbered along the rows; 8 lanes work on each
struct RowPlace {
  int row, kb, col;
  bool on, below;   // the row is there, another one follows
  __device__ __forceinline__ RowPlace(int rows, FastDiv nkb) {
    const uint32_t b = blockIdx.x * (kThreads / 8) + threadIdx.x / 8;
    const int r = (int)nkb.div(b);
    kb = (int)(b - (uint32_t)r * nkb.d);
    col = kb * kFp8Block + 16 * (threadIdx.x & 7);
    on = r < rows;
    row = min(r, rows - 1);
    below = r < rows - 1;
  }
  __device__ __forceinline__ bool more(int ld) const { return below && ld >= 16; }
};

template <bool WHOLE>
__device__ __forceinline__ void put_row_block(const Fp8Mat& q, const RowPlace& p, int cols, const float (&v)[16]) {
  const uint32_t s = scale_byte(group_max<8>(piece_amax(v)));
  uint32_t w[4];
  encode_piece(v, scale_value(s), w);
  if (!p.on) return;
  store_codes<WHOLE, 16>(q.codes + (int64_t)p.row * q.ld, 0, p.col, cols, w);
  if ((threadIdx.x & 7) == 0) q.scales[(int64_t)p.row * q.lds + p.kb] = (uint8_t)s;
}

// Bound by memory where the matrix is large: 8192 x 16384 in bf16 69.9 us, 5.8 TB/s
// read and written (a 1 GiB copy runs at 5.1); 2048 x 4096 5.4 us; one row of
// 4096 1.75 us, of which the launch is all. Eight lanes a block and no loop, so that
// every load of a round of workgroups is under way at once.
template <class T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(const T* x, int ldx, int rows, int cols, Fp8Mat q, FastDiv nkb) {
  const RowPlace p(rows, nkb);
  float v[16];
  load_piece<WHOLE>(x + (int64_t)p.row * ldx, 0, p.col, cols, p.on, p.more(ldx), v);
  put_row_block<WHOLE>(q, p, cols, v);
}

// h = silu(g) u, and g and u kept, from one reading of both: 4096 x 11008 in bf16
// 58 us, 5.4 TB/s (memory); one row of 11008 2.0 us. h stays in 32 bits until its
// code. The three blocks follow one another in registers, each found and written
// before the next.
// KEPT: what the kernel is given of the matrices that keep gate and up (an empty
// struct if they are not wanted)
struct Kept {
  Fp8Mat gate, up;
};
struct NotKept {};

template <class T, bool WHOLE, class KEPT>
__global__ __launch_bounds__(kThreads) void fp8_swiglu_kernel(const T* gate, const T* up, int ld_gate, int ld_up, int rows,
                                                              int cols, Fp8Mat out, FastDiv nkb, KEPT kept) {
  const RowPlace p(rows, nkb);
  float g[16], u[16], h[16];
  load_piece<WHOLE>(gate + (int64_t)p.row * ld_gate, 0, p.col, cols, p.on, p.more(ld_gate), g);
  load_piece<WHOLE>(up + (int64_t)p.row * ld_up, 0, p.col, cols, p.on, p.more(ld_up), u);
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
  put_row_block<WHOLE>(out, p, cols, h);
  if constexpr (sizeof(KEPT) == sizeof(Kept)) {
    put_row_block<WHOLE>(kept.gate, p, cols, g);
    put_row_block<WHOLE>(kept.up, p, cols, u);
  }
}

// ------------------------------------------------------------------ tiles

// Tile of 128 x 128 held by T threads: thread t has columns kPiece * (t % L) .. + kPiece
// of rows 4 * (t / L) .. + 4, L = 128 / kPiece lanes side by side.
constexpr int kPiece = 8;   // columns of a thread
struct TilePlace {
  static constexpr int L = kTile / kPiece;
  static constexpr int T = L * (kTile / 4);
  uint32_t t;            // thread
  int r0, c0, ch, j;     // tile origin, piece and row group in it
  int nrows, ncols;      // of the matrix
  __device__ __forceinline__ TilePlace(int nrows, int ncols, FastDiv ncb) : nrows(nrows), ncols(ncols) {
    const uint32_t rb = ncb.div(blockIdx.x);
    r0 = (int)rb * kTile;
    c0 = (int)(blockIdx.x - rb * ncb.d) * kTile;
    t = threadIdx.x;
    ch = t % L;
    j = t / L;
  }
  // row i of this thread (rows past the end read the last one), whether it is there
  __device__ __forceinline__ uint32_t row(int i) const { return (uint32_t)min(4 * j + i, nrows - 1 - r0); }
  __device__ __forceinline__ bool on(int i) const { return r0 + 4 * j + i < nrows; }
  // another row of the matrix follows, a piece on or more
  __device__ __forceinline__ bool more(int i, int ld) const { return r0 + 4 * j + i < nrows - 1 && ld >= kPiece; }
  __device__ __forceinline__ int col() const { return kPiece * ch; }
  __device__ __forceinline__ int cols() const { return ncols - c0; }
  // Addresses: the tile's corner, the same in all threads, and a 32-bit offset
  // from it (pitches are under 2^22, so a tile's rows lie within 2^31 bytes)
  template <class U>
  __device__ __forceinline__ U* corner(U* x, int64_t ld) const { return x + (int64_t)r0 * ld + c0; }
  __device__ __forceinline__ uint8_t* scales(const Fp8Mat& q) const { return q.scales + (int64_t)r0 * q.lds + c0 / kTile; }
};
__device__ __forceinline__ uint32_t offset(uint32_t row, int64_t ld) { return __umul24(row, (uint32_t)ld); }

// LDS of up to N tiles' turn: the transposed codes and the columns' scales. The
// three arrays share no byte: put_turned relies on it from one call to the next.
template <int N>
struct TileLds {
  static constexpr int WAVES = TilePlace::T / 64;
  alignas(16) uint32_t turn[N][kTile][kTile / 4];  // [column][word of 4 rows], swizzled
  alignas(16) uint32_t part[N][WAVES][kTile];      // a wave's largest magnitude of each column
  alignas(16) float scale[N][kTile];
};

// The 16-byte pieces of a column's 128 transposed codes are permuted by the
// column, so that the words that a wave writes for its L pieces of columns and
// the pieces that it reads back spread over the banks.
__device__ __forceinline__ int turn_word(int col, int word) {
  return (((word >> 2) ^ (col / kPiece)) & 7) * 4 + (word & 3);
}

// Writes the transposed codes and scales of N tiles of values (of those whose
// codes are not NULL). All threads of the workgroup call it. given < 0: the LDS
// may be the one of an earlier call, as the same TileLds<L>: waves that are still
// there read `turn` only, which this call writes behind its second barrier, and
// `part` and `scale`, which it writes before, lie outside it. given >= 0: the scale
// byte of every block (128 x 128 blocks), already written, and no call came before.
template <int N, int L>
__device__ __forceinline__ void put_turned(const Fp8Mat (&qt)[N], const TilePlace& p, const float (&v)[N][4][kPiece],
                                           int given, TileLds<L>& lds) {
  static_assert(N <= L, "more tiles than the LDS holds");
  constexpr int T = TilePlace::T;
  const int t = p.t;
  if (given < 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t m[kPiece], top = 0;
#pragma unroll
      for (int c = 0; c < kPiece; ++c) {
        m[c] = __builtin_bit_cast(uint32_t, max_abs(max_abs(v[n][0][c], v[n][1][c]), v[n][2][c], v[n][3][c]));
        top = max(top, m[c]);
      }
      if (__builtin_expect(top >= kInfBits, 0)) {
#pragma unroll
        for (int c = 0; c < kPiece; ++c) {
          m[c] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) m[c] = max(m[c], finite_bits(v[n][i][c]));
        }
      }
      stride_max(m);
      *(u32x2*)&lds.part[n][t / 64][kPiece * p.ch + 4 * (t >> 5 & 1) + 2 * (t >> 4 & 1)] = u32x2{m[0], m[1]};
    }
    __syncthreads();
    if (t < N * kTile) {
      const int n = t / kTile, c = t % kTile;
      uint32_t a = 0;
#pragma unroll
      for (int w = 0; w < TileLds<L>::WAVES; ++w) a = max(a, lds.part[n][w][c]);
      const uint32_t b = scale_byte(a);
      lds.scale[n][c] = scale_value(b);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k == n && qt[k].codes && c < p.cols())
          qt[k].scales[(int64_t)p.c0 * qt[k].lds + p.r0 / kTile + offset(c, qt[k].lds)] = (uint8_t)b;
    }
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s[kPiece];
#pragma unroll
    for (int c = 0; c < kPiece; ++c) s[c] = scale_value((uint32_t)given);
    if (given < 0) __builtin_memcpy(s, &lds.scale[n][kPiece * p.ch], sizeof s);
#pragma unroll
    for (int c = 0; c < kPiece; ++c) {
      const int col = kPiece * p.ch + c;
      lds.turn[n][col][turn_word(col, p.j)] = to_fp8x4(v[n][0][c], v[n][1][c], v[n][2][c], v[n][3][c], s[c]);
    }
  }
  __syncthreads();
  // 8 lanes write the 128 codes of a column
  const int piece = t % 8, valid = p.nrows - p.r0 - 16 * piece;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!qt[n].codes) continue;
    uint8_t* const corner = qt[n].codes + (int64_t)p.c0 * qt[n].ld + p.r0;
#pragma unroll
    for (int k = 0; k < kTile * 8 / T; ++k) {
      const int col = k * (T / 8) + t / 8;
      const uint32_t* const w = &lds.turn[n][col][turn_word(col, 4 * piece)];
      if (col >= p.cols()) continue;
      uint8_t* const to = corner + (offset(col, qt[n].ld) + 16 * piece);
      put_bytes(to, *(const u32x4*)w, valid);
    }
  }
}

// a thread's piece of its row i, blocks along the rows
template <bool WHOLE>
__device__ __forceinline__ void put_row(const Fp8Mat& q, const TilePlace& p, int i, const float (&v)[kPiece], int given) {
  const uint32_t s = given < 0 ? scale_byte(group_max<TilePlace::L>(piece_amax(v))) : (uint32_t)given;
  uint32_t w[kPiece / 4];
  encode_piece(v, scale_value(s), w);
  if (p.on(i)) {
    store_codes<WHOLE, kPiece>(p.corner(q.codes, q.ld), offset(p.row(i), q.ld), p.col(), p.cols(), w);
    if (given < 0 && p.ch == 0) p.scales(q)[offset(p.row(i), q.lds)] = (uint8_t)s;
  }
}

// x -> rows and / or columns, or 128 x 128 blocks. Both directions of 8192 x 16384
// in bf16 111 us, 4.8 TB/s (a 1 GiB copy: 5.1); 4096 x 11008 39 us; 128 x 128 blocks
// of 11008 x 4096 in fp32, both directions, 54 us, 5.0 TB/s; 8 bits turned around,
// 4095 x 4096, 8.5 us. The small ones are one round of workgroups, which load, turn
// and store in step: what one waits for is not hidden by another. 128 x 128 is the
// least tile that holds whole blocks of both directions.
template <class T, bool WHOLE>
__global__ __launch_bounds__(TilePlace::T) void fp8_tile_kernel(Fp8QuantArgs a, FastDiv ncb) {
  __shared__ TileLds<1> lds;
  const TilePlace p(a.rows, a.cols, ncb);
  float all[1][4][kPiece];
  float(&v)[4][kPiece] = all[0];
  if constexpr (sizeof(T) == 1) {
    uint32_t w[4][kPiece / 4];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_codes<WHOLE>(p.corner(a.x8.codes, a.x8.ld), offset(p.row(i), a.x8.ld), p.col(), p.cols(), w[i]);
      const uint8_t b = p.scales(a.x8)[offset(p.row(i), a.x8.lds)];
      s[i] = scale_value(b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) decode(w[i], s[i], on_mask(p.on(i) && p.col() < p.cols()), v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_piece<WHOLE>(p.corner((const T*)a.x, a.ldx), offset(p.row(i), a.ldx), p.col(), p.cols(), p.on(i), p.more(i, a.ldx), v[i]);
  }
  int given = -1;
  if (a.block == kTile) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, piece_amax(v[i]));
    m = group_max<64>(m);
    if ((threadIdx.x & 63) == 0) lds.part[0][0][threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TileLds<1>::WAVES; ++w) m = max(m, lds.part[0][0][w]);
    given = (int)scale_byte(m);
    if (threadIdx.x == 0) {
      if (a.q.codes) a.q.scales[(int64_t)(p.r0 / kTile) * a.q.lds + p.c0 / kTile] = (uint8_t)given;
      if (a.qt.codes) a.qt.scales[(int64_t)(p.c0 / kTile) * a.qt.lds + p.r0 / kTile] = (uint8_t)given;
    }
  }
  if (a.q.codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) put_row<WHOLE>(a.q, p, i, v[i], given);
  }
  if (a.qt.codes) {
    const Fp8Mat qt[1] = {a.qt};
    put_turned(qt, p, all, given, lds);
  }
}

// One tile's inputs as they came, and their loads.
template <class T>
struct BwdInputs {
  Piece<T, kPiece> d[4];
  uint32_t g[4][kPiece / 4], u[4][kPiece / 4];
  uint8_t sg[4], su[4];
  template <bool WHOLE>
  __device__ __forceinline__ void load(const Fp8SwigluBwdArgs& a, const TilePlace& p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t row = p.row(i);
      d[i].template load<WHOLE>(p.corner((const T*)a.dh, a.ld_dh), offset(row, a.ld_dh), p.col(), p.cols(), p.on(i),
                                  p.more(i, a.ld_dh));
      load_codes<WHOLE>(p.corner(a.gate8.codes, a.gate8.ld), offset(row, a.gate8.ld), p.col(), p.cols(), g[i]);
      load_codes<WHOLE>(p.corner(a.up8.codes, a.up8.ld), offset(row, a.up8.ld), p.col(), p.cols(), u[i]);
      sg[i] = p.scales(a.gate8)[offset(row, a.gate8.lds)];
      su[i] = p.scales(a.up8)[offset(row, a.up8.lds)];
    }
  }
};

// With s = sigma(g):  h = g s u,  dgate = dh u s (1 + g (1 - s)),  dup = dh g s,
// at the kept 8-bit g and u. A result stays in registers until both directions
// of blocks have their codes. The inputs stay too, as they came; dgate and dup
// are formed first and h, for which sigma is computed again, when their
// registers are free: 113 a thread, so 4 waves fit a SIMD. All three at once
// spill at that width (4096 x 11008: 143 us against 100), and with 2 waves a SIMD,
// the next tile's loads under way, take 123; 6 waves a SIMD, the results formed one
// at a time, 164. 4096 x 11008 in bf16: 101 us, 4.0 TB/s; its loads and stores with
// nothing formed between them take 88, the vector units are busy two thirds of the
// time (40 instructions a value, two of them exp and two rcp).
template <class T, bool WHOLE>
__global__ __launch_bounds__(512, 4) void fp8_swiglu_bwd_kernel(Fp8SwigluBwdArgs a, FastDiv ncb) {
  __shared__ TileLds<2> lds;
  const TilePlace p(a.rows, a.cols, ncb);
  BwdInputs<T> in;
  in.template load<WHOLE>(a, p);
  {
    float v[2][4][kPiece];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t on = on_mask(p.on(i) && p.col() < p.cols());
      float g[kPiece], u[kPiece];
      decode(in.g[i], scale_value(in.sg[i]), on, g);
      decode(in.u[i], scale_value(in.su[i]), on, u);
#pragma unroll
      for (int c = 0; c < kPiece; ++c) {
        const float d = in.d[i].value(c), s = sigmoid(g[c]), gs = g[c] * s;
        v[0][i][c] = d * u[c] * __builtin_fmaf(gs, 1.0f - s, s);
        v[1][i][c] = d * gs;
      }
      put_row<WHOLE>(a.dgate, p, i, v[0][i], -1);
      put_row<WHOLE>(a.dup, p, i, v[1][i], -1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (a.dgate_t.codes || a.dup_t.codes) {
      const Fp8Mat qt[2] = {a.dgate_t, a.dup_t};
      put_turned(qt, p, v, -1, lds);
    }
  }
  if (a.h_t.codes) {
    float v[1][4][kPiece];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t on = on_mask(p.on(i) && p.col() < p.cols());
#pragma unroll
      for (int k = 0; k < kPiece / 4; ++k) asm volatile("" : "+v"(in.g[i][k]), "+v"(in.u[i][k]));
      float g[kPiece], u[kPiece];
      decode(in.g[i], scale_value(in.sg[i]), on, g);
      decode(in.u[i], scale_value(in.su[i]), on, u);
#pragma unroll
      for (int c = 0; c < kPiece; ++c) v[0][i][c] = g[c] * sigmoid(g[c]) * u[c];
      __builtin_amdgcn_sched_barrier(0);
    }
    const Fp8Mat qt[1] = {a.h_t};
    put_turned(qt, p, v, -1, lds);
  }
}

// One result of a tile: dgate, dup or h
template <int PART, class T, bool WHOLE>
__device__ __forceinline__ void swiglu_bwd_part(const Fp8SwigluBwdArgs& a, const TilePlace& p, TileLds<1>& lds) {
  const Fp8Mat qt[1] = {PART == 0 ? a.dgate_t : PART == 1 ? a.dup_t : a.h_t};
  if (PART == 2 && !qt[0].codes) return;
  BwdInputs<T> in;
  in.template load<WHOLE>(a, p);
  float v[1][4][kPiece];
  // a wave has 16 rows: none of them there, nothing to form (1 x 11008: 4.1 us, otherwise 6.5)
  if (p.r0 + 16 * __builtin_amdgcn_readfirstlane(p.t / 64) < p.nrows) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t on = on_mask(p.on(i) && p.col() < p.cols());
      float g[kPiece], u[kPiece];
      decode(in.g[i], scale_value(in.sg[i]), on, g);
      if constexpr (PART != 1) decode(in.u[i], scale_value(in.su[i]), on, u);
#pragma unroll
      for (int c = 0; c < kPiece; ++c) {
        const float s = sigmoid(g[c]), gs = g[c] * s;
        if constexpr (PART == 0) v[0][i][c] = in.d[i].value(c) * u[c] * __builtin_fmaf(gs, 1.0f - s, s);
        if constexpr (PART == 1) v[0][i][c] = in.d[i].value(c) * gs;
        if constexpr (PART == 2) v[0][i][c] = gs * u[c];
      }
      if constexpr (PART < 2) put_row<WHOLE>(PART == 0 ? a.dgate : a.dup, p, i, v[0][i], -1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < kPiece; ++c) v[0][i][c] = 0.0f;
  }
  if (qt[0].codes) put_turned(qt, p, v, -1, lds);
}

// The same with a workgroup for each result of a tile (blockIdx.y), for matrices of
// few tiles: the vector units of one CU take 4.4 us for all three of a tile while
// others are idle. In fp16, one workgroup a tile and three:
//     16 x 1376    7.9 us   4.3        2048 x 1920   12.7   12.4
//   1001 x 1376   11.6      8.2        2048 x 2688   17.5   15.3
//   1024 x 2048   10.4      8.4        2048 x 4096   18.6   19.7
// so as long as four workgroups a CU hold them all.
constexpr uint32_t kPartsTiles = 4 * kFp8Cus / 3;
template <class T, bool WHOLE>
__global__ __launch_bounds__(512) void fp8_swiglu_bwd_parts_kernel(Fp8SwigluBwdArgs a, FastDiv ncb) {
  __shared__ TileLds<1> lds;
  const TilePlace p(a.rows, a.cols, ncb);
  switch (blockIdx.y) {
    case 0: swiglu_bwd_part<0, T, WHOLE>(a, p, lds); break;
    case 1: swiglu_bwd_part<1, T, WHOLE>(a, p, lds); break;
    default: swiglu_bwd_part<2, T, WHOLE>(a, p, lds); break;
  }
}

uint32_t blocks_of(int n) { return (uint32_t)((n + kFp8Block - 1) / kFp8Block); }

// Calls launch(first row, rows, grid) for parts of the rows whose blocks, 8 threads
// each, are 2^31 threads at most.
template <class F>
hipError_t by_rows(int rows, uint32_t nkb, F launch) {
  const int part = (int)(((uint32_t)1 << 28) / nkb);
  for (int r = 0; r < rows;) {
    const int n = std::min(part, rows - r);
    launch(r, n, dim3(((uint32_t)n * nkb * 8 + kThreads - 1) / kThreads));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    r += n;
  }
  return hipSuccess;
}
Fp8Mat from_row(const Fp8Mat& q, int r) {
  return Fp8Mat{q.codes + (int64_t)r * q.ld, q.scales + (int64_t)r * q.lds, q.ld, q.lds};
}

// Values, types and whether all pieces of 16 are whole and aligned choose the kernel.
template <bool WHOLE>
hipError_t quantize(const Fp8QuantArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  const FastDiv d = FastDiv::make(nkb);
  if (a.block == 1 && !a.qt.codes) {
    return by_rows(a.rows, nkb, [&](int r, int rows, dim3 grid) {
#define ROWS(T)                                                                                                      \
  hipLaunchKernelGGL((fp8_rows_kernel<T, WHOLE>), grid, dim3(kThreads), 0, s, (const T*)a.x + (int64_t)r * a.ldx, a.ldx, \
                     rows, a.cols, from_row(a.q, r), d)
      switch (a.x_type) {
        case T_FP16: ROWS(f16); break;
        case T_BF16: ROWS(bf16); break;
        default: ROWS(float); break;
      }
#undef ROWS
    });
  }
  const dim3 grid(blocks_of(a.rows) * nkb), block(TilePlace::T);
  switch (a.x_type) {
    case T_FP16: hipLaunchKernelGGL((fp8_tile_kernel<f16, WHOLE>), grid, block, 0, s, a, d); break;
    case T_BF16: hipLaunchKernelGGL((fp8_tile_kernel<bf16, WHOLE>), grid, block, 0, s, a, d); break;
    case T_FP32: hipLaunchKernelGGL((fp8_tile_kernel<float, WHOLE>), grid, block, 0, s, a, d); break;
    default: hipLaunchKernelGGL((fp8_tile_kernel<uint8_t, WHOLE>), grid, block, 0, s, a, d); break;
  }
  return hipGetLastError();
}

template <class T, bool WHOLE>
hipError_t swiglu(const Fp8SwigluArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  const FastDiv d = FastDiv::make(nkb);
  return by_rows(a.rows, nkb, [&](int r, int rows, dim3 grid) {
    const T* const gate = (const T*)a.gate + (int64_t)r * a.ld_gate;
    const T* const up = (const T*)a.up + (int64_t)r * a.ld_up;
    if (a.gate8.codes)
      hipLaunchKernelGGL((fp8_swiglu_kernel<T, WHOLE, Kept>), grid, dim3(kThreads), 0, s, gate, up, a.ld_gate, a.ld_up,
                         rows, a.cols, from_row(a.h, r), d, Kept{from_row(a.gate8, r), from_row(a.up8, r)});
    else
      hipLaunchKernelGGL((fp8_swiglu_kernel<T, WHOLE, NotKept>), grid, dim3(kThreads), 0, s, gate, up, a.ld_gate, a.ld_up,
                         rows, a.cols, from_row(a.h, r), d, NotKept{});
  });
}

template <class T, bool WHOLE>
hipError_t swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  const uint32_t tiles = blocks_of(a.rows) * nkb;
  const dim3 block(TilePlace::T);
  if (tiles <= kPartsTiles)
    hipLaunchKernelGGL((fp8_swiglu_bwd_parts_kernel<T, WHOLE>), dim3(tiles, 3), block, 0, s, a, FastDiv::make(nkb));
  else
    hipLaunchKernelGGL((fp8_swiglu_bwd_kernel<T, WHOLE>), dim3(tiles), block, 0, s, a, FastDiv::make(nkb));
  return hipGetLastError();
}

}  // namespace

// The host has checked that rows * blocks fit 31 bits and the tiles one launch.
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t s) {
  return (a.x_type == T_FP8 || a.vec) && a.cols % 16 == 0 ? quantize<true>(a, s) : quantize<false>(a, s);
}

hipError_t launch_fp8_swiglu(const Fp8SwigluArgs& a, hipStream_t s) {
  if (a.vec && a.cols % 16 == 0) return a.type == T_FP16 ? swiglu<f16, true>(a, s) : swiglu<bf16, true>(a, s);
  return a.type == T_FP16 ? swiglu<f16, false>(a, s) : swiglu<bf16, false>(a, s);
}

hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s) {
  if (a.vec && a.cols % 16 == 0) return a.type == T_FP16 ? swiglu_bwd<f16, true>(a, s) : swiglu_bwd<bf16, true>(a, s);
  return a.type == T_FP16 ? swiglu_bwd<f16, false>(a, s) : swiglu_bwd<bf16, false>(a, s);
}

}  // namespace iris
