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
//          either direction lies in it. A thread holds 4 rows x 16 columns (8
//          columns where three values per entry are alive); codes of 4 rows of
//          one column are one 32-bit word of the transposed tile, which turns
//          around in LDS and leaves in rows of 128 bytes.
#include "fp8.hpp"

namespace iris {
namespace {

constexpr int kTile = 128;

// ------------------------------------------------------------------- rows

// blocks (row, kb) are numbered along the rows; 8 lanes work on each
struct RowPlace {
  int row, kb, col, valid;
  bool on;
};
__device__ __forceinline__ RowPlace row_place(int rows, int cols, FastDiv nkb) {
  const uint32_t b = blockIdx.x * (kThreads / 8) + threadIdx.x / 8;
  RowPlace p;
  p.row = (int)nkb.div(b);
  p.kb = (int)(b - (uint32_t)p.row * nkb.d);
  p.col = p.kb * kFp8Block + 16 * (threadIdx.x & 7);
  p.on = p.row < rows;
  p.valid = p.on ? max(0, min(16, cols - p.col)) : 0;
  return p;
}

__device__ __forceinline__ void put_row_block(const Fp8Mat& q, const RowPlace& p, const float (&v)[16]) {
  const uint32_t s = scale_byte(group_max<8>(piece_amax(v)));
  uint32_t w[4];
  encode_piece(v, scale_inverse(s), w);
  if (!p.on) return;
  store_codes<16>(q.codes + (int64_t)p.row * q.ld + p.col, p.valid, w);
  if ((threadIdx.x & 7) == 0) q.scales[(int64_t)p.row * q.lds + p.kb] = (uint8_t)s;
}

template <class T>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(Fp8QuantArgs a, FastDiv nkb) {
  const RowPlace p = row_place(a.rows, a.cols, nkb);
  float v[16];
  load_piece<16>((const T*)a.x + (int64_t)p.row * a.ldx + p.col, p.valid, a.vec, v);
  put_row_block(a.q, p, v);
}

template <class T>
__global__ __launch_bounds__(kThreads) void fp8_swiglu_kernel(Fp8SwigluArgs a, FastDiv nkb) {
  const RowPlace p = row_place(a.rows, a.cols, nkb);
  float g[16], u[16], h[16];
  load_piece<16>((const T*)a.gate + (int64_t)p.row * a.ld_gate + p.col, p.valid, a.vec, g);
  load_piece<16>((const T*)a.up + (int64_t)p.row * a.ld_up + p.col, p.valid, a.vec, u);
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
  put_row_block(a.h, p, h);
  if (a.gate8.codes) {
    put_row_block(a.gate8, p, g);
    put_row_block(a.up8, p, u);
  }
}

// ------------------------------------------------------------------ tiles

// Tile of 128 x 128 held by T threads: thread t has columns C * (t % L) .. + C
// of rows 4 * (t / L) .. + 4, L = 128 / C lanes side by side.
template <int C>
struct TilePlace {
  static constexpr int L = kTile / C;
  static constexpr int T = L * (kTile / 4);
  int r0, c0, ch, j;     // tile origin, piece and row group in it
  int rows, cols;        // rows and columns of the tile inside the matrix
  __device__ __forceinline__ TilePlace(int nrows, int ncols, FastDiv ncb) {
    const uint32_t rb = ncb.div(blockIdx.x);
    r0 = (int)rb * kTile;
    c0 = (int)(blockIdx.x - rb * ncb.d) * kTile;
    ch = threadIdx.x % L;
    j = threadIdx.x / L;
    rows = min(kTile, nrows - r0);
    cols = min(kTile, ncols - c0);
  }
  __device__ __forceinline__ int row(int i) const { return r0 + 4 * j + i; }
  __device__ __forceinline__ int col() const { return c0 + C * ch; }
  // valid columns of this thread's piece in its row i
  __device__ __forceinline__ int valid(int i) const {
    return 4 * j + i < rows ? max(0, min(C, cols - C * ch)) : 0;
  }
};

// LDS of a tile's turn: the transposed codes and the columns' scales
template <int C>
struct TileLds {
  static constexpr int WAVES = TilePlace<C>::T / 64;
  alignas(16) uint32_t turn[kTile][kTile / 4];  // [column][word of 4 rows], swizzled
  uint32_t part[WAVES][kTile];      // a wave's largest magnitude of each column
  float inv[kTile];
};

// The 16-byte pieces of a column's 128 transposed codes are permuted by the
// column, so that the words that a wave writes for its L pieces of columns and
// the pieces that it reads back spread over the banks.
template <int C>
__device__ __forceinline__ int turn_word(int col, int word) {
  return (((word >> 2) ^ (col / C)) & 7) * 4 + (word & 3);
}

// Writes the tile's transposed codes and scales. All threads of the workgroup
// call it; starts and ends with the LDS free for the next use only after a
// barrier of the caller's (it begins with one).
// given >= 0: the scale byte of every block (128 x 128 blocks).
template <int C>
__device__ void put_turned(const Fp8Mat& qt, const TilePlace<C>& p, const float (&v)[4][C], int given,
                           TileLds<C>& lds) {
  constexpr int T = TilePlace<C>::T, L = TilePlace<C>::L;
  const int t = threadIdx.x;
  __syncthreads();
  float inv[C];
  if (given < 0) {
    uint32_t m[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      m[c] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m[c] = max(m[c], finite_bits(v[i][c]));
    }
    // over the wave's 64 / L row groups: lanes t, t + L, t + 2 L, ...
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int d = L; d < 64; d *= 2) m[c] = max(m[c], (uint32_t)__shfl_xor((int)m[c], d));
    }
    if ((t & 63) < L) {
#pragma unroll
      for (int c = 0; c < C; ++c) lds.part[t / 64][C * p.ch + c] = m[c];
    }
    __syncthreads();
    if (t < kTile) {
      uint32_t a = 0;
#pragma unroll
      for (int w = 0; w < TileLds<C>::WAVES; ++w) a = max(a, lds.part[w][t]);
      const uint32_t s = scale_byte(a);
      lds.inv[t] = scale_inverse(s);
      if (t < p.cols) qt.scales[(int64_t)(p.c0 + t) * qt.lds + p.r0 / kTile] = (uint8_t)s;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) inv[c] = lds.inv[C * p.ch + c];
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) inv[c] = scale_inverse((uint32_t)given);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = C * p.ch + c;
    lds.turn[col][turn_word<C>(col, p.j)] =
        to_fp8x4(v[0][c] * inv[c], v[1][c] * inv[c], v[2][c] * inv[c], v[3][c] * inv[c]);
  }
  __syncthreads();
  // 8 lanes write the 128 codes of a column
#pragma unroll
  for (int n = 0; n < kTile * 8 / T; ++n) {
    const int col = n * (T / 8) + t / 8, piece = t % 8;
    uint32_t w[4];
    *(u32x4*)w = *(const u32x4*)&lds.turn[col][turn_word<C>(col, 4 * piece)];
    if (col < p.cols)
      store_codes<16>(qt.codes + (int64_t)(p.c0 + col) * qt.ld + p.r0 + 16 * piece, max(0, min(16, p.rows - 16 * piece)), w);
  }
}

// a thread's four row pieces, blocks along the rows
template <int C>
__device__ __forceinline__ void put_rows(const Fp8Mat& q, const TilePlace<C>& p, const float (&v)[4][C], int given) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s =
        given < 0 ? scale_byte(group_max<TilePlace<C>::L>(piece_amax(v[i]))) : (uint32_t)given;
    uint32_t w[C / 4];
    encode_piece(v[i], scale_inverse(s), w);
    const int valid = p.valid(i);
    if (4 * p.j + i < p.rows) {
      store_codes<C>(q.codes + (int64_t)p.row(i) * q.ld + p.col(), valid, w);
      if (given < 0 && p.ch == 0) q.scales[(int64_t)p.row(i) * q.lds + p.c0 / kTile] = (uint8_t)s;
    }
  }
}

// x -> rows and / or columns, or 128 x 128 blocks
template <class T>
__global__ __launch_bounds__(256) void fp8_tile_kernel(Fp8QuantArgs a, FastDiv ncb) {
  constexpr int C = 16;
  __shared__ TileLds<C> lds;
  const TilePlace<C> p(a.rows, a.cols, ncb);
  float v[4][C];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int valid = p.valid(i);
    if constexpr (sizeof(T) == 1) {
      float s = 0.0f;
      if (valid > 0) s = scale_value(a.x8.scales[(int64_t)p.row(i) * a.x8.lds + p.c0 / kTile]);
      load_codes<C>(a.x8.codes + (int64_t)p.row(i) * a.x8.ld + p.col(), valid, s, v[i]);
    } else {
      load_piece<C>((const T*)a.x + (int64_t)p.row(i) * a.ldx + p.col(), valid, a.vec, v[i]);
    }
  }
  int given = -1;
  if (a.block == kTile) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, piece_amax(v[i]));
    m = group_max<64>(m);
    if ((threadIdx.x & 63) == 0) lds.part[0][threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TileLds<C>::WAVES; ++w) m = max(m, lds.part[0][w]);
    given = (int)scale_byte(m);
    if (threadIdx.x == 0) {
      if (a.q.codes) a.q.scales[(int64_t)(p.r0 / kTile) * a.q.lds + p.c0 / kTile] = (uint8_t)given;
      if (a.qt.codes) a.qt.scales[(int64_t)(p.c0 / kTile) * a.qt.lds + p.r0 / kTile] = (uint8_t)given;
    }
  }
  if (a.q.codes) put_rows<C>(a.q, p, v, given);
  if (a.qt.codes) put_turned<C>(a.qt, p, v, given, lds);
}

// With s = sigma(g):  h = g s u,  dgate = dh u s (1 + g (1 - s)),  dup = dh g s,
// at the kept 8-bit g and u. Three values per entry stay in registers until
// both directions of blocks have their codes.
template <class T>
__global__ __launch_bounds__(512) void fp8_swiglu_bwd_kernel(Fp8SwigluBwdArgs a, FastDiv ncb) {
  constexpr int C = 8;
  __shared__ TileLds<C> lds;
  const TilePlace<C> p(a.rows, a.cols, ncb);
  float dg[4][C], du[4][C], h[4][C];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int valid = p.valid(i);
    const int64_t row = p.row(i);
    float sg = 0.0f, su = 0.0f;
    if (valid > 0) {
      sg = scale_value(a.gate8.scales[row * a.gate8.lds + p.c0 / kTile]);
      su = scale_value(a.up8.scales[row * a.up8.lds + p.c0 / kTile]);
    }
    float d[C], g[C], u[C];
    load_piece<C>((const T*)a.dh + row * a.ld_dh + p.col(), valid, a.vec, d);
    load_codes<C>(a.gate8.codes + row * a.gate8.ld + p.col(), valid, sg, g);
    load_codes<C>(a.up8.codes + row * a.up8.ld + p.col(), valid, su, u);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float s = sigmoid(g[c]), silu = g[c] * s;
      dg[i][c] = d[c] * u[c] * (s * (1.0f + g[c] * (1.0f - s)));
      du[i][c] = d[c] * silu;
      h[i][c] = silu * u[c];
    }
  }
  put_rows<C>(a.dgate, p, dg, -1);
  put_rows<C>(a.dup, p, du, -1);
  if (a.dgate_t.codes) put_turned<C>(a.dgate_t, p, dg, -1, lds);
  if (a.dup_t.codes) put_turned<C>(a.dup_t, p, du, -1, lds);
  if (a.h_t.codes) put_turned<C>(a.h_t, p, h, -1, lds);
}

uint32_t blocks_of(int n) { return (uint32_t)((n + kFp8Block - 1) / kFp8Block); }

}  // namespace

// The host has checked that rows * blocks and the tiles fit 31 bits.
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  if (a.block == 1 && !a.qt.codes) {
    const FastDiv d = FastDiv::make(nkb);
    const uint32_t grid = (uint32_t)(((uint64_t)a.rows * nkb * 8 + kThreads - 1) / kThreads);
    switch (a.x_type) {
      case T_FP16: hipLaunchKernelGGL((fp8_rows_kernel<f16>), dim3(grid), dim3(kThreads), 0, s, a, d); break;
      case T_BF16: hipLaunchKernelGGL((fp8_rows_kernel<bf16>), dim3(grid), dim3(kThreads), 0, s, a, d); break;
      default: hipLaunchKernelGGL((fp8_rows_kernel<float>), dim3(grid), dim3(kThreads), 0, s, a, d); break;
    }
    return hipGetLastError();
  }
  const FastDiv d = FastDiv::make(nkb);
  const dim3 grid(blocks_of(a.rows) * nkb), block(TilePlace<16>::T);
  switch (a.x_type) {
    case T_FP16: hipLaunchKernelGGL((fp8_tile_kernel<f16>), grid, block, 0, s, a, d); break;
    case T_BF16: hipLaunchKernelGGL((fp8_tile_kernel<bf16>), grid, block, 0, s, a, d); break;
    case T_FP32: hipLaunchKernelGGL((fp8_tile_kernel<float>), grid, block, 0, s, a, d); break;
    default: hipLaunchKernelGGL((fp8_tile_kernel<uint8_t>), grid, block, 0, s, a, d); break;
  }
  return hipGetLastError();
}

hipError_t launch_fp8_swiglu(const Fp8SwigluArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  const FastDiv d = FastDiv::make(nkb);
  const uint32_t grid = (uint32_t)(((uint64_t)a.rows * nkb * 8 + kThreads - 1) / kThreads);
  if (a.type == T_FP16)
    hipLaunchKernelGGL((fp8_swiglu_kernel<f16>), dim3(grid), dim3(kThreads), 0, s, a, d);
  else
    hipLaunchKernelGGL((fp8_swiglu_kernel<bf16>), dim3(grid), dim3(kThreads), 0, s, a, d);
  return hipGetLastError();
}

hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s) {
  const uint32_t nkb = blocks_of(a.cols);
  const FastDiv d = FastDiv::make(nkb);
  const dim3 grid(blocks_of(a.rows) * nkb), block(TilePlace<8>::T);
  if (a.type == T_FP16)
    hipLaunchKernelGGL((fp8_swiglu_bwd_kernel<f16>), grid, block, 0, s, a, d);
  else
    hipLaunchKernelGGL((fp8_swiglu_bwd_kernel<bf16>), grid, block, 0, s, a, d);
  return hipGetLastError();
}

}  // namespace iris
