// Dropout with a mask that is computed and never stored.
//
// Value (i, j) of a matrix is dropped by a 16-bit number u(i, j) of its own: half
// j % 8 (the low half of a word first) of Philox4x32-10 (Salmon, Moraes, Dror, Shaw:
// Parallel random numbers: as easy as 1, 2, 3; SC 2011) at counter
// (j / 8, i, offset low, offset high) and key (seed low, seed high). It is kept if
// u >= t, t = 65536 p rounded, and then divided by 1 - t / 65536. The mask goes by
// the value's place alone: any kernel, split or pitch gives the same one, so what one
// operator dropped in a forward pass another drops in the backward pass.
//
// 16 bits a value, so that a thread's 8 values of a row take one call: p is held to
// 2^-17, and a kept value's factor is exact for the p that is held. A call is 20
// multiplications of 32 x 32 into 64 bits.
#pragma once

#include "fp8_common.hpp"

namespace iris {

struct DropArgs {
  uint64_t seed, offset;
  const uint64_t* offset_at;   // device: added to offset, or NULL
  uint32_t threshold;          // 0: nothing is dropped
  float scale;                 // of what is kept
};

// The words of one launch's generator, read once a thread.
struct Drop {
  uint32_t k0, k1, c2, c3, threshold;
  float scale;
  __device__ __forceinline__ explicit Drop(const DropArgs& a) {
    uint64_t offset = a.offset;
    if (a.threshold != 0 && a.offset_at) offset += *a.offset_at;
    k0 = (uint32_t)a.seed;
    k1 = (uint32_t)(a.seed >> 32);
    c2 = (uint32_t)offset;
    c3 = (uint32_t)(offset >> 32);
    threshold = a.threshold;
    scale = a.scale;
  }
  static __device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);   // a ^ b ^ c, by its truth table
  }
  // the 128 bits of columns 8 piece .. + 7 of a row
  __device__ __forceinline__ u32x4 bits(uint32_t row, uint32_t piece) const {
    uint32_t a = piece, b = row, c = c2, d = c3, x = k0, y = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t m0 = (uint64_t)a * 0xD2511F53u, m1 = (uint64_t)c * 0xCD9E8D57u;
      a = xor3((uint32_t)(m1 >> 32), b, x);
      b = (uint32_t)m1;
      c = xor3((uint32_t)(m0 >> 32), d, y);
      d = (uint32_t)m0;
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
    return u32x4{a, b, c, d};
  }
  // v: columns 8 piece .. + 7 of U rows. What is dropped becomes 0, whatever it was.
  template <int U>
  __device__ __forceinline__ void apply(const int (&row)[U], uint32_t piece, float (&v)[U][8]) const {
    if (threshold == 0) {
      if (scale == 1.0f) return;
#pragma unroll
      for (int k = 0; k < 8 * U; ++k) v[k / 8][k % 8] *= scale;
      return;
    }
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const u32x4 w = bits((uint32_t)row[r], piece);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
        v[r][i] = u >= threshold ? v[r][i] * scale : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void apply(uint32_t row, uint32_t piece, float (&v)[8]) const {
    apply<1>({(int)row}, piece, *(float (*)[1][8])&v);
  }
  // v without what is dropped, which becomes 0, as it is. Its product with a dropped gradient
  // is then 0 whatever v held, and not 0 times an infinity.
  __device__ __forceinline__ void clear(uint32_t row, uint32_t piece, float (&v)[8]) const {
    const u32x4 w = bits(row, piece);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu) >= threshold ? v[i] : 0.0f;
  }
  __device__ __forceinline__ float apply(uint32_t row, uint32_t col, float v) const {
    if (threshold == 0) return v * scale;
    const u32x4 w = bits(row, col >> 3);
    const uint32_t word = col & 4 ? (col & 2 ? w[3] : w[2]) : (col & 2 ? w[1] : w[0]);
    return ((word >> (col & 1 ? 16 : 0)) & 0xffffu) >= threshold ? v * scale : 0.0f;
  }
};

// 8 values of a row from column `col` (a multiple of 8) on, as they lie in memory; zeros
// past the last column and where a lane is off.
template <class T>
struct Raw8 {
  static constexpr int WORDS = 2 * (int)sizeof(T);
  uint32_t w[WORDS];
  // WHOLE: the row is 16-byte aligned, and all or none of the 8 are inside. Else any
  // alignment: the row's last piece is read from 8 columns before its end on and moved
  // down, so that nothing past the row is read and only that piece's wave does more.
  template <bool WHOLE>
  __device__ __forceinline__ void load(const T* row, int col, int cols, bool on = true) {
    fetch<WHOLE>(row, col, cols, on);
    settle<WHOLE>(col, cols, on);
  }
  // the same in two steps: the values are waited for in the second
  template <bool WHOLE>
  __device__ __forceinline__ void settle(int col, int cols, bool on) {
    if constexpr (WHOLE) {
      const uint32_t m = on_mask(on && col < cols);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] &= m;
    } else if (cols >= 8) {
      const int down = on ? min(col - min(col, cols - 8), 8) : 8;
      if (down > 0) move_down(down);
    }
  }
  template <bool WHOLE>
  __device__ __forceinline__ void fetch(const T* row, int col, int cols, bool on) {
    if constexpr (WHOLE) {
      const char* const at = (const char*)row + (on && col < cols ? col : 0) * (int)sizeof(T);
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i) {
        const u32x4 v = *(const u32x4*)(at + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
      }
    } else if (cols >= 8) {
      __builtin_memcpy(w, row + min(col, cols - 8), sizeof w);
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll 1
      for (int i = on && col == 0 ? cols - 1 : -1; i >= 0; --i) {   // from the last on, each pushes the others up
        T t[2] = {row[i], {}};
        uint32_t first = 0;
        __builtin_memcpy(&first, t, sizeof first);
#pragma unroll
        for (int k = WORDS - 1; k > 0; --k) w[k] = sizeof(T) == 4 ? w[k - 1] : __builtin_amdgcn_alignbit(w[k], w[k - 1], 16);
        w[0] = sizeof(T) == 4 ? first : (w[0] << 16) | first;
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    T t[8];
    __builtin_memcpy(t, w, sizeof w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = widen(t[i]);
  }

 private:
  // the values from number n (1 to 8) on become the first, zeros follow
  __device__ __forceinline__ void move_down(int n) {
    constexpr int E = 4 / (int)sizeof(T);   // values of a word
#pragma unroll
    for (int words = WORDS; words >= 1; words /= 2) {
      const uint32_t keep = on_mask((n & (words * E)) == 0);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = (w[i] & keep) | ((i + words < WORDS ? w[i + words] : 0u) & ~keep);
    }
    if constexpr (E == 2) {
      const uint32_t bits = (n & 1) * 16;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = __builtin_amdgcn_alignbit(i + 1 < WORDS ? w[i + 1] : 0u, w[i], bits);
    }
  }
};
template <bool WHOLE, class T>
__device__ __forceinline__ void load8(const T* row, int col, int cols, float (&v)[8], bool on = true) {
  Raw8<T> r;
  r.template load<WHOLE>(row, col, cols, on);
  r.values(v);
}
// 8 values to a row, each rounded once, none past the last column. WHOLE: as above
template <bool WHOLE, class T>
__device__ __forceinline__ void store8(T* row, int col, int cols, const float (&v)[8]) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) narrow(v[i], t[i]);
  const int n = cols - col;
  if constexpr (WHOLE) {
    u32x4 w[sizeof t / 16];
    __builtin_memcpy(w, t, sizeof t);
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < (int)(sizeof t / 16); ++i) ((u32x4*)(row + col))[i] = w[i];
    }
  } else if (n >= 8) {
    __builtin_memcpy(row + col, t, sizeof t);
  } else if (n > 0) {
    T* to = row + col;
    if (n & 4) {
      __builtin_memcpy(to, t, 4 * sizeof(T));
      to += 4;
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = t[4 + i];
    }
    if (n & 2) {
      __builtin_memcpy(to, t, 2 * sizeof(T));
      to += 2;
      t[0] = t[2];
    }
    if (n & 1) to[0] = t[0];
  }
}

struct DropoutArgs {
  const void *x, *residual;   // residual: NULL: none
  void* out;
  int32_t ldx, ldr, ldo;
  int32_t rows, cols;
  int32_t type, vec;          // vec: rows start at multiples of 16 bytes
  uint32_t first_row;         // of this launch's rows (set by the launch)
  DropArgs drop;
};
// with sums over the rows: shares of the rows, a row of partial sums each
struct DropoutPlan {
  int32_t share, parts, pitch;
  size_t ws_bytes;
};
DropoutPlan dropout_plan(int64_t rows, int64_t cols);
// sums: `cols` values of the type, or NULL (then plan and ws are of no account)
hipError_t launch_dropout(const DropoutArgs& a, const DropoutPlan& plan, void* sums, void* ws, hipStream_t s);

}  // namespace iris
