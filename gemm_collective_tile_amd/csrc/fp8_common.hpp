// Device-side pieces shared by the 8-bit operators: the block scale, the
// conversions to and from e4m3, and loads and stores of short row pieces.
//
// Format. A block-scaled matrix holds one e4m3 code per entry (OCP form: no
// infinity, 0x7f / 0xff are NaN, largest value 448) and one scale byte s per
// block, standing for 2^(s - 127). Blocks run along the row: 1 x 128 or
// 128 x 128 entries, the last ones of a row or column may be shorter. The
// scales are powers of two because that is what v_mfma_scale_f32_* applies
// to its operands as it multiplies (one byte per 32 values along k, four
// equal bytes for a block of 128): the product then needs no work of its own
// for the scales. It also makes the quantiser exact up to its one rounding:
// x / 2^e is exact in 32 bits.
//
// Scale of a block: the smallest power of two that brings the largest finite
// magnitude to 448 or less, at least 2^-126; 1 for a block of zeros.
// Infinities and NaN become NaN codes and do not count for the scale, so an
// overflowed gradient shows in every sum that it enters and its neighbours in
// the block keep their precision.
#pragma once
#include <type_traits>

#include "device_common.hpp"

namespace iris {

constexpr int kFp8Block = 128;

// A block-scaled matrix: `ld` bytes from one row of codes to the next, `lds`
// from one row of scales to the next (pitches are at most 2^22; kernels' arguments
// are kept short, the host writes them for every launch: 0.6 us for 200 bytes
// more).
struct Fp8Mat {
  uint8_t* codes;
  uint8_t* scales;
  int32_t ld, lds;
};

struct bf16 {
  uint16_t bits;
};

// magnitude bits of a 32-bit float, 0 for an infinity or NaN
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
// The bits of non-negative floats order as the floats do, so the running
// largest magnitude is kept as an integer: no NaN can get into it.

// scale byte of a block whose largest finite magnitude has these bits:
// 448 = 1.75 * 2^8, so a mantissa above 1.75 needs the next power of two
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax_bits == 0 ? 127u : (uint32_t)(e < 1 ? 1 : e);
}
// 2^(s - 127) for any byte a caller may pass (0: 2^-127, subnormal; 255: NaN)
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : (s == 255 ? 0x7fc00000u : s << 23));
}

// Four values over their scale (a power of two), to four e4m3 codes, each
// rounded to nearest even (v_cvt_scalef32_pk_fp8_f32 divides and rounds at
// once; |value / scale| <= 448 but for infinities and NaN, which give NaN codes).
__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d, float scale) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  i16x2 w;
  asm("" : "=v"(w));   // both halves are written below
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// four codes times a scale (a power of two), exactly
__device__ __forceinline__ void from_fp8x4(uint32_t w, float scale, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
  const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

__device__ __forceinline__ float widen(f16 v) { return (float)v; }
__device__ __forceinline__ float widen(bf16 v) { return __builtin_bit_cast(float, (uint32_t)v.bits << 16); }
__device__ __forceinline__ float widen(float v) { return v; }

// one rounding, to nearest even
__device__ __forceinline__ void narrow(float v, f16& o) { o = (f16)v; }
__device__ __forceinline__ void narrow(float v, float& o) { o = v; }
__device__ __forceinline__ void narrow(float v, bf16& o) {
  o.bits = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// all bits where `on`, and not a condition to the compiler, which would branch on it
__device__ __forceinline__ uint32_t on_mask(bool on) {
  uint32_t m = on ? ~0u : 0u;
  asm("" : "+v"(m));
  return m;
}

// 16 bytes at any multiple of 2 or 4
typedef uint32_t u32x4_at_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at_4 __attribute__((ext_vector_type(4), aligned(4)));

// C consecutive values of a row, as they came. WHOLE: the row's pieces are whole
// and 16-byte aligned. A piece at `col` has its values from cols - col on as zeros.
// `row` is the offset of the row's first value from `x`, `more`: another row of the
// matrix follows, at least C values on, so that a ragged piece may be read whole
// (into that row, in the matrix's own memory) and cut. Only the last row's ragged
// piece is read value by value: nothing past the matrix's last value is read.
template <class T, int C>
struct Piece {
  static constexpr int N = C * (int)sizeof(T) / 4;
  uint32_t w[N];
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(float, w[i]);
    } else {
      const uint16_t h = (uint16_t)(w[i / (4 / sizeof(T))] >> (16 * (i & 1)));
      return widen(__builtin_bit_cast(T, h));
    }
  }
  template <bool WHOLE>
  __device__ __forceinline__ void load(const T* x, uint32_t row, int col, int cols, bool on, bool more) {
    // a piece that is off reads the row's first one and drops it: no branch
    // between the loads
    static_assert(N % 4 == 0, "piece shorter than a 16-byte load");
    on = on && col < cols;
    const uint32_t at = row + (on ? col : 0), m = on_mask(on);
    const char* const first = (const char*)x + at * (uint32_t)sizeof(T);
    if constexpr (WHOLE) {
      take<u32x4>(first);
    } else {
      const int n = cols - (on ? col : 0);   // values up to the row's end
      if (n >= C || more) {
        take<std::conditional_t<sizeof(T) == 2, u32x4_at_2, u32x4_at_4>>(first);
      } else {
        T t[C];
#pragma unroll
        for (int i = 0; i < C; ++i) t[i] = x[at + min(i, n - 1)];
        __builtin_memcpy(w, t, sizeof t);
      }
      if (n < C) {
        constexpr int E = 4 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int k = n - E * i;   // values of this word inside the row
          w[i] &= k >= E ? ~0u : (k <= 0 ? 0u : 0xffffu);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] &= m;
  }

 private:
  template <class U>
  __device__ __forceinline__ void take(const char* x) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = *(const U*)(x + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
    }
  }
};
// The values, any signalling NaN quiet: the maxima below drop the neighbour of a
// signalling one. Conversion from fp16 has that effect, bf16 and fp32 come as they
// are (one instruction a value; computed values are quiet by themselves).
template <bool WHOLE, int C, class T>
__device__ __forceinline__ void load_piece(const T* x, uint32_t row, int col, int cols, bool on, bool more,
                                           float (&v)[C]) {
  Piece<T, C> p;
  p.template load<WHOLE>(x, row, col, cols, on, more);
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = std::is_same_v<T, f16> ? p.value(i) : __builtin_canonicalizef(p.value(i));
}

// 8 consecutive codes. Rows of codes start at multiples of 16 bytes, which are
// allocated up to the next one, so a piece is one load. Codes past the row's
// last one become zeros.
template <bool WHOLE>
__device__ __forceinline__ void load_codes(const uint8_t* x, uint32_t row, int col, int cols, uint32_t (&w)[2]) {
  const uint8_t* p = x + (row + (col < cols ? col : 0));
  *(u32x2*)w = *(const u32x2*)p;
  if constexpr (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = cols - col - 4 * i;   // codes of this word inside the row
      w[i] = n >= 4 ? w[i] : (n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u));
    }
  }
}
// their values; all zeros where the mask is
__device__ __forceinline__ void decode(const uint32_t (&w)[2], float scale, uint32_t on, float (&v)[8]) {
  from_fp8x4(w[0] & on, scale, v);
  from_fp8x4(w[1] & on, scale, v + 4);
}

// the first n of at most 16 bytes to a multiple of 16 (n <= 0: none)
__device__ __forceinline__ void put_bytes(uint8_t* to, u32x4 w, int n) {
  if (n >= 16) {
    *(u32x4*)to = w;
    return;
  }
  if (n <= 0) return;
  if (n & 8) {
    *(u32x2*)to = u32x2{w[0], w[1]};
    w = u32x4{w[2], w[3], 0, 0};
    to += 8;
  }
  if (n & 4) {
    *(uint32_t*)to = w[0];
    w[0] = w[1];
    to += 4;
  }
  if (n & 2) {
    *(uint16_t*)to = (uint16_t)w[0];
    w[0] >>= 16;
    to += 2;
  }
  if (n & 1) *to = (uint8_t)w[0];
}
// C codes (8 or 16) to a row, none past its last column
template <bool WHOLE, int C>
__device__ __forceinline__ void store_codes(uint8_t* x, uint32_t row, int col, int cols, const uint32_t (&w)[C / 4]) {
  if (WHOLE ? col < cols : col + C <= cols) {
    if constexpr (C == 16)
      *(u32x4*)(x + (row + col)) = *(const u32x4*)w;
    else
      *(u32x2*)(x + (row + col)) = *(const u32x2*)w;
  } else if constexpr (!WHOLE) {
    u32x4 v{w[0], w[1], 0, 0};
    if constexpr (C == 16) v = *(const u32x4*)w;
    put_bytes(x + (row + col), v, cols - col);
  }
}

template <int C>
__device__ __forceinline__ void encode_piece(const float (&v)[C], float scale, uint32_t (&w)[C / 4]) {
#pragma unroll
  for (int i = 0; i < C / 4; ++i) w[i] = to_fp8x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], scale);
}

// Largest magnitudes, as bits. v_max3_f32 takes two values at once and their
// magnitudes for free, and passes over a quiet NaN (values are quiet here, see
// load_piece: at a signalling NaN it would pass over the other value as well). An
// infinity, or nothing but NaN, leaves something that is not finite, and only
// then are the values looked at one by one.
__device__ __forceinline__ float max_abs(float a, float b) {
  float m;
  asm("v_max_f32 %0, |%1|, |%2|" : "=v"(m) : "v"(a), "v"(b));
  return m;
}
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  asm("v_max3_f32 %0, |%1|, |%2|, %0" : "+v"(m) : "v"(a), "v"(b));
  return m;
}
constexpr uint32_t kInfBits = 0x7f800000u;

template <int C>
__device__ __forceinline__ uint32_t piece_amax(const float (&v)[C]) {
  float f = max_abs(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < C; i += 2) f = max_abs(f, v[i], v[i + 1]);
  uint32_t m = __builtin_bit_cast(uint32_t, f);
  if (__builtin_expect(m >= kInfBits, 0)) {
    m = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) m = max(m, finite_bits(v[i]));
  }
  return m;
}

// the larger of this lane's and another lane's (0, what a lane outside gives, loses)
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t m) {
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xf, 0xf, true));
}
// the largest over each aligned group of N lanes, in all of them
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  static_assert(N == 8 || N == 16 || N == 64, "");
  m = max_dpp<0xb1>(m);    // lane ^ 1
  m = max_dpp<0x4e>(m);    // lane ^ 2
  m = max_dpp<0x141>(m);   // 7 - lane: the other four of eight
  if constexpr (N >= 16) m = max_dpp<0x140>(m);  // 15 - lane
  if constexpr (N == 64) {
    const auto x = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max((uint32_t)x[0], (uint32_t)x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max((uint32_t)y[0], (uint32_t)y[1]);
  }
  return m;
}

// For 8 numbers, the largest over the lanes l, l + 16, l + 32, l + 48 of the wave.
// One swap of two registers' halves and one maximum reduce both registers; what
// is left in m[0] and m[1] is that of the numbers 4 * (lane / 32) +
// 2 * (lane / 16 % 2) + 0 and 1.
__device__ __forceinline__ void stride_max(uint32_t (&m)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const auto r = __builtin_amdgcn_permlane32_swap(m[c], m[c + 4], false, false);
    m[c] = max((uint32_t)r[0], (uint32_t)r[1]);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const auto r = __builtin_amdgcn_permlane16_swap(m[c], m[c + 2], false, false);
    m[c] = max((uint32_t)r[0], (uint32_t)r[1]);
  }
}

// silu and its derivative from sigma(g) = 1 / (1 + 2^(-g log2 e)). v_exp_f32
// and v_rcp_f32 are good to an ulp, and the product's rounding adds |g| / 2
// of them: under 1e-5 relative for any g whose sigmoid is not 0 or 1, four
// hundred times finer than half a step of the e4m3 codes the results become.
// A large negative g gives 2^x = inf and sigma = 0.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

}  // namespace iris
