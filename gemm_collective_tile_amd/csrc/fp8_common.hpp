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

#include "device_common.hpp"

namespace iris {

constexpr int kFp8Block = 128;

// A block-scaled matrix: `ld` bytes from one row of codes to the next, `lds`
// from one row of scales to the next.
struct Fp8Mat {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, lds;
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
// 2^(127 - s): s is in [1, 247], so this is a normal number
__device__ __forceinline__ float scale_inverse(uint32_t s) { return __builtin_bit_cast(float, (254u - s) << 23); }
// 2^(s - 127) for any byte a caller may pass (0: 2^-127, subnormal; 255: NaN)
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : (s == 255 ? 0x7fc00000u : s << 23));
}

// Four values, already divided by their scale, to four e4m3 codes, each
// rounded to nearest even (v_cvt_pk_fp8_f32; values beyond the format, which
// are only infinities and NaN here, give NaN codes).
__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void from_fp8x4(uint32_t w, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
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

// C consecutive values of a row starting at p, widened; those from `valid` on
// read as 0. `vec`: p is 16-byte aligned whenever the piece is whole.
template <int C, class T>
__device__ __forceinline__ void load_piece(const T* p, int valid, bool vec, float (&v)[C]) {
  if (vec && valid >= C) {
    constexpr int W = C * (int)sizeof(T) / 16;
    static_assert(W >= 1, "piece shorter than a 16-byte load");
    u32x4 w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = ld16((const char*)p + 16 * i);
    T t[C];
    __builtin_memcpy(t, w, sizeof t);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = widen(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = i < valid ? widen(p[i]) : 0.0f;
  }
}

// C consecutive codes (C = 8 or 16) times their scale. Rows of codes start at
// multiples of 16 bytes and pieces at multiples of C, so a whole piece is one
// load; past `valid` no byte is read.
template <int C>
__device__ __forceinline__ void load_codes(const uint8_t* p, int valid, float scale, float (&v)[C]) {
  uint32_t w[C / 4];
  if (valid >= C) {
    if constexpr (C == 16)
      *(u32x4*)w = *(const u32x4*)p;
    else
      *(u32x2*)w = *(const u32x2*)p;
  } else {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      w[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (4 * i + b < valid) w[i] |= (uint32_t)p[4 * i + b] << (8 * b);
    }
  }
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    from_fp8x4(w[i], v + 4 * i);
#pragma unroll
    for (int b = 0; b < 4; ++b) v[4 * i + b] *= scale;
  }
}

// C codes to row memory, no byte past `valid`
template <int C>
__device__ __forceinline__ void store_codes(uint8_t* p, int valid, const uint32_t (&w)[C / 4]) {
  if (valid >= C) {
    if constexpr (C == 16)
      *(u32x4*)p = *(const u32x4*)w;
    else
      *(u32x2*)p = *(const u32x2*)w;
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < valid) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

template <int C>
__device__ __forceinline__ void encode_piece(const float (&v)[C], float inv, uint32_t (&w)[C / 4]) {
#pragma unroll
  for (int i = 0; i < C / 4; ++i)
    w[i] = to_fp8x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
}

template <int C>
__device__ __forceinline__ uint32_t piece_amax(const float (&v)[C]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) m = max(m, finite_bits(v[i]));
  return m;
}

// the largest over each aligned group of N lanes, in all of them
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
  for (int d = 1; d < N; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  return m;
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
