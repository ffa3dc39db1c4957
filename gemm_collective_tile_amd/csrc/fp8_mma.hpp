// Pieces that the 8-bit products share: operands of the matrix instructions
// and the last steps of an output.
#pragma once

#include "fp8_common.hpp"

namespace iris {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes times a scale (its bits: byte << 23). Exact under bytes 3 to 246: the last
// bit of a code is 2^-9, bf16's last subnormal bit 2^-133 (which the matrix
// instructions take), and 448 * 2^119 is below 2^128.
__device__ __forceinline__ bf16x8 to_bf16x8(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// bytes of a 16-byte piece from `valid` on become 0
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, int valid) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = valid - 4 * i;
    v[i] = n >= 4 ? v[i] : (n <= 0 ? 0u : v[i] & ((1u << (8 * n)) - 1u));
  }
  return v;
}

__device__ __forceinline__ i32x8 pair(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// 16 bytes per lane from global memory into LDS: lane l's go to base + 16 l
// (base is the same in all lanes; lanes that are off load nothing). Complete
// after wait_loads.
__device__ __forceinline__ void load_to_lds(const uint8_t* src, char* base) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)base, 16, 0, 0);
}
// until at most N of this wave's vector loads are under way
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// until this wave's LDS reads are in registers
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// V values of a row of C: biases and old values added, then the one rounding.
// `left`: columns from here to the row's end (> 0). C has its type's alignment
// only, which one wide access of a piece does not mind (C with 8191 columns, 8192 deep:
// 485 us value by value, 436 so).
template <int V, class OUT>
__device__ __forceinline__ void put_row_piece(OUT* c, int left, int accumulate, float bm, const float (&bn)[V],
                                              float (&v)[V]) {
  constexpr int BYTES = V * (int)sizeof(OUT);
  static_assert(BYTES == 16 || BYTES == 8, "");
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] += bn[e] + bm;
  OUT o[V];
  if (left >= V) {
    if (accumulate) {
      __builtin_memcpy(o, c, BYTES);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += widen(o[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) narrow(v[e], o[e]);
    __builtin_memcpy(c, o, BYTES);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < left) {
        if (accumulate) v[e] += widen(c[e]);
        narrow(v[e], c[e]);
      }
  }
}

// one value of C
template <class OUT>
__device__ __forceinline__ void put_output(OUT* c, float v, const OUT* bias, int64_t bias_at, int accumulate) {
  if (bias) v += widen(bias[bias_at]);
  if (accumulate) v += widen(*c);
  narrow(v, *c);
}

}  // namespace iris
