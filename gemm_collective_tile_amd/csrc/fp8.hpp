// Host-side view of the 8-bit operators' kernels: what each launch takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_common.hpp"

namespace iris {

// A launch's threads are counted in 32 bits (beyond, the count wraps without an error).
constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 1;     // tiles of 128 x 128, 512 threads each
constexpr int64_t kMaxMmTiles = ((int64_t)1 << 24) - 256; // of a product, 256 threads each, in rounds of 256

enum Fp8Type : int32_t { T_FP16 = 1, T_BF16 = 2, T_FP32 = 3, T_FP8 = 4 };

struct Fp8MmArgs {
  Fp8Mat A, B;
  const void* bias;       // in C's type, or NULL
  void* C;
  int32_t ldc;            // elements
  int32_t M, N, K;
  int32_t splits, split_steps;  // set by launch_fp8_mm
  uint8_t b_block;        // rows of B per scale row: 1 or 128
  uint8_t bias_along_m;
  uint8_t accumulate;     // add to C's old values
  uint8_t c_type;
};
// How a product runs: its tile, and over how many workgroups the contraction of
// one tile is split (their sums go through ws_bytes of workspace).
struct Fp8MmPlan {
  int32_t bm = 256, bn = 256, splits = 1, split_steps = 0;   // bm 0: the kernel for few rows
  size_t ws_bytes = 0;
};
Fp8MmPlan fp8_mm_plan(int64_t M, int64_t N, int64_t K, bool fp32);
hipError_t launch_fp8_mm(const Fp8MmArgs& a, const Fp8MmPlan& plan, void* ws, hipStream_t s);
constexpr int kFp8Cus = 256;   // compute units of the chip
// Few rows of A (at most kFp8FewRows): blocks of 16 rows of B for a workgroup. From
// 17 rows of A on its time goes with what a CU loads, B's rows and A's once
// for every workgroup, so the least of (workgroups a CU gets) * (blocks of both).
// Up to kFp8AlwaysFew rows this kernel always runs: one order of sums for any N.
constexpr int kFp8AlwaysFew = 64, kFp8FewRows = 96;
inline int64_t fp8_few_loads(int64_t M, int64_t N, int nb) {
  return ((N + 16 * nb - 1) / (16 * nb) + kFp8Cus - 1) / kFp8Cus * (16 * nb + M);
}
inline int fp8_few_blocks(int64_t M, int64_t N) {
  int best = 1;
  if (M > 16)
    for (int nb = 2; nb <= 3; ++nb)
      if (fp8_few_loads(M, N, nb) < fp8_few_loads(M, N, best)) best = nb;
  return best;
}
hipError_t launch_fp8_mm_few(const Fp8MmArgs& a, hipStream_t s);

struct Fp8QuantArgs {
  const void* x;          // fp16, bf16 or fp32 values with a row pitch of ldx elements
  int32_t ldx;
  Fp8Mat x8;              // or 8-bit values with 1 x 128 blocks (x_type T_FP8)
  int32_t x_type;
  int32_t block;          // 1: blocks of 1 x 128, 128: of 128 x 128
  int32_t vec;            // whole pieces of x are 16-byte aligned
  Fp8Mat q, qt;           // codes NULL: not wanted
  int32_t rows, cols;
};
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t s);

struct Fp8SwigluArgs {
  const void *gate, *up;
  int32_t ld_gate, ld_up;
  int32_t type, vec;
  Fp8Mat h, gate8, up8;   // gate8, up8: codes NULL: not wanted
  int32_t rows, cols;
};
hipError_t launch_fp8_swiglu(const Fp8SwigluArgs& a, hipStream_t s);

struct Fp8SwigluBwdArgs {
  const void* dh;
  int32_t ld_dh;
  int32_t type, vec;
  Fp8Mat gate8, up8, dgate, dup, dgate_t, dup_t, h_t;  // the transposed ones: codes NULL: not wanted
  int32_t rows, cols;
};
hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s);

}  // namespace iris
