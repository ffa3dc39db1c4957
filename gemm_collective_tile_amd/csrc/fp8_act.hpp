// Host-side view of the 8-bit product with an activation in its epilogue.
#pragma once

#include "dropout.hpp"
#include "fp8.hpp"

namespace iris {

enum Act : uint8_t { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// What becomes of a product's sum v:
//   forward    z = v + bias;  c = residual + scale m act(z)
//   backward   c = scale m v act'(z), z given; dbias: the sums of c over the rows
// c goes to g.C and / or, in blocks of 1 x 128, to q.
struct Fp8ActArgs {
  Fp8MmArgs g;            // C NULL: not wanted; bias along N or NULL
  void* z;                // (M, N) of C's type: kept (forward, NULL: not), or read (backward)
  const void* residual;   // (M, N) of C's type, or NULL
  Fp8Mat q;               // codes NULL: not wanted
  float* dbias_part;      // sums of a tile's (or a join's) rows, `ldp` floats each, or NULL
  int32_t ldz, ldr, ldp;
  uint8_t act, backward;
  uint8_t whole;          // N is a multiple of 8, rows of C, z and residual start at multiples of 16 bytes
  DropArgs drop;          // scale: alpha / (1 - p)
};

// The product's plan; `sums`: into 32-bit sums in the workspace first, then through the
// epilogue (splits, or few rows whose epilogue needs whole blocks or columns); `parts` rows
// of partial column sums lie at part_at bytes of the workspace.
struct Fp8ActPlan {
  Fp8MmPlan mm;
  bool sums;
  int32_t parts;
  size_t part_at, ws_bytes;
};
Fp8ActPlan fp8_mm_act_plan(int64_t M, int64_t N, int64_t K, bool fp32, bool to8, bool dbias);
hipError_t launch_fp8_mm_act(const Fp8ActArgs& a, const Fp8ActPlan& plan, void* dbias, void* ws, hipStream_t s);

}  // namespace iris
