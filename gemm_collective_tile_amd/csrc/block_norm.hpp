// Host-side view of the block norms: what their launches take.
#pragma once

#include "dropout.hpp"
#include "fp8.hpp"

namespace iris {

constexpr int kNormMaxCols = 16384;
// Waves of a backward workgroup whose rows W waves hold each. 8 of them with 256 registers
// a lane where rows are whole, up to 4096 columns: the parameters and the next row fit.
// 16 a compute unit, with 128 each, where they don't, and for ragged rows, which gain
// nothing (4096 x 4096 in bf16 with fp32 streams 79.5 us with 128, 73.3 with 256; 2048 x
// 8192 78.4 with 128, 88.0 with 256; 4095 x 4093, streams in bf16, 63.4 and 73.4).
constexpr int norm_bwd_waves(int W) { return W < 8 ? 8 : W; }
constexpr bool norm_bwd_ahead(int W, bool whole) { return W <= 8 && whole; }

// Parameters of the norms: weights and biases are of y's type or (param32) fp32, the gate too (gate32).
struct NormParams {
  const void *pre_w, *pre_b, *post_w, *post_b, *gate;
  int32_t ld_gate;
  int32_t rows_per_gate;      // > 0
  float eps, w_offset;
  uint8_t layer, post, param32, gate32;
  DropArgs drop;              // scale: alpha / (1 - p)
};

struct NormArgs {
  const void *x, *y;          // y: NULL: none
  void *r, *n;                // NULL: not wanted
  Fp8Mat q;                   // codes NULL: not wanted
  float* stats;               // rows x 4, or NULL
  int32_t ldx, ldy, ldr, ldn;
  int32_t rows, cols;
  uint32_t first_row;         // of this launch's rows
  NormParams p;
};

struct NormBwdArgs {
  const void *dn, *dr, *r, *y;  // dn, dr, y: NULL: none
  const float* stats;
  void *dx, *dy;
  float *dpre_w, *dpre_b, *dpost_w, *dpost_b, *dgate;  // NULL: not wanted
  int32_t ld_dn, ld_dr, ld_r, ld_y, ld_dx, ld_dy;
  int32_t rows, cols;
  int32_t wg_rows, wgs;         // rows of a workgroup, workgroups
  float* part;                  // their sums of columns
  NormParams p;
};

// Workgroups share the rows in equal, contiguous shares, in steps of the rows that a
// workgroup works on at a time.
struct NormBwdPlan {
  int wgs, wg_rows;
  size_t ws_bytes;
};
NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols, bool whole);

// by the type of y (T), the stream's (x, r: fp32 or T) and whether all rows are whole and aligned
template <class T>
hipError_t launch_norm(const NormArgs& a, bool stream32, bool whole, hipStream_t s);
template <class T>
hipError_t launch_norm_bwd(const NormBwdArgs& a, bool stream32, bool whole, hipStream_t s);
hipError_t launch_norm_join(const NormBwdArgs& a, hipStream_t s);

}  // namespace iris
