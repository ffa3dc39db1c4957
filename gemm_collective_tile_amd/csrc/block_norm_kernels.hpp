// The norms before and after a block, with the block's gate, residual scale, dropout
// and residual sum between them:
//
//   p = post ? norm(y) post_w + post_b : y
//   r = x + alpha gate m p                        (the residual stream)
//   n = norm(r) pre_w + pre_b                     (the next block's input)
//   norm(v) = (v - mean) rstd,  rstd = 1 / sqrt(mean((v - mean)^2) + eps), mean = 0 for
//   the root-mean-square kind
//
// and the backward pass of all of it. Bound by memory: a row lies in registers while
// its two norms are formed, every value is read once and written once. W waves of P
// pieces of 8 values a lane hold a row (512 W P columns at most); sums go over the
// lanes by exchanging registers, over the waves through LDS. The variance is the mean
// of squares of what the mean has been taken off, from registers, not a difference of
// two large sums. n is formed from r before r's rounding.
#pragma once

#include "block_norm.hpp"

namespace iris {
namespace {

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// the sum over the lanes, the same in all of them
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0xb1>(v);    // lane ^ 1
  v = add_dpp<0x4e>(v);    // lane ^ 2
  v = add_dpp<0x141>(v);   // 7 - lane
  v = add_dpp<0x140>(v);   // 15 - lane
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
  const uint32_t t = __builtin_bit_cast(uint32_t, v);
  const auto y = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  return __builtin_bit_cast(float, (uint32_t)y[0]) + __builtin_bit_cast(float, (uint32_t)y[1]);
}
// The sums of N numbers over the W waves of a row. `slot`: W * N floats of LDS that
// nobody reads any more; all waves of the workgroup call it together.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* slot, int w, int lane) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if constexpr (W > 1) {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) slot[k * W + w] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += slot[k * W + i];
      v[k] = s;
    }
  }
}

// 8 values of a parameter vector, of T or fp32; 0 past the last column
template <class T, bool WHOLE>
__device__ __forceinline__ void load_param(const void* p, bool f32, int col, int cols, float (&v)[8]) {
  if (f32)
    load8<WHOLE>((const float*)p, col, cols, v);
  else
    load8<WHOLE>((const T*)p, col, cols, v);
}

// values past the last column become 0
template <bool WHOLE>
__device__ __forceinline__ void cut8(int col, int cols, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = col + (WHOLE ? 0 : i) < cols ? v[i] : 0.0f;
}

// mean and rstd of a row whose values lie in v, zeros past the last column; afterwards
// v holds (v - mean) rstd, zeros there again
template <int W, int P, bool WHOLE>
__device__ __forceinline__ f32x2 normalise(float (&v)[P][8], const int (&col)[P], int cols, float inv_cols, bool layer,
                                           float eps, float* slots, int w, int lane) {
  float mean = 0.0f;
  if (layer) {
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[j][i];
    row_sums<W>(s, slots, w, lane);
    mean = s[0] * inv_cols;
#pragma unroll
    for (int j = 0; j < P; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] -= mean;
      cut8<WHOLE>(col[j], cols, v[j]);
    }
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(v[j][i], v[j][i], s[0]);
  row_sums<W>(s, slots + W, w, lane);
  const float rstd = 1.0f / __builtin_sqrtf(s[0] * inv_cols + eps);
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] *= rstd;
  return f32x2{mean, rstd};
}

// v = v (w + offset) + b, zeros past the last column
template <class T, bool WHOLE>
__device__ __forceinline__ void affine(const void* w, const void* b, bool f32, float offset, int col, int cols, float (&v)[8]) {
  float t[8];
  if (w) {
    load_param<T, WHOLE>(w, f32, col, cols, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= t[i] + offset;
  }
  if (b) {
    load_param<T, WHOLE>(b, f32, col, cols, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
}

// Rows of up to 512 columns take a wave, wider ones one for each 512 (a value read once
// and 8 of them a lane: 64 registers, so eight waves on a vector unit, hide the row's
// four round trips to memory, LDS and back), beyond 8192 columns two pieces a lane.
// 8192 x 4096 in bf16 with both norms, a gate, dropout, an fp32 stream and 8-bit n:
// 437 MB, 82 us, 5.3 TB/s, a copy's rate. 1 x 4096 in fp16 2.3 us (a launch 2.2). Rows at
// odd addresses cost the memory path more: 1023 x 4093 9.4-10.5 us, 1024 x 4096 8.1.
template <class T, class X, int W, int P, bool WHOLE>
__global__ __launch_bounds__(W < 4 ? 256 : W * 64, P == 1 ? 8 : 4) void block_norm_kernel(NormArgs a, float inv_cols, FastDiv gate_rows) {
  constexpr int RG = W < 4 ? 4 / W : 1;   // rows of a workgroup
  __shared__ float slots[RG][4][W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / W, w = wave % W;
  const int at = blockIdx.x * RG + sub, row = min(at, a.rows - 1);
  const bool on = at < a.rows;
  int col[P];
#pragma unroll
  for (int j = 0; j < P; ++j) col[j] = 8 * ((j * W + w) * 64 + lane);
  float v[P][8];
  if (a.y) {
    float p[P][8];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      load8<WHOLE>((const T*)a.y + (int64_t)row * a.ldy, col[j], a.cols, p[j]);
      load8<WHOLE>((const X*)a.x + (int64_t)row * a.ldx, col[j], a.cols, v[j]);
    }
    f32x2 stat{0.0f, 0.0f};
    if (a.p.post) {
      stat = normalise<W, P, WHOLE>(p, col, a.cols, inv_cols, a.p.layer, a.p.eps, slots[sub][0], w, lane);
#pragma unroll
      for (int j = 0; j < P; ++j)
        affine<T, WHOLE>(a.p.post_w, a.p.post_b, a.p.param32, a.p.w_offset, col[j], a.cols, p[j]);
    }
    if (a.stats && on && w == 0 && lane == 0) *(f32x2*)(a.stats + 4 * (int64_t)row) = stat;
    const Drop drop(a.p.drop);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      drop.apply(a.first_row + row, (uint32_t)col[j] >> 3, p[j]);
      if (a.p.gate) {
        const int64_t skip = (int64_t)gate_rows.div(a.first_row + row) * a.p.ld_gate * (a.p.gate32 ? 4 : (int)sizeof(T));
        float g[8];
        load_param<T, WHOLE>((const char*)a.p.gate + skip, a.p.gate32, col[j], a.cols, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[j][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += p[j][i];
      if (a.r && on) store8<WHOLE>((X*)a.r + (int64_t)row * a.ldr, col[j], a.cols, v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < P; ++j)
      load8<WHOLE>((const X*)a.x + (int64_t)row * a.ldx, col[j], a.cols, v[j]);
    if (a.stats && on && w == 0 && lane == 0) *(f32x2*)(a.stats + 4 * (int64_t)row) = f32x2{0.0f, 0.0f};
  }
  if (!a.n && !a.q.codes && !a.stats) return;
  const f32x2 stat = normalise<W, P, WHOLE>(v, col, a.cols, inv_cols, a.p.layer, a.p.eps, slots[sub][2], w, lane);
  if (a.stats && on && w == 0 && lane == 0) *(f32x2*)(a.stats + 4 * (int64_t)row + 2) = stat;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    affine<T, WHOLE>(a.p.pre_w, a.p.pre_b, a.p.param32, a.p.w_offset, col[j], a.cols, v[j]);
    if (a.n && on) store8<WHOLE>((T*)a.n + (int64_t)row * a.ldn, col[j], a.cols, v[j]);
    if (a.q.codes) {
      const uint32_t s = scale_byte(group_max<16>(piece_amax(v[j])));
      uint32_t c[2];
      encode_piece(v[j], scale_value(s), c);
      if (on) {
        store_codes<WHOLE, 8>(a.q.codes + (int64_t)row * a.q.ld, 0, col[j], a.cols, c);
        if ((lane & 15) == 0 && col[j] < a.cols) a.q.scales[(int64_t)row * a.q.lds + col[j] / kFp8Block] = (uint8_t)s;
      }
    }
  }
}

// BIAS: dpre_b or dpost_b is wanted (16 registers a piece more).
//
// A workgroup's rows: RG of them at a time, each by W of its waves.
//
// With hat = (r - mean) rstd, a = dn pre_w and means over the row:
//   t = dr + rstd (a - mean(a) - hat mean(a hat))             the gradient of r, and so of x
//   d = alpha gate m t                                        of p
//   hat_y = (y - mean_y) rstd_y, c = d post_w
//   dy = rstd_y (c - mean(c) - hat_y mean(c hat_y))           or d, without a norm after the block
// (the root-mean-square kind has no mean(a), mean(c)) and, over the rows,
//   dpre_w = sum dn hat, dpre_b = sum dn, dgate = sum alpha m t p, dpost_w = sum d hat_y, dpost_b = sum d.
// A thread keeps the sums of its columns in registers over all the workgroup's rows;
// they go to the workspace once, a row for every workgroup, and block_norm_join adds
// those in order: no atomics, the same bits every time. dgate's sums end with each
// group of rows that shares a gate; a group that lies in one workgroup is done there,
// what a workgroup has of its first and of its last other group goes to the workspace.
//
// Bound by memory: 4096 x 4096 in bf16 with both norms, a gate, dropout and fp32 streams,
// 302 MB and 12 MB of partial sums, 69 us (4.6 TB/s) and 4.0 to join them. A row is a chain
// of loads, two reductions over the waves and stores; the next row's loads go out ahead
// of it, and the parameters stay in registers, as a load of them would be waited for
// behind the next row's (without either, two workgroups a CU with 128 registers: 74 and
// 6.2). 333 x 1376 in fp16 as a layer norm with all gradients 9.5 us and 2.8.
template <class T, class X, int W, int P, bool WHOLE, bool BIAS>
__global__ __launch_bounds__(64 * norm_bwd_waves(W), norm_bwd_ahead(W, WHOLE) ? 2 : 4) void block_norm_bwd_kernel(
    NormBwdArgs a, float inv_cols, FastDiv gate_rows) {
  constexpr int WAVES = norm_bwd_waves(W), RG = WAVES / W, WIDE = W * 512 * P;
  constexpr bool AHEAD = norm_bwd_ahead(W, WHOLE);   // 256 registers a lane: the next row is under way while one is worked on
  __shared__ float slots[2][2][RG][2 * W];   // by turns, so that a row's sums are read before the next row's but one are written
  __shared__ __align__(16) float comb[RG > 1 ? 4 * RG * WIDE : 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / W, w = wave % W;
  const int first = blockIdx.x * a.wg_rows, last = min(first + a.wg_rows, a.rows);
  const int64_t pitch = (a.cols + 7) & ~7;
  int col[P];
#pragma unroll
  for (int j = 0; j < P; ++j) col[j] = 8 * ((j * W + w) * 64 + lane);

  // sums of the row groups' columns, each to one row of floats (or nowhere: NULL), N at a time
  const auto put_sums = [&](auto n_of, const float (*const (&s)[4])[8], float* const (&to)[4]) {
    constexpr int N = decltype(n_of)::value;
    if constexpr (RG == 1) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!to[k]) continue;
#pragma unroll
        for (int j = 0; j < P; ++j) store8<false>(to[k], col[j], a.cols, s[k][j]);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!to[k]) continue;
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *(f32x4*)(comb + (k * RG + sub) * WIDE + col[j] + 4 * h) =
                f32x4{s[k][j][4 * h], s[k][j][4 * h + 1], s[k][j][4 * h + 2], s[k][j][4 * h + 3]};
      }
      __syncthreads();
      for (int c = 4 * threadIdx.x; c < a.cols; c += 256 * WAVES) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (!to[k]) continue;
          f32x4 v = *(const f32x4*)(comb + k * RG * WIDE + c);
#pragma unroll
          for (int g = 1; g < RG; ++g) v += *(const f32x4*)(comb + (k * RG + g) * WIDE + c);
          if (c + 4 <= a.cols)
            __builtin_memcpy(to[k] + c, &v, 16);
          else
            for (int e = 0; c + e < a.cols; ++e) to[k][c + e] = v[e];
        }
      }
    }
  };

  // AHEAD: the next row, as it lies in memory
  struct {
    f32x4 st;   // mean and rstd of y, of r
    Raw8<T> y, dn;
    Raw8<X> dr, r;
  } in;
  const auto fetch = [&](int base, int end) {
    const int row = min(base + sub, end - 1);
    const bool on = base + sub < end;
    in.st = *(const f32x4*)(a.stats + 4 * (int64_t)row);
    if (a.dn) {
      in.dn.template fetch<WHOLE>((const T*)a.dn + (int64_t)row * a.ld_dn, col[0], a.cols, on);
      in.r.template fetch<WHOLE>((const X*)a.r + (int64_t)row * a.ld_r, col[0], a.cols, on);
    }
    if (a.dr) in.dr.template fetch<WHOLE>((const X*)a.dr + (int64_t)row * a.ld_dr, col[0], a.cols, on);
    if (a.y) in.y.template fetch<WHOLE>((const T*)a.y + (int64_t)row * a.ld_y, col[0], a.cols, on);
  };
  // v times a weight's columns, with a bias's; times a row of gates
  const auto times_weight = [&](const void* w, const void* b, int j, float (&v)[8]) {
    affine<T, WHOLE>(w, b, a.p.param32, a.p.w_offset, col[j], a.cols, v);
  };
  const auto times_gate = [&](uint32_t group, int j, float (&v)[8]) {
    if (!a.p.gate) return;
    float g[8];
    load_param<T, WHOLE>((const char*)a.p.gate + (int64_t)group * a.p.ld_gate * (a.p.gate32 ? 4 : (int)sizeof(T)), a.p.gate32,
                         col[j], a.cols, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i];
  };

  float s_pre_w[P][8] = {}, s_pre_b[P][8] = {}, s_post_w[P][8] = {}, s_post_b[P][8] = {}, s_gate[P][8] = {};
  float pre_w[8], post_w[8], post_b[8], gate[8];   // AHEAD: held over the rows
  const auto fill = [](float (&v)[8], float with) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = with;
  };
  const auto group_end = [&](int row0) {
    const int64_t g1 = a.p.gate ? ((int64_t)gate_rows.div(row0) + 1) * a.p.rows_per_gate : last;
    return g1 < last ? (int)g1 : last;
  };
  if constexpr (AHEAD) {
    if (first < last) fetch(first, group_end(first));
    fill(pre_w, 1.0f), fill(post_w, 1.0f), fill(post_b, 0.0f);
    times_weight(a.p.pre_w, nullptr, 0, pre_w);
    times_weight(a.p.post_w, nullptr, 0, post_w);
    if (a.dgate) times_weight(nullptr, a.p.post_b, 0, post_b);
  }
  const Drop drop(a.p.drop);
  int turn = 0;
  for (int row0 = first; row0 < last;) {
    const uint32_t group = a.p.gate ? gate_rows.div(row0) : 0;
    const int64_t g0 = (int64_t)group * a.p.rows_per_gate, g1 = g0 + a.p.rows_per_gate;
    const int end = AHEAD ? group_end(row0) : a.p.gate && g1 < last ? (int)g1 : last;
    if constexpr (AHEAD) {
      fill(gate, 1.0f);
      times_gate(group, 0, gate);
    }
    for (int base = row0; base < end; base += RG, turn ^= 1) {
      const int at = base + sub, row = min(at, end - 1);
      const bool on = at < end;
      f32x4 st;
      Raw8<T> y[P];
      float t[P][8], hat[P][8], d[P][8];
      if constexpr (AHEAD) {
        st = in.st;
        if (a.dn) {
          in.dn.template settle<WHOLE>(col[0], a.cols, on);
          in.r.template settle<WHOLE>(col[0], a.cols, on);
          in.dn.values(d[0]);
          in.r.values(hat[0]);
        }
        if (a.dr) {
          in.dr.template settle<WHOLE>(col[0], a.cols, on);
          in.dr.values(t[0]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[0][i] = 0.0f;
        }
        if (a.y) {
          in.y.template settle<WHOLE>(col[0], a.cols, on);
          y[0] = in.y;
        }
        const int next = base + RG < end ? base + RG : end;
        if (next < last) fetch(next, next < end ? end : group_end(next));
      } else {
        st = *(const f32x4*)(a.stats + 4 * (int64_t)row);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (a.y) y[j].template load<WHOLE>((const T*)a.y + (int64_t)row * a.ld_y, col[j], a.cols, on);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (a.dr) {
            load8<WHOLE>((const X*)a.dr + (int64_t)row * a.ld_dr, col[j], a.cols, t[j], on);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[j][i] = 0.0f;
          }
        }
      }
      if (a.dn) {
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if constexpr (!AHEAD) {
            load8<WHOLE>((const T*)a.dn + (int64_t)row * a.ld_dn, col[j], a.cols, d[j], on);
            load8<WHOLE>((const X*)a.r + (int64_t)row * a.ld_r, col[j], a.cols, hat[j], on);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            hat[j][i] = (hat[j][i] - st[2]) * st[3];
            s_pre_w[j][i] = __builtin_fmaf(d[j][i], hat[j][i], s_pre_w[j][i]);
            if (BIAS) s_pre_b[j][i] += d[j][i];
          }
          if constexpr (!AHEAD) times_weight(a.p.pre_w, nullptr, j, d[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (AHEAD) d[j][i] *= pre_w[i];
            s[0] += d[j][i];
            s[1] = __builtin_fmaf(d[j][i], hat[j][i], s[1]);
          }
        }
        row_sums<W>(s, slots[turn][0][sub], w, lane);
        const float m0 = a.p.layer ? s[0] * inv_cols : 0.0f, m1 = s[1] * inv_cols;
#pragma unroll
        for (int j = 0; j < P; ++j) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] += st[3] * (d[j][i] - m0 - hat[j][i] * m1);
          cut8<WHOLE>(col[j], a.cols, t[j]);
        }
      }
      if (a.dx && on) {
#pragma unroll
        for (int j = 0; j < P; ++j) store8<WHOLE>((X*)a.dx + (int64_t)row * a.ld_dx, col[j], a.cols, t[j]);
      }
      if (!a.y) continue;
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < P; ++j) {
        y[j].values(hat[j]);
        drop.apply((uint32_t)row, (uint32_t)col[j] >> 3, t[j]);
        if (a.p.post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) hat[j][i] = (hat[j][i] - st[0]) * st[1];
        }
        if (a.dgate) {
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = AHEAD ? __builtin_fmaf(hat[j][i], post_w[i], post_b[i]) : hat[j][i];
          if constexpr (!AHEAD) times_weight(a.p.post_w, a.p.post_b, j, p);
          // y as it is, without a norm that would spread it over the row: what is dropped has no say. The mask
          // is computed again for the rare piece that holds something not finite, so that others pay 8
          // products for it (kept from above for all, it took 2 % at 4096 x 4096 and 10 % of ragged rows with biases).
          if (!a.p.post && drop.threshold != 0) {
            float zero = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) zero = __builtin_fmaf(p[i], 0.0f, zero);
            if (zero != 0.0f) drop.clear((uint32_t)row, (uint32_t)col[j] >> 3, p);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s_gate[j][i] = __builtin_fmaf(t[j][i], p[i], s_gate[j][i]);
        }
        if constexpr (!AHEAD) times_gate(group, j, t[j]);
        if constexpr (AHEAD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] *= gate[i];
        }
        if (a.p.post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s_post_w[j][i] = __builtin_fmaf(t[j][i], hat[j][i], s_post_w[j][i]);
            if (BIAS) s_post_b[j][i] += t[j][i];
          }
          if constexpr (!AHEAD) times_weight(a.p.post_w, nullptr, j, t[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (AHEAD) t[j][i] *= post_w[i];
            s[0] += t[j][i];
            s[1] = __builtin_fmaf(t[j][i], hat[j][i], s[1]);
          }
        }
      }
      if (a.p.post) {
        row_sums<W>(s, slots[turn][1][sub], w, lane);
        const float m0 = a.p.layer ? s[0] * inv_cols : 0.0f, m1 = s[1] * inv_cols;
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] = st[1] * (t[j][i] - m0 - hat[j][i] * m1);
      }
      if (a.dy && on) {
#pragma unroll
        for (int j = 0; j < P; ++j) store8<WHOLE>((T*)a.dy + (int64_t)row * a.ld_dy, col[j], a.cols, t[j]);
      }
    }
    if (a.dgate) {
      const bool here = g0 >= first && (g1 <= last || last == a.rows);
      float* const to = here ? a.dgate + (int64_t)group * a.cols
                             : a.part + ((int64_t)4 * a.wgs + 2 * blockIdx.x + (row0 == first ? 0 : 1)) * pitch;
      put_sums(std::integral_constant<int, 1>{}, {s_gate, nullptr, nullptr, nullptr}, {to, nullptr, nullptr, nullptr});
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_gate[j][i] = 0.0f;
    }
    row0 = end;
  }
  float* const outs[4] = {a.dpre_w, a.dpre_b, a.dpost_w, a.dpost_b};
  float* to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    to[k] = !outs[k] || (!BIAS && k % 2 == 1) ? nullptr : a.wgs == 1 ? outs[k] : a.part + ((int64_t)k * a.wgs + blockIdx.x) * pitch;
  put_sums(std::integral_constant<int, 4>{}, {s_pre_w, s_pre_b, s_post_w, s_post_b}, {to[0], to[1], to[2], to[3]});
}

// launch(waves of a row, pieces of a lane)
template <class F>
void by_width(int cols, F launch) {
  using std::integral_constant;
  if (cols <= 512) launch(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (cols <= 1024) launch(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  else if (cols <= 2048) launch(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (cols <= 4096) launch(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (cols <= 8192) launch(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else launch(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

template <class T, class X, bool WHOLE>
hipError_t norm_of(const NormArgs& args, hipStream_t s) {
  const float inv = 1.0f / (float)args.cols;
  const FastDiv gates = FastDiv::make((uint32_t)args.p.rows_per_gate);
  constexpr int kRows = 1 << 20;   // rows of a launch: its threads are counted in 32 bits
  for (int r = 0; r < args.rows; r += kRows) {
    NormArgs a = args;
    a.rows = args.rows - r < kRows ? args.rows - r : kRows;
    a.first_row = (uint32_t)r;
    a.x = (const X*)args.x + (int64_t)r * a.ldx;
    if (a.y) a.y = (const T*)args.y + (int64_t)r * a.ldy;
    if (a.r) a.r = (X*)args.r + (int64_t)r * a.ldr;
    if (a.n) a.n = (T*)args.n + (int64_t)r * a.ldn;
    if (a.q.codes) a.q.codes += (int64_t)r * a.q.ld, a.q.scales += (int64_t)r * a.q.lds;
    if (a.stats) a.stats += 4 * (int64_t)r;
    const auto launch = [&](auto waves, auto pieces) {
      constexpr int W = decltype(waves)::value, P = decltype(pieces)::value, RG = W < 4 ? 4 / W : 1;
      hipLaunchKernelGGL((block_norm_kernel<T, X, W, P, WHOLE>), dim3((a.rows + RG - 1) / RG), dim3(RG * W * 64), 0, s, a,
                         inv, gates);
    };
    by_width(a.cols, launch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T, class X, bool WHOLE>
hipError_t norm_bwd_of(const NormBwdArgs& a, hipStream_t s) {
  const float inv = 1.0f / (float)a.cols;
  const FastDiv gates = FastDiv::make((uint32_t)a.p.rows_per_gate);
  by_width(a.cols, [&](auto waves, auto pieces) {
    constexpr int W = decltype(waves)::value, P = decltype(pieces)::value;
    const dim3 grid(a.wgs), block(64 * norm_bwd_waves(W));
    if (a.dpre_b || a.dpost_b)
      hipLaunchKernelGGL((block_norm_bwd_kernel<T, X, W, P, WHOLE, true>), grid, block, 0, s, a, inv, gates);
    else
      hipLaunchKernelGGL((block_norm_bwd_kernel<T, X, W, P, WHOLE, false>), grid, block, 0, s, a, inv, gates);
  });
  return hipGetLastError();
}

}  // namespace

template <class T>
hipError_t launch_norm(const NormArgs& a, bool stream32, bool whole, hipStream_t s) {
  if (stream32) return whole ? norm_of<T, float, true>(a, s) : norm_of<T, float, false>(a, s);
  return whole ? norm_of<T, T, true>(a, s) : norm_of<T, T, false>(a, s);
}
template <class T>
hipError_t launch_norm_bwd(const NormBwdArgs& a, bool stream32, bool whole, hipStream_t s) {
  if (stream32) return whole ? norm_bwd_of<T, float, true>(a, s) : norm_bwd_of<T, float, false>(a, s);
  return whole ? norm_bwd_of<T, T, true>(a, s) : norm_bwd_of<T, T, false>(a, s);
}

}  // namespace iris
