// Entry points of what lies between a block's products and its residual stream: dropout,
// the norms, and the 8-bit product with an activation in its epilogue. Argument checks
// (all of them before any HIP call) and launches.
#include <cmath>

#include "block_norm.hpp"
#include "dropout.hpp"
#include "fp8_act.hpp"
#include "fp8_checks.hpp"

namespace {

// the generator's place, and the factor of what is kept
int check_drop(const iris_drop_t* d, float alpha, iris::DropArgs* out) {
  *out = iris::DropArgs{};
  if (!std::isfinite(alpha)) return fail(IRIS_ERR_INVALID_ARG, "alpha must be finite");
  out->scale = alpha;
  if (!d) return IRIS_OK;
  if (!(d->p >= 0.0 && d->p < 1.0)) return fail(IRIS_ERR_INVALID_ARG, "dropout: p must be in [0, 1) (got %g)", d->p);
  const double t = std::rint(d->p * 65536.0);
  if (t > 65535.0) return fail(IRIS_ERR_INVALID_ARG, "dropout: p rounds to 1 at 16 bits (got %.17g)", d->p);
  if ((uintptr_t)d->offset_at % 8 != 0) return fail(IRIS_ERR_ALIGNMENT, "dropout: offset_at is not 8-byte aligned");
  out->seed = d->seed;
  out->offset = d->offset;
  out->offset_at = d->offset_at;
  out->threshold = (uint32_t)t;
  out->scale = (float)((double)alpha * 65536.0 / (65536.0 - t));
  if (!std::isfinite(out->scale)) return fail(IRIS_ERR_INVALID_ARG, "dropout: alpha / (1 - p) leaves 32 bits (alpha %g)", (double)alpha);
  return IRIS_OK;
}

int check_rows(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0)
    return fail(IRIS_ERR_INVALID_ARG, "rows and cols must not be negative (got %lld, %lld)", (long long)rows, (long long)cols);
  if (rows > (1 << 30) || cols > kMaxPitch)
    return fail(IRIS_ERR_UNSUPPORTED, "matrix too large (limits: 2^30 rows, 2^22 columns)");
  return IRIS_OK;
}

// a matrix that may be absent
int check_optional(const void* x, int32_t type, int64_t ld, int64_t rows, int64_t cols, const char* name) {
  return x ? check_plain(x, type, true, ld, rows, cols, name) : IRIS_OK;
}

int check_vector(const void* x, int32_t type, const char* name) {
  if (x && (uintptr_t)x % type_bytes(type) != 0) return fail(IRIS_ERR_ALIGNMENT, "%s is not aligned to its type", name);
  return IRIS_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return IRIS_OK;
  if (bytes < need) return fail(IRIS_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", bytes, need);
  if ((uintptr_t)workspace % 256 != 0) return fail(IRIS_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return IRIS_OK;
}

int check_norm(const iris_norm_t* p, bool y, int64_t rows, int64_t cols, iris::NormParams* out) {
  if (!p) return fail(IRIS_ERR_INVALID_ARG, "norm is NULL");
  if (p->kind != IRIS_NORM_RMS && p->kind != IRIS_NORM_LAYER)
    return fail(IRIS_ERR_INVALID_ARG, "norm: unknown kind %d", p->kind);
  if (p->type != IRIS_TYPE_FP16 && p->type != IRIS_TYPE_BF16)
    return fail(IRIS_ERR_INVALID_ARG, "norm: type %d is not served here", p->type);
  const struct {
    int32_t type;
    const char* name;
  } types[] = {{p->stream_type, "stream_type"}, {p->param_type, "param_type"}, {p->gate_type, "gate_type"}};
  for (const auto& t : types)
    if (t.type != p->type && t.type != IRIS_TYPE_FP32)
      return fail(IRIS_ERR_INVALID_ARG, "norm: %s must be type or fp32 (got %d)", t.name, t.type);
  if (!(p->eps > 0.0f) || !std::isfinite(p->eps)) return fail(IRIS_ERR_INVALID_ARG, "norm: eps must be positive");
  if (!std::isfinite(p->w_offset)) return fail(IRIS_ERR_INVALID_ARG, "norm: w_offset must be finite");
  if (cols > iris::kNormMaxCols)
    return fail(IRIS_ERR_UNSUPPORTED, "norm: %lld columns (limit %d)", (long long)cols, iris::kNormMaxCols);
  if (rows > 0 && cols > 0 && !y && (p->post || p->gate || p->drop))
    return fail(IRIS_ERR_INVALID_ARG, "a norm after the block, a gate and dropout need y");
  if (!p->post && (p->post_w || p->post_b)) return fail(IRIS_ERR_INVALID_ARG, "norm: post_w and post_b need post");
  int st;
  if ((st = check_vector(p->pre_w, p->param_type, "pre_w")) || (st = check_vector(p->pre_b, p->param_type, "pre_b")) ||
      (st = check_vector(p->post_w, p->param_type, "post_w")) || (st = check_vector(p->post_b, p->param_type, "post_b")) ||
      (st = check_vector(p->gate, p->gate_type, "gate")) || (st = check_drop(p->drop, p->alpha, &out->drop)))
    return st;
  int64_t every = rows > 0 ? rows : 1;
  if (p->gate) {
    if (p->rows_per_gate < 1) return fail(IRIS_ERR_INVALID_ARG, "norm: rows_per_gate must be positive");
    every = p->rows_per_gate < every ? p->rows_per_gate : every;
    const int64_t groups = (rows + every - 1) / every;
    if ((st = check_plain(p->gate, p->gate_type, true, groups > 1 ? p->ld_gate : cols, rows, cols, "gate"))) return st;
    out->ld_gate = groups > 1 ? (int32_t)p->ld_gate : (int32_t)cols;
  }
  out->pre_w = p->pre_w;
  out->pre_b = p->pre_b;
  out->post_w = p->post_w;
  out->post_b = p->post_b;
  out->gate = p->gate;
  out->rows_per_gate = (int32_t)every;
  out->eps = p->eps;
  out->w_offset = p->w_offset;
  out->layer = p->kind == IRIS_NORM_LAYER;
  out->post = p->post != 0;
  out->param32 = p->param_type == IRIS_TYPE_FP32;
  out->gate32 = p->gate_type == IRIS_TYPE_FP32;
  return IRIS_OK;
}

bool aligned16(const void* x) { return (uintptr_t)x % 16 == 0; }

// a NULL matrix is no hindrance to 16-byte accesses
bool rows16_or_none(const void* x, int64_t ld, int32_t type, int64_t rows) {
  return !x || (rows > 1 ? rows16(x, ld, type) : aligned16(x));
}

// whether every row and vector can be read and written in whole, aligned pieces of 8
bool params16(const iris_norm_t* p, const iris::NormParams& n, int64_t rows) {
  return aligned16(p->pre_w) && aligned16(p->pre_b) && aligned16(p->post_w) && aligned16(p->post_b) &&
         rows16_or_none(p->gate, n.ld_gate, p->gate_type, rows > n.rows_per_gate ? 2 : 1);
}

int check_mm(int32_t c_type, const iris_fp8_t* A, const iris_fp8_t* B, int64_t M, int64_t N, int64_t K, int32_t act) {
  int st;
  if ((st = check_mm_dims(M, N, K))) return st;
  if (c_type != IRIS_TYPE_FP16 && c_type != IRIS_TYPE_BF16 && c_type != IRIS_TYPE_FP32)
    return fail(IRIS_ERR_INVALID_ARG, "C: type %d is not served here", c_type);
  if (act < IRIS_ACT_NONE || act > IRIS_ACT_SILU) return fail(IRIS_ERR_INVALID_ARG, "unknown activation %d", act);
  if ((st = check_blocks1(A, M, K, "A")) || (st = check_fp8(B, N, K, "B"))) return st;
  if ((st = check_scale_words(A, M, K, "A")) || (st = check_scale_words(B, N, K, "B"))) return st;
  return IRIS_OK;
}

iris::Fp8ActArgs mm_args(void* C, int32_t c_type, int64_t ldc, const iris_fp8_t* A, const iris_fp8_t* B, int64_t M, int64_t N,
                         int64_t K, int32_t act) {
  iris::Fp8ActArgs a{};
  a.g.A = mat(A);
  a.g.B = mat(B);
  a.g.b_block = (uint8_t)B->block;
  a.g.C = C;
  a.g.c_type = (uint8_t)c_type;
  a.g.ldc = (int32_t)ldc;
  a.g.M = (int)M;
  a.g.N = (int)N;
  a.g.K = (int)K;
  a.act = (uint8_t)act;
  return a;
}

// the launches, in the caller's workspace or the library's
int run_mm(const iris::Fp8ActArgs& a, const iris::Fp8ActPlan& plan, void* dbias, void* workspace, void* stream, const char* what) {
  int dev = 0, cus = 0, st;
  if ((st = iris::use_device(&dev, &cus))) return st;
  std::unique_lock<std::mutex> hold;   // over all launches of the call
  if (plan.ws_bytes > 0 && !workspace && (st = iris::fp8_own_workspace(dev, stream, plan.ws_bytes, &workspace, &hold))) return st;
  return launched(iris::launch_fp8_mm_act(a, plan, dbias, workspace, (hipStream_t)stream), what);
}

}  // namespace

extern "C" {

size_t iris_dropout_workspace_size(int64_t rows, int64_t cols) try {
  if (check_rows(rows, cols) || rows == 0 || cols == 0) return 0;
  return iris::dropout_plan(rows, cols).ws_bytes;
} catch (const std::exception&) {
  return 0;
}

int iris_dropout(void* out, int64_t ld_out, const void* x, int64_t ldx, const void* residual, int64_t ld_residual, int32_t type,
                 float alpha, const iris_drop_t* drop, void* sums, int64_t rows, int64_t cols, void* workspace,
                 size_t workspace_bytes, void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  iris::DropoutArgs a{};
  if ((st = check_rows(rows, cols)) || (st = check_plain(out, type, true, ld_out, rows, cols, "out")) ||
      (st = check_plain(x, type, true, ldx, rows, cols, "x")) ||
      (st = check_optional(residual, type, ld_residual, rows, cols, "residual")) || (st = check_vector(sums, type, "sums")) ||
      (st = check_drop(drop, alpha, &a.drop)))
    return st;
  if (cols == 0 || (rows == 0 && !sums)) return IRIS_OK;
  iris::DropoutPlan plan{};
  if (sums) plan = iris::dropout_plan(rows, cols);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes))) return st;
  if ((st = check_distinct({{out, "out", true}, {sums, "sums", true}, {workspace, "workspace", true}, {x, "x", false},
                            {residual, "residual", false}, {drop ? (const void*)drop->offset_at : nullptr, "offset_at", false}})))
    return st;
  int dev = 0, cus = 0;
  if ((st = iris::use_device(&dev, &cus))) return st;
  std::unique_lock<std::mutex> hold;   // over both launches
  if (plan.ws_bytes > 0 && !workspace && (st = iris::fp8_own_workspace(dev, stream, plan.ws_bytes, &workspace, &hold))) return st;
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.ldx = (int32_t)ldx;
  a.ldr = (int32_t)ld_residual;
  a.ldo = (int32_t)ld_out;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.type = type;
  a.vec = rows16_or_none(x, ldx, type, rows) && rows16_or_none(out, ld_out, type, rows) &&
          rows16_or_none(residual, ld_residual, type, rows);
  return launched(iris::launch_dropout(a, plan, sums, workspace, (hipStream_t)stream), "iris_dropout");
} catch (const std::exception& e) {
  return caught(e);
}

int iris_block_norm(void* r, int64_t ld_r, void* n, int64_t ld_n, const iris_fp8_t* q, float* stats, const void* x, int64_t ld_x,
                    const void* y, int64_t ld_y, const iris_norm_t* norm, int64_t rows, int64_t cols, void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  iris::NormArgs a{};
  if ((st = check_rows(rows, cols)) || (st = check_norm(norm, y != nullptr, rows, cols, &a.p))) return st;
  const int32_t type = norm->type, xt = norm->stream_type;
  if ((st = check_plain(x, xt, true, ld_x, rows, cols, "x")) || (st = check_optional(y, type, ld_y, rows, cols, "y")) ||
      (st = check_optional(r, xt, ld_r, rows, cols, "r")) || (st = check_optional(n, type, ld_n, rows, cols, "n")))
    return st;
  if (q && (st = check_blocks1(q, rows, cols, "q"))) return st;
  if ((uintptr_t)stats % 16 != 0) return fail(IRIS_ERR_ALIGNMENT, "stats must be 16-byte aligned");
  if (rows == 0 || cols == 0) return IRIS_OK;   // pointers may be NULL
  if (!y && r) return fail(IRIS_ERR_INVALID_ARG, "r without y would be a copy of x");
  if (!r && !n && !q && !stats) return fail(IRIS_ERR_INVALID_ARG, "no output is wanted");
  if ((st = check_distinct({{r, "r", true}, {n, "n", true}, {q, "q", true}, {stats, "stats", true}, {x, "x", false}, {y, "y", false},
                            {norm->pre_w, "pre_w", false}, {norm->pre_b, "pre_b", false}, {norm->post_w, "post_w", false},
                            {norm->post_b, "post_b", false}, {norm->gate, "gate", false},
                            {norm->drop ? (const void*)norm->drop->offset_at : nullptr, "offset_at", false}})))
    return st;
  if ((st = ready())) return st;
  a.x = x;
  a.y = y;
  a.r = r;
  a.n = n;
  a.q = mat(q);
  a.stats = stats;
  a.ldx = (int32_t)ld_x;
  a.ldy = (int32_t)ld_y;
  a.ldr = (int32_t)ld_r;
  a.ldn = (int32_t)ld_n;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  const bool whole = cols % 8 == 0 && params16(norm, a.p, rows) && rows16_or_none(x, ld_x, xt, rows) &&
                     rows16_or_none(y, ld_y, type, rows) && rows16_or_none(r, ld_r, xt, rows) && rows16_or_none(n, ld_n, type, rows);
  const auto launch = type == IRIS_TYPE_FP16 ? iris::launch_norm<iris::f16> : iris::launch_norm<iris::bf16>;
  return launched(launch(a, xt == IRIS_TYPE_FP32, whole, (hipStream_t)stream), "iris_block_norm");
} catch (const std::exception& e) {
  return caught(e);
}

size_t iris_block_norm_bwd_workspace_size(int64_t rows, int64_t cols) try {
  if (check_rows(rows, cols) || cols > iris::kNormMaxCols || rows == 0 || cols == 0) return 0;
  return iris::norm_bwd_plan(rows, cols, false).ws_bytes;
} catch (const std::exception&) {
  return 0;
}

int iris_block_norm_bwd(void* dx, int64_t ld_dx, void* dy, int64_t ld_dy, float* dpre_w, float* dpre_b, float* dpost_w,
                        float* dpost_b, float* dgate, const void* dn, int64_t ld_dn, const void* dr, int64_t ld_dr, const void* r,
                        int64_t ld_r, const void* y, int64_t ld_y, const float* stats, const iris_norm_t* norm, int64_t rows,
                        int64_t cols, void* workspace, size_t workspace_bytes, void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  iris::NormBwdArgs a{};
  if ((st = check_rows(rows, cols)) || (st = check_norm(norm, y != nullptr, rows, cols, &a.p))) return st;
  const int32_t type = norm->type, xt = norm->stream_type;
  if ((st = check_optional(dx, xt, ld_dx, rows, cols, "dx")) || (st = check_optional(dy, type, ld_dy, rows, cols, "dy")) ||
      (st = check_optional(dn, type, ld_dn, rows, cols, "dn")) || (st = check_optional(dr, xt, ld_dr, rows, cols, "dr")) ||
      (st = check_optional(y, type, ld_y, rows, cols, "y")) || (st = check_optional(r, xt, ld_r, rows, cols, "r")))
    return st;
  if (rows > 0 && cols > 0 && !dx && !dy && !dpre_w && !dpre_b && !dpost_w && !dpost_b && !dgate)
    return fail(IRIS_ERR_INVALID_ARG, "no gradient is wanted");
  if (rows > 0 && cols > 0 && !dn && !dr) return fail(IRIS_ERR_INVALID_ARG, "dn and dr are both NULL");
  if (rows > 0 && cols > 0 && dn && !r) return fail(IRIS_ERR_INVALID_ARG, "dn needs r");
  if (rows > 0 && !stats) return fail(IRIS_ERR_INVALID_ARG, "stats is NULL");
  if (rows > 0 && cols > 0 && !y && (dy || dgate || dpost_w || dpost_b))
    return fail(IRIS_ERR_INVALID_ARG, "dy, dgate, dpost_w and dpost_b need y");
  if (dgate && !norm->gate) return fail(IRIS_ERR_INVALID_ARG, "dgate needs a gate");
  if (!norm->post && (dpost_w || dpost_b)) return fail(IRIS_ERR_INVALID_ARG, "dpost_w and dpost_b need post");
  if ((uintptr_t)stats % 16 != 0) return fail(IRIS_ERR_ALIGNMENT, "stats must be 16-byte aligned");
  const struct {
    float* p;
    const char* name;
  } sums[] = {{dpre_w, "dpre_w"}, {dpre_b, "dpre_b"}, {dpost_w, "dpost_w"}, {dpost_b, "dpost_b"}, {dgate, "dgate"}};
  for (const auto& v : sums)
    if ((st = check_vector(v.p, IRIS_TYPE_FP32, v.name))) return st;
  if (cols == 0 || (rows == 0 && !dpre_w && !dpre_b && !dpost_w && !dpost_b && !dgate)) return IRIS_OK;
  const bool whole = cols % 8 == 0 && params16(norm, a.p, rows) && rows16_or_none(dx, ld_dx, xt, rows) &&
                     rows16_or_none(dy, ld_dy, type, rows) && rows16_or_none(dn, ld_dn, type, rows) &&
                     rows16_or_none(dr, ld_dr, xt, rows) && rows16_or_none(r, ld_r, xt, rows) && rows16_or_none(y, ld_y, type, rows);
  const iris::NormBwdPlan plan = iris::norm_bwd_plan(rows, cols, whole);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes))) return st;
  if ((st = check_distinct({{dx, "dx", true}, {dy, "dy", true}, {dpre_w, "dpre_w", true}, {dpre_b, "dpre_b", true},
                            {dpost_w, "dpost_w", true}, {dpost_b, "dpost_b", true}, {dgate, "dgate", true},
                            {workspace, "workspace", true}, {dn, "dn", false}, {dr, "dr", false}, {r, "r", false}, {y, "y", false},
                            {stats, "stats", false}, {norm->pre_w, "pre_w", false}, {norm->post_w, "post_w", false},
                            {norm->post_b, "post_b", false}, {norm->gate, "gate", false},
                            {norm->drop ? (const void*)norm->drop->offset_at : nullptr, "offset_at", false}})))
    return st;
  int dev = 0, cus = 0;
  if ((st = iris::use_device(&dev, &cus))) return st;
  std::unique_lock<std::mutex> hold;   // over both launches
  if (plan.ws_bytes > 0 && !workspace && (st = iris::fp8_own_workspace(dev, stream, plan.ws_bytes, &workspace, &hold))) return st;
  const bool past = dy || dgate || dpost_w || dpost_b;   // the sum
  a.dn = dn;
  a.dr = dr;
  a.r = r;
  a.y = past ? y : nullptr;
  a.stats = stats;
  a.dx = dx;
  a.dy = dy;
  a.dpre_w = dpre_w;
  a.dpre_b = dpre_b;
  a.dpost_w = dpost_w;
  a.dpost_b = dpost_b;
  a.dgate = dgate;
  a.ld_dn = (int32_t)ld_dn;
  a.ld_dr = (int32_t)ld_dr;
  a.ld_r = (int32_t)ld_r;
  a.ld_y = (int32_t)ld_y;
  a.ld_dx = (int32_t)ld_dx;
  a.ld_dy = (int32_t)ld_dy;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.wg_rows = plan.wg_rows;
  a.wgs = plan.wgs;
  a.part = (float*)workspace;
  const auto launch = type == IRIS_TYPE_FP16 ? iris::launch_norm_bwd<iris::f16> : iris::launch_norm_bwd<iris::bf16>;
  hipError_t e = launch(a, xt == IRIS_TYPE_FP32, whole, (hipStream_t)stream);
  if (e == hipSuccess && (dpre_w || dpre_b || dpost_w || dpost_b || a.dgate)) e = iris::launch_norm_join(a, (hipStream_t)stream);
  return launched(e, "iris_block_norm_bwd");
} catch (const std::exception& e) {
  return caught(e);
}

size_t iris_fp8_mm_act_workspace_size(int64_t M, int64_t N, int64_t K, int32_t c_type, int32_t to8, int32_t dbias) try {
  if (check_mm_dims(M, N, K) || M == 0 || N == 0) return 0;
  return iris::fp8_mm_act_plan(M, N, K, c_type == IRIS_TYPE_FP32, to8 != 0, dbias != 0).ws_bytes;
} catch (const std::exception&) {
  return 0;
}

int iris_fp8_mm_act(void* C, int32_t c_type, int64_t ldc, void* z, int64_t ld_z, const iris_fp8_t* q, const iris_fp8_t* A,
                    const iris_fp8_t* B, const void* bias, int32_t act, float alpha, const iris_drop_t* drop, const void* residual,
                    int64_t ld_residual, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                    void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  if ((st = check_mm(c_type, A, B, M, N, K, act))) return st;
  if (M > 0 && N > 0 && !C && !q) return fail(IRIS_ERR_INVALID_ARG, "C and q are both NULL");
  iris::DropArgs d;
  if ((st = check_optional(C, c_type, ldc, M, N, "C")) || (st = check_optional(z, c_type, ld_z, M, N, "z")) ||
      (st = check_optional(residual, c_type, ld_residual, M, N, "residual")) || (st = check_vector(bias, c_type, "bias")) ||
      (st = check_drop(drop, alpha, &d)))
    return st;
  if (q && (st = check_blocks1(q, M, N, "q"))) return st;
  if (M == 0 || N == 0) return IRIS_OK;
  const iris::Fp8ActPlan plan = iris::fp8_mm_act_plan(M, N, K, c_type == IRIS_TYPE_FP32, q != nullptr, false);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes))) return st;
  if ((st = check_distinct({{C, "C", true}, {z, "z", true}, {q, "q", true}, {workspace, "workspace", true}, {A, "A", false},
                            {B, "B", false}, {bias, "bias", false}, {residual, "residual", false},
                            {drop ? (const void*)drop->offset_at : nullptr, "offset_at", false}})))
    return st;
  iris::Fp8ActArgs a = mm_args(C, c_type, ldc, A, B, M, N, K, act);
  a.g.bias = bias;
  a.z = z;
  a.ldz = (int32_t)ld_z;
  a.residual = residual;
  a.ldr = (int32_t)ld_residual;
  a.q = mat(q);
  a.drop = d;
  a.whole = N % 8 == 0 && rows16_or_none(C, ldc, c_type, M) && rows16_or_none(z, ld_z, c_type, M) &&
            rows16_or_none(residual, ld_residual, c_type, M);
  return run_mm(a, plan, nullptr, workspace, stream, "iris_fp8_mm_act");
} catch (const std::exception& e) {
  return caught(e);
}

int iris_fp8_mm_act_bwd(void* C, int32_t c_type, int64_t ldc, void* dbias, const iris_fp8_t* A, const iris_fp8_t* B, const void* z,
                        int64_t ld_z, int32_t act, float alpha, const iris_drop_t* drop, int64_t M, int64_t N, int64_t K,
                        void* workspace, size_t workspace_bytes, void* stream) try {
  iris::set_error(IRIS_OK, "");
  int st;
  if ((st = check_mm(c_type, A, B, M, N, K, act))) return st;
  if (act == IRIS_ACT_NONE) return fail(IRIS_ERR_INVALID_ARG, "no activation, so nothing to go back through: see iris_fp8_mm");
  iris::DropArgs d;
  if ((st = check_plain(C, c_type, true, ldc, M, N, "C")) || (st = check_plain(z, c_type, true, ld_z, M, N, "z")) ||
      (st = check_vector(dbias, c_type, "dbias")) || (st = check_drop(drop, alpha, &d)))
    return st;
  if (N == 0 || (M == 0 && !dbias)) return IRIS_OK;
  const iris::Fp8ActPlan plan = iris::fp8_mm_act_plan(M, N, K, c_type == IRIS_TYPE_FP32, false, dbias != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes))) return st;
  if ((st = check_distinct({{C, "C", true}, {dbias, "dbias", true}, {workspace, "workspace", true}, {A, "A", false}, {B, "B", false},
                            {z, "z", false}, {drop ? (const void*)drop->offset_at : nullptr, "offset_at", false}})))
    return st;
  iris::Fp8ActArgs a = mm_args(C, c_type, ldc, A, B, M, N, K, act);
  a.backward = 1;
  a.z = const_cast<void*>(z);
  a.ldz = (int32_t)ld_z;
  a.drop = d;
  a.whole = N % 8 == 0 && rows16_or_none(C, ldc, c_type, M) && rows16_or_none(z, ld_z, c_type, M);
  return run_mm(a, plan, dbias, workspace, stream, "iris_fp8_mm_act_bwd");
} catch (const std::exception& e) {
  return caught(e);
}

}  // extern "C"
