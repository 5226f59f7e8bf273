// C-ABI entry points of the operators around the GLU (block norms, linear products, expert
// routing): host-side validation, then the launches on the caller's stream.  As in api.cpp,
// every check runs before any HIP call and the glu_check_* exports run the same checks without
// a device.
#include "../../include/glu_mx.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "ffn_launch.h"

namespace {

using glu::aligned16;
using glu::any_overflow;
using glu::check_no_overlap;
using glu::mat;
using glu::Operand;
using glu::status_of;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;      // one workgroup or index a row
constexpr int64_t kMaxLinearWidth = (int64_t)1 << 20;     // N and K of a linear product
constexpr int64_t kMaxMoeRowBytes = (int64_t)1 << 24;

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// ---- norms -----------------------------------------------------------------------------------

constexpr int kNormFlags = GLU_NORM_PRE | GLU_NORM_POST | GLU_NORM_F32_STREAM | GLU_NORM_F32_PARAMS |
                           GLU_NORM_GATE_GROUPED | GLU_NORM_W_GROUPED | GLU_NORM_B_GROUPED;

glu_status check_norm_shape(int kind, int flags, int64_t M, int64_t H, int64_t groups) {
  if ((kind != GLU_NORM_RMS && kind != GLU_NORM_LAYER) || (flags & ~kNormFlags) != 0) return GLU_ERR_ARG;
  if (M < 0 || H < 0 || groups < 1 || M > kMaxRows || M % groups != 0) return GLU_ERR_SHAPE;
  if (H > glu::kMaxNormWidth) return GLU_ERR_SHAPE;
  return GLU_OK;
}

// A parameter: contiguous [groups, H], or [H] for all rows.
Operand norm_param(const void* p, int flags, int grouped, int64_t groups, int64_t H) {
  const int64_t esz = (flags & GLU_NORM_F32_PARAMS) ? 4 : 2;
  return mat(p, (flags & grouped) ? groups : 1, H, H, esz);
}

glu_status check_norm_inputs(int flags, int64_t H, const void* x, int64_t ld_x, const uint16_t* y, int64_t ld_y,
                             const void* gate, const void* w_pre, const void* b_pre, const void* w_post) {
  if (x == nullptr) return GLU_ERR_NULL;
  if (ld_x < H || (y != nullptr && ld_y < H)) return GLU_ERR_STRIDE;
  const bool pre = flags & GLU_NORM_PRE, post = flags & GLU_NORM_POST;
  if (!pre && (w_pre != nullptr || b_pre != nullptr)) return GLU_ERR_ARG;
  if (!post && w_post != nullptr) return GLU_ERR_ARG;
  if (y == nullptr && (post || gate != nullptr || !pre)) return GLU_ERR_ARG;   // y is what they act on
  for (const void* p : {x, (const void*)y, gate, w_pre, b_pre, w_post})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  return GLU_OK;
}

glu_status check_norm(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x, int64_t ld_x,
                      const uint16_t* y, int64_t ld_y, const void* gate, const void* w_pre, const void* b_pre,
                      const void* w_post, void* x_out, int64_t ld_xo, uint16_t* h, int64_t ld_h, uint8_t* q,
                      uint8_t* s, bool mx, float* stats) {
  glu_status st = check_norm_shape(kind, flags, M, H, groups);
  if (st != GLU_OK || M == 0 || H == 0) return st;
  if ((st = check_norm_inputs(flags, H, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post)) != GLU_OK) return st;
  const bool pre = flags & GLU_NORM_PRE;
  if (stats == nullptr) return GLU_ERR_NULL;
  if (y != nullptr && x_out == nullptr) return GLU_ERR_NULL;
  if (y == nullptr && x_out != nullptr) return GLU_ERR_ARG;
  if (x_out != nullptr && ld_xo < H) return GLU_ERR_STRIDE;
  if (mx) {
    if (!pre) return GLU_ERR_ARG;
    if (q == nullptr || s == nullptr) return GLU_ERR_NULL;
    if (H % 32 != 0) return GLU_ERR_SHAPE;
    if (ld_x % 8 != 0 || (y != nullptr && (ld_y % 8 != 0 || ld_xo % 8 != 0))) return GLU_ERR_STRIDE;
  } else if (pre) {
    if (h == nullptr) return GLU_ERR_NULL;
    if (ld_h < H) return GLU_ERR_STRIDE;
  } else if (h != nullptr) {
    return GLU_ERR_ARG;
  }
  for (const void* p : {(const void*)x_out, (const void*)h, (const void*)q, (const void*)s, (const void*)stats})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  const int64_t e = (flags & GLU_NORM_F32_STREAM) ? 4 : 2;
  const Operand X = mat(x, M, H, ld_x, e), Y = mat(y, M, H, ld_y, 2), XO = mat(x_out, M, H, ld_xo, e),
                Hh = mat(h, M, H, ld_h, 2), Q = mat(q, M, H, H, 1), S = mat(s, M, H / 32, H / 32, 1),
                T = mat(stats, M, 4, 4, 4), G = norm_param(gate, flags, GLU_NORM_GATE_GROUPED, groups, H),
                W = norm_param(w_pre, flags, GLU_NORM_W_GROUPED, groups, H),
                B = norm_param(b_pre, flags, GLU_NORM_B_GROUPED, groups, H), P = norm_param(w_post, flags, 0, 1, H);
  if (any_overflow({X, Y, XO, Hh, Q, S, T, G, W, B, P})) return GLU_ERR_SHAPE;
  return check_no_overlap({XO, Hh, Q, S, T}, {X, Y, G, W, B, P});
}

glu::NormArgs norm_args(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x, int64_t ld_x,
                        const uint16_t* y, int64_t ld_y, const void* gate, const void* w_pre, const void* b_pre,
                        const void* w_post, float res_scale, float eps, void* x_out, int64_t ld_xo, float* stats) {
  glu::NormArgs a{};
  a.kind = kind;
  a.flags = flags;
  a.M = M;
  a.H = H;
  a.rows_per_group = M / groups;
  a.x = x;
  a.ld_x = ld_x;
  a.y = y;
  a.ld_y = ld_y;
  a.gate = {gate, (flags & GLU_NORM_GATE_GROUPED) ? H : 0};
  a.w_pre = {w_pre, (flags & GLU_NORM_W_GROUPED) ? H : 0};
  a.b_pre = {b_pre, (flags & GLU_NORM_B_GROUPED) ? H : 0};
  a.w_post = {w_post, 0};
  a.res_scale = res_scale;
  a.eps = eps;
  a.x_out = x_out;
  a.ld_xo = ld_xo;
  a.stats = stats;
  return a;
}

// ---- linear products -------------------------------------------------------------------------

bool valid_linear_act(int act) { return act >= GLU_LINEAR_NONE && act <= GLU_LINEAR_GELU_ERF; }

glu_status check_linear_shape(int act, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped) {
  if (!valid_linear_act(act)) return GLU_ERR_ARG;
  if (M < 0 || N < 0 || K < 0 || groups < 1 || M > kMaxRows || groups > glu::kMaxExperts) return GLU_ERR_SHAPE;
  if (N % 8 != 0 || K % 8 != 0 || N > kMaxLinearWidth || K > kMaxLinearWidth) return GLU_ERR_SHAPE;
  return grouped || groups == 1 ? GLU_OK : GLU_ERR_NULL;
}

// A BF16 matrix operand of the products: 16-byte rows.
glu_status check_linear_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows == 0 || cols == 0) return GLU_OK;
  if (p == nullptr) return GLU_ERR_NULL;
  if (ld < cols || ld % 8 != 0 || ld > glu::kMaxLinearStride) return GLU_ERR_STRIDE;
  return aligned16(p) ? GLU_OK : GLU_ERR_ALIGN;
}

}  // namespace

extern "C" {

// ---- norms -----------------------------------------------------------------------------------

glu_status glu_check_block_norm(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                float eps, void* x_out, int64_t ld_xo, uint16_t* h, int64_t ld_h, float* stats) {
  (void)res_scale;
  if (!(eps >= 0.0f)) return GLU_ERR_ARG;
  return check_norm(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post, x_out, ld_xo, h, ld_h,
                    nullptr, nullptr, false, stats);
}

glu_status glu_block_norm(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x, int64_t ld_x,
                          const uint16_t* y, int64_t ld_y, const void* gate, const void* w_pre,
                          const void* b_pre, const void* w_post, float res_scale, float eps, void* x_out,
                          int64_t ld_xo, uint16_t* h, int64_t ld_h, float* stats, void* stream) {
  const glu_status st = glu_check_block_norm(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post,
                                             res_scale, eps, x_out, ld_xo, h, ld_h, stats);
  if (st != GLU_OK || M == 0 || H == 0) return st;
  glu::NormArgs a = norm_args(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post, res_scale, eps,
                              x_out, ld_xo, stats);
  a.h = h;
  a.ld_h = ld_h;
  return status_of(glu::launch_block_norm(a, (hipStream_t)stream));
}

glu_status glu_check_block_norm_mxfp8(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                      int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                      const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                      float eps, void* x_out, int64_t ld_xo, uint8_t* q, uint8_t* s, float* stats) {
  (void)res_scale;
  if (!(eps >= 0.0f)) return GLU_ERR_ARG;
  return check_norm(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post, x_out, ld_xo, nullptr, 0,
                    q, s, true, stats);
}

glu_status glu_block_norm_mxfp8(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                int64_t ld_x, const uint16_t* y, int64_t ld_y, const void* gate,
                                const void* w_pre, const void* b_pre, const void* w_post, float res_scale,
                                float eps, void* x_out, int64_t ld_xo, uint8_t* q, uint8_t* s, float* stats,
                                void* stream) {
  const glu_status st = glu_check_block_norm_mxfp8(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre,
                                                   w_post, res_scale, eps, x_out, ld_xo, q, s, stats);
  if (st != GLU_OK || M == 0 || H == 0) return st;
  glu::NormArgs a = norm_args(kind, flags, M, H, groups, x, ld_x, y, ld_y, gate, w_pre, b_pre, w_post, res_scale, eps,
                              x_out, ld_xo, stats);
  a.q = q;
  a.s = s;
  return status_of(glu::launch_block_norm(a, (hipStream_t)stream));
}

int64_t glu_block_norm_bwd_work_bytes(int64_t M, int64_t H, int64_t groups) {
  if (check_norm_shape(GLU_NORM_RMS, 0, M, H, groups) != GLU_OK) return -1;
  if (M == 0 || H == 0) return 0;
  return 4 * 4 * H * glu::norm_bwd_plan(M, H, M / groups).blocks;
}

glu_status glu_check_block_norm_bwd(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                                    int64_t ld_x, const uint16_t* y, int64_t ld_y, const float* stats,
                                    const void* dx_out, int64_t ld_dxo, const uint16_t* dh, int64_t ld_dh,
                                    const void* gate, const void* w_pre, const void* w_post, float res_scale,
                                    void* dx, int64_t ld_dx, uint16_t* dy, int64_t ld_dy, void* dgate,
                                    void* dw_pre, void* db_pre, void* dw_post, void* work, int64_t work_bytes) {
  (void)res_scale;
  glu_status st = check_norm_shape(kind, flags, M, H, groups);
  if (st != GLU_OK || H == 0) return st;
  const bool pre = flags & GLU_NORM_PRE, post = flags & GLU_NORM_POST;
  if (!pre && (dw_pre != nullptr || db_pre != nullptr)) return GLU_ERR_ARG;
  if (!post && dw_post != nullptr) return GLU_ERR_ARG;
  const int64_t e = (flags & GLU_NORM_F32_STREAM) ? 4 : 2;
  const Operand DG = norm_param(dgate, flags, GLU_NORM_GATE_GROUPED, groups, H),
                DW = norm_param(dw_pre, flags, GLU_NORM_W_GROUPED, groups, H),
                DB = norm_param(db_pre, flags, GLU_NORM_B_GROUPED, groups, H),
                DP = norm_param(dw_post, flags, 0, 1, H);
  for (const void* p : {(const void*)dgate, (const void*)dw_pre, (const void*)db_pre, (const void*)dw_post})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  if (M == 0) {   // the parameters' gradients are still written (zero)
    if (any_overflow({DG, DW, DB, DP})) return GLU_ERR_SHAPE;
    return check_no_overlap({DG, DW, DB, DP}, {});
  }
  if ((st = check_norm_inputs(flags, H, x, ld_x, y, ld_y, gate, w_pre, nullptr, w_post)) != GLU_OK) return st;
  if (stats == nullptr || dx == nullptr || (pre && dh == nullptr)) return GLU_ERR_NULL;
  if (!pre && dh != nullptr) return GLU_ERR_ARG;
  if (y != nullptr && dy == nullptr) return GLU_ERR_NULL;
  if (y == nullptr && (dy != nullptr || dgate != nullptr)) return GLU_ERR_ARG;
  if (!pre && dx_out == nullptr) return GLU_ERR_NULL;
  if ((dx_out != nullptr && ld_dxo < H) || (dh != nullptr && ld_dh < H) || ld_dx < H || (dy != nullptr && ld_dy < H))
    return GLU_ERR_STRIDE;
  const int64_t need = glu_block_norm_bwd_work_bytes(M, H, groups);
  if (work == nullptr && (dgate || dw_pre || db_pre || dw_post)) return GLU_ERR_NULL;
  if (work != nullptr && work_bytes < need) return GLU_ERR_SHAPE;
  for (const void* p : {(const void*)stats, dx_out, (const void*)dh, (const void*)dx, (const void*)dy, (const void*)work})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  const Operand X = mat(x, M, H, ld_x, e), Y = mat(y, M, H, ld_y, 2), T = mat(stats, M, 4, 4, 4),
                DXO = mat(dx_out, M, H, ld_dxo, e), DH = mat(dh, M, H, ld_dh, 2), DX = mat(dx, M, H, ld_dx, e),
                DY = mat(dy, M, H, ld_dy, 2), WS = mat(work, 1, need, need, 1),
                G = norm_param(gate, flags, GLU_NORM_GATE_GROUPED, groups, H),
                W = norm_param(w_pre, flags, GLU_NORM_W_GROUPED, groups, H), P = norm_param(w_post, flags, 0, 1, H);
  if (any_overflow({X, Y, T, DXO, DH, DX, DY, WS, G, W, P, DG, DW, DB, DP})) return GLU_ERR_SHAPE;
  return check_no_overlap({DX, DY, DG, DW, DB, DP, WS}, {X, Y, T, DXO, DH, G, W, P});
}

glu_status glu_block_norm_bwd(int kind, int flags, int64_t M, int64_t H, int64_t groups, const void* x,
                              int64_t ld_x, const uint16_t* y, int64_t ld_y, const float* stats,
                              const void* dx_out, int64_t ld_dxo, const uint16_t* dh, int64_t ld_dh,
                              const void* gate, const void* w_pre, const void* w_post, float res_scale,
                              void* dx, int64_t ld_dx, uint16_t* dy, int64_t ld_dy, void* dgate, void* dw_pre,
                              void* db_pre, void* dw_post, void* work, int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_block_norm_bwd(kind, flags, M, H, groups, x, ld_x, y, ld_y, stats, dx_out, ld_dxo,
                                                 dh, ld_dh, gate, w_pre, w_post, res_scale, dx, ld_dx, dy, ld_dy,
                                                 dgate, dw_pre, db_pre, dw_post, work, work_bytes);
  if (st != GLU_OK || H == 0) return st;
  const glu::NormBwdArgs a{kind, flags, M, H, M == 0 ? 1 : M / groups, x, ld_x, y, ld_y, stats, dx_out, ld_dxo, dh,
                           ld_dh,
                           {gate, (flags & GLU_NORM_GATE_GROUPED) ? H : 0, dgate},
                           {w_pre, (flags & GLU_NORM_W_GROUPED) ? H : 0, dw_pre},
                           {nullptr, (flags & GLU_NORM_B_GROUPED) ? H : 0, db_pre},
                           {w_post, 0, dw_post},
                           res_scale, dx, ld_dx, dy, ld_dy, (float*)work};
  return status_of(glu::launch_block_norm_bwd(a, groups, (hipStream_t)stream));
}

// ---- linear products -------------------------------------------------------------------------

int64_t glu_linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, int grouped) {
  if (check_linear_shape(GLU_LINEAR_NONE, M, N, K, groups, grouped != 0) != GLU_OK) return -1;
  return glu::linear_work_bytes(M, N, K, groups, grouped != 0);
}

glu_status glu_check_linear(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                            const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* bias,
                            const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y, uint16_t* pre,
                            void* work, int64_t work_bytes) {
  glu_status st = check_linear_shape(act, M, N, K, groups, offsets != nullptr);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  if (!aligned4(offsets)) return GLU_ERR_ALIGN;
  if ((st = check_linear_matrix(x, M, K, ld_x)) != GLU_OK) return st;
  if ((st = check_linear_matrix(w, groups * N, K, K)) != GLU_OK) return st;
  if ((st = check_linear_matrix(y, M, N, ld_y)) != GLU_OK) return st;
  if (residual != nullptr && (st = check_linear_matrix(residual, M, N, ld_res)) != GLU_OK) return st;
  if (!aligned16(bias) || !aligned16(pre) || !aligned16(work)) return GLU_ERR_ALIGN;
  const int64_t need = glu::linear_work_bytes(M, N, K, groups, offsets != nullptr);
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  const Operand X = mat(x, M, K, ld_x, 2), W = mat(w, groups * N, K, K, 2), B = mat(bias, groups, N, N, 2),
                R = mat(residual, M, N, ld_res, 2), Y = mat(y, M, N, ld_y, 2), P = mat(pre, M, N, N, 2),
                O = mat(offsets, 1, groups + 1, groups + 1, 4), WS = mat(work, 1, need, need, 1);
  if (any_overflow({X, W, B, R, Y, P, O, WS})) return GLU_ERR_SHAPE;
  return check_no_overlap({Y, P, WS}, {X, W, B, R, O});
}

glu_status glu_linear(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                      const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* bias,
                      const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y, uint16_t* pre,
                      void* work, int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_linear(act, M, N, K, groups, offsets, x, ld_x, w, bias, residual, ld_res, y, ld_y,
                                         pre, work, work_bytes);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  const glu::LinearArgs a{act, M, N, K, groups, offsets, x, ld_x, w, bias, residual, ld_res, y, ld_y, pre,
                          (float*)work};
  return status_of(glu::launch_linear(a, (hipStream_t)stream));
}

int64_t glu_linear_bwd_work_bytes(int act, int64_t M, int64_t N, int64_t K, int64_t groups, int grouped,
                                  int with_bias) {
  if (check_linear_shape(act, M, N, K, groups, grouped != 0) != GLU_OK) return -1;
  return glu::linear_bwd_work_bytes(act, M, N, K, groups, grouped != 0, with_bias != 0);
}

glu_status glu_check_linear_bwd(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                                const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ld_x,
                                const uint16_t* w, const uint16_t* pre, uint16_t* dx, int64_t ld_dx,
                                uint16_t* dw, uint16_t* db, void* work, int64_t work_bytes) {
  glu_status st = check_linear_shape(act, M, N, K, groups, offsets != nullptr);
  if (st != GLU_OK) return st;
  if (!aligned4(offsets)) return GLU_ERR_ALIGN;
  if ((st = check_linear_matrix(dy, M, N, ld_dy)) != GLU_OK) return st;
  if (act != GLU_LINEAR_NONE && M > 0 && N > 0 && pre == nullptr) return GLU_ERR_NULL;
  if (act == GLU_LINEAR_NONE && pre != nullptr) return GLU_ERR_ARG;
  if (dx != nullptr) {
    if ((st = check_linear_matrix(w, groups * N, K, K)) != GLU_OK) return st;
    if ((st = check_linear_matrix(dx, M, K, ld_dx)) != GLU_OK) return st;
  }
  if (dw != nullptr && (st = check_linear_matrix(x, M, K, ld_x)) != GLU_OK) return st;
  if (!aligned16(pre) || !aligned16(dw) || !aligned16(db) || !aligned16(work)) return GLU_ERR_ALIGN;
  const int64_t need = glu::linear_bwd_work_bytes(act, M, N, K, groups, offsets != nullptr, db != nullptr);
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  const Operand DY = mat(dy, M, N, ld_dy, 2), X = mat(dw ? x : nullptr, M, K, ld_x, 2),
                W = mat(dx ? w : nullptr, groups * N, K, K, 2), P = mat(pre, M, N, N, 2),
                O = mat(offsets, 1, groups + 1, groups + 1, 4), DX = mat(M ? dx : nullptr, M, K, ld_dx, 2),
                DW = mat(dw, groups * N, K, K, 2), DB = mat(db, groups, N, N, 2), WS = mat(work, 1, need, need, 1);
  if (any_overflow({X, W, DY, P, O, DX, DW, DB, WS})) return GLU_ERR_SHAPE;
  return check_no_overlap({DX, DW, DB, WS}, {DY, X, W, P, O});
}

glu_status glu_linear_bwd(int act, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                          const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ld_x, const uint16_t* w,
                          const uint16_t* pre, uint16_t* dx, int64_t ld_dx, uint16_t* dw, uint16_t* db,
                          void* work, int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_linear_bwd(act, M, N, K, groups, offsets, dy, ld_dy, x, ld_x, w, pre, dx, ld_dx, dw,
                                             db, work, work_bytes);
  if (st != GLU_OK) return st;
  // what has no elements is not launched for; with M == 0, dw and db are still written (zero)
  const glu::LinearBwdArgs a{act, M, N, K, groups, offsets, dy, ld_dy, x, ld_x, w, pre, M && K ? dx : nullptr, ld_dx,
                             N && K ? dw : nullptr, N ? db : nullptr, (uint8_t*)work};
  if (a.dx == nullptr && a.dw == nullptr && a.db == nullptr) return GLU_OK;
  return status_of(glu::launch_linear_bwd(a, (hipStream_t)stream));
}

// ---- expert routing --------------------------------------------------------------------------

int64_t glu_moe_sort_work_bytes(int64_t tokens, int64_t choices, int experts) {
  int64_t n;
  if (tokens < 0 || choices < 0 || experts < 1 || __builtin_mul_overflow(tokens, choices, &n)) return -1;
  const int64_t blocks = glu::moe_sort_blocks(n);
  return blocks > 1 ? 4 * blocks * experts : 0;
}

static glu_status check_moe(int64_t tokens, int64_t choices, int experts) {
  int64_t n;
  if (tokens < 0 || choices < 0 || experts < 1 || experts > glu::kMaxExperts) return GLU_ERR_SHAPE;
  if (__builtin_mul_overflow(tokens, choices, &n) || n > kMaxRows) return GLU_ERR_SHAPE;
  return GLU_OK;
}

glu_status glu_check_moe_sort(int64_t tokens, int64_t choices, int experts, const void* ids, int id_bytes,
                              int32_t* rows, int32_t* offsets, void* work, int64_t work_bytes) {
  const glu_status st = check_moe(tokens, choices, experts);
  if (st != GLU_OK) return st;
  if (id_bytes != 4 && id_bytes != 8) return GLU_ERR_ARG;
  const int64_t n = tokens * choices, need = glu_moe_sort_work_bytes(tokens, choices, experts);
  if (offsets == nullptr || (n > 0 && (ids == nullptr || rows == nullptr))) return GLU_ERR_NULL;
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  if (!aligned16(ids) || !aligned16(rows) || !aligned16(offsets) || !aligned16(work)) return GLU_ERR_ALIGN;
  const Operand I = mat(ids, 1, n, n, id_bytes), R = mat(rows, 1, n, n, 4),
                O = mat(offsets, 1, experts + 1, experts + 1, 4), W = mat(work, 1, need, need, 1);
  if (any_overflow({I, R, O, W})) return GLU_ERR_SHAPE;
  return check_no_overlap({R, O, W}, {I});
}

glu_status glu_moe_sort(int64_t tokens, int64_t choices, int experts, const void* ids, int id_bytes, int32_t* rows,
                        int32_t* offsets, void* work, int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_moe_sort(tokens, choices, experts, ids, id_bytes, rows, offsets, work, work_bytes);
  if (st != GLU_OK) return st;
  const glu::MoeSortArgs a{tokens * choices, experts, id_bytes, ids, rows, offsets, (int32_t*)work};
  return status_of(glu::launch_moe_sort(a, (hipStream_t)stream));
}

glu_status glu_check_moe_permute(int64_t tokens, int64_t choices, int experts, int64_t row_bytes, const void* x,
                                 int64_t ld_x, const int32_t* rows, const int32_t* offsets, void* xs,
                                 int64_t ld_xs) {
  const glu_status st = check_moe(tokens, choices, experts);
  if (st != GLU_OK) return st;
  if (row_bytes < 0 || row_bytes > kMaxMoeRowBytes) return GLU_ERR_SHAPE;
  const int64_t n = tokens * choices;
  if (n == 0 || row_bytes == 0) return GLU_OK;
  if (x == nullptr || rows == nullptr || offsets == nullptr || xs == nullptr) return GLU_ERR_NULL;
  if (ld_x < row_bytes || ld_xs < row_bytes) return GLU_ERR_STRIDE;
  if (!aligned16(x) || !aligned16(rows) || !aligned16(offsets) || !aligned16(xs)) return GLU_ERR_ALIGN;
  const Operand X = mat(x, tokens, row_bytes, ld_x, 1), R = mat(rows, 1, n, n, 4),
                O = mat(offsets, 1, experts + 1, experts + 1, 4), XS = mat(xs, n, row_bytes, ld_xs, 1);
  if (any_overflow({X, R, O, XS})) return GLU_ERR_SHAPE;
  return check_no_overlap({XS}, {X, R, O});
}

glu_status glu_moe_permute(int64_t tokens, int64_t choices, int experts, int64_t row_bytes, const void* x,
                           int64_t ld_x, const int32_t* rows, const int32_t* offsets, void* xs, int64_t ld_xs,
                           void* stream) {
  const glu_status st = glu_check_moe_permute(tokens, choices, experts, row_bytes, x, ld_x, rows, offsets, xs, ld_xs);
  if (st != GLU_OK || tokens * choices == 0 || row_bytes == 0) return st;
  const glu::MoePermuteArgs a{tokens, choices, row_bytes, ld_x, ld_xs, experts, (const uint8_t*)x, rows, offsets,
                              (uint8_t*)xs};
  return status_of(glu::launch_moe_permute(a, (hipStream_t)stream));
}

glu_status glu_check_moe_combine(int64_t tokens, int64_t choices, int64_t H, const uint16_t* y, int64_t ld_y,
                                 const int32_t* rows, const float* weights, const uint16_t* residual,
                                 int64_t ld_res, uint16_t* out, int64_t ld_out) {
  const glu_status st = check_moe(tokens, choices, 1);
  if (st != GLU_OK) return st;
  if (H < 0 || H > kMaxMoeRowBytes / 2) return GLU_ERR_SHAPE;
  if (tokens == 0 || H == 0) return GLU_OK;
  const int64_t n = tokens * choices;
  if (out == nullptr || (n > 0 && (y == nullptr || rows == nullptr))) return GLU_ERR_NULL;
  if (ld_out < H || (n > 0 && ld_y < H) || (residual != nullptr && ld_res < H)) return GLU_ERR_STRIDE;
  if (!aligned16(y) || !aligned16(rows) || !aligned16(weights) || !aligned16(residual) || !aligned16(out))
    return GLU_ERR_ALIGN;
  const Operand Y = mat(n ? y : nullptr, n, H, ld_y, 2), R = mat(rows, 1, n, n, 4), W = mat(weights, 1, n, n, 4),
                S = mat(residual, tokens, H, ld_res, 2), O = mat(out, tokens, H, ld_out, 2);
  if (any_overflow({Y, R, W, S, O})) return GLU_ERR_SHAPE;
  return check_no_overlap({O}, {Y, R, W, S});
}

glu_status glu_moe_combine(int64_t tokens, int64_t choices, int64_t H, const uint16_t* y, int64_t ld_y,
                           const int32_t* rows, const float* weights, const uint16_t* residual, int64_t ld_res,
                           uint16_t* out, int64_t ld_out, void* stream) {
  const glu_status st = glu_check_moe_combine(tokens, choices, H, y, ld_y, rows, weights, residual, ld_res, out,
                                              ld_out);
  if (st != GLU_OK || tokens == 0 || H == 0) return st;
  const glu::MoeCombineArgs a{tokens, choices, H, y, ld_y, rows, weights, residual, ld_res, out, ld_out};
  return status_of(glu::launch_moe_combine(a, (hipStream_t)stream));
}

glu_status glu_check_moe_combine_bwd(int64_t tokens, int64_t choices, int64_t H, int experts, const uint16_t* dout,
                                     int64_t ld_dout, const uint16_t* y, int64_t ld_y, const int32_t* rows,
                                     const float* weights, const int32_t* offsets, uint16_t* dy, int64_t ld_dy,
                                     float* dweights) {
  const glu_status st = check_moe(tokens, choices, experts);
  if (st != GLU_OK) return st;
  if (H < 0 || H > kMaxMoeRowBytes / 2) return GLU_ERR_SHAPE;
  const int64_t n = tokens * choices;
  if (n == 0) return GLU_OK;
  if (rows == nullptr || weights == nullptr || offsets == nullptr || dweights == nullptr) return GLU_ERR_NULL;
  if (H > 0 && (dout == nullptr || y == nullptr || dy == nullptr)) return GLU_ERR_NULL;
  if (ld_dout < H || ld_y < H || ld_dy < H) return GLU_ERR_STRIDE;
  for (const void* p : {(const void*)dout, (const void*)y, (const void*)rows, (const void*)weights,
                        (const void*)offsets, (const void*)dy, (const void*)dweights})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  const Operand D = mat(dout, tokens, H, ld_dout, 2), Y = mat(y, n, H, ld_y, 2), R = mat(rows, 1, n, n, 4),
                W = mat(weights, 1, n, n, 4), O = mat(offsets, 1, experts + 1, experts + 1, 4),
                DY = mat(dy, n, H, ld_dy, 2), DW = mat(dweights, 1, n, n, 4);
  if (any_overflow({D, Y, R, W, O, DY, DW})) return GLU_ERR_SHAPE;
  return check_no_overlap({DY, DW}, {D, Y, R, W, O});
}

glu_status glu_moe_combine_bwd(int64_t tokens, int64_t choices, int64_t H, int experts, const uint16_t* dout,
                               int64_t ld_dout, const uint16_t* y, int64_t ld_y, const int32_t* rows,
                               const float* weights, const int32_t* offsets, uint16_t* dy, int64_t ld_dy,
                               float* dweights, void* stream) {
  const glu_status st = glu_check_moe_combine_bwd(tokens, choices, H, experts, dout, ld_dout, y, ld_y, rows, weights,
                                                  offsets, dy, ld_dy, dweights);
  if (st != GLU_OK || tokens * choices == 0) return st;
  const glu::MoeCombineBwdArgs a{tokens, choices, H, experts, dout, ld_dout, y, ld_y, rows, weights, offsets, dy,
                                 ld_dy, dweights};
  return status_of(glu::launch_moe_combine_bwd(a, (hipStream_t)stream));
}

}  // extern "C"
