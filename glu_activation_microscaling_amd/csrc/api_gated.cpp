// C-ABI entry points of the gated projections and of the GLU's 8-bit checkpoints: host-side
// validation, then the launches on the caller's stream.  As in api.cpp, every check runs before
// any HIP call and the glu_check_* exports run the same checks without a device.
#include "../../include/glu_mx.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "ffn_launch.h"
#include "gated_launch.h"

namespace {

using glu::aligned16;
using glu::any_overflow;
using glu::check_no_overlap;
using glu::mat;
using glu::Operand;
using glu::status_of;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxSum = (int64_t)1 << 20;   // K of a product

bool valid_act(int act) { return act >= GLU_SWIGLU && act <= GLU_RELU2; }
bool valid_layout(int layout) { return layout == GLU_SPLIT || layout == GLU_PAIRED; }
int64_t scale_columns(int64_t N) { return 2 * ((N + 31) / 32); }

glu_status check_gated_shape(int act, int w_layout, int save, int64_t M, int64_t N, int64_t K, int64_t groups,
                             bool grouped) {
  if (!valid_act(act) || !valid_layout(w_layout) || save < GLU_SAVE_NONE || save > GLU_SAVE_MXFP8) return GLU_ERR_ARG;
  if (M < 0 || N < 0 || K < 0 || groups < 1 || M > kMaxRows || groups > glu::kMaxExperts) return GLU_ERR_SHAPE;
  if (N % 8 != 0 || K % 8 != 0 || N > glu::kMaxGatedWidth || K > kMaxSum) return GLU_ERR_SHAPE;
  return grouped || groups == 1 ? GLU_OK : GLU_ERR_NULL;
}

// A BF16 matrix operand: 16-byte rows.
glu_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows == 0 || cols == 0) return GLU_OK;
  if (p == nullptr) return GLU_ERR_NULL;
  if (ld < cols || ld % 8 != 0 || ld > glu::kMaxLinearStride) return GLU_ERR_STRIDE;
  return aligned16(p) ? GLU_OK : GLU_ERR_ALIGN;
}

// What is kept of [gate | up]: the pointers that go with `save`.
glu_status check_kept(int save, const void* pre, const uint8_t* extra) {
  if ((pre == nullptr) != (save == GLU_SAVE_NONE)) return pre == nullptr ? GLU_ERR_NULL : GLU_ERR_ARG;
  if ((extra == nullptr) != (save == GLU_SAVE_NONE)) return extra == nullptr ? GLU_ERR_NULL : GLU_ERR_ARG;
  return aligned16(pre) && aligned16(extra) ? GLU_OK : GLU_ERR_ALIGN;
}
Operand kept(int save, const void* pre, int64_t M, int64_t N) {
  return mat(pre, M, 2 * N, 2 * N, save == GLU_SAVE_MXFP8 ? 1 : 2);
}
Operand kept_extra(int save, const uint8_t* extra, int64_t M, int64_t N) {
  const int64_t cols = save == GLU_SAVE_MXFP8 ? scale_columns(N) : N;
  return mat(extra, M, cols, cols, 1);
}

glu_status check_ckpt_shape(int act, int layout, int64_t M, int64_t N) {
  if (!valid_act(act) || !valid_layout(layout)) return GLU_ERR_ARG;
  return M < 0 || N < 0 || N % 8 != 0 || M > kMaxRows || N > glu::kMaxCkptWidth ? GLU_ERR_SHAPE : GLU_OK;
}

// A BF16 operand or output of the element-wise kernels.
glu_status check_rows(const void* p, int64_t cols, int64_t ld) {
  if (ld < cols || ld % 8 != 0) return GLU_ERR_STRIDE;
  return aligned16(p) ? GLU_OK : GLU_ERR_ALIGN;
}

}  // namespace

extern "C" {

// ---- gated projections -----------------------------------------------------------------------

int64_t glu_gated_linear_work_bytes(int save, int64_t M, int64_t N, int64_t K, int64_t groups, int grouped) {
  if (check_gated_shape(GLU_SWIGLU, GLU_SPLIT, save, M, N, K, groups, grouped != 0) != GLU_OK) return -1;
  return glu::gated_linear_work_bytes(save, M, N, K, groups, grouped != 0);
}

glu_status glu_check_gated_linear(int act, int w_layout, int save, int64_t M, int64_t N, int64_t K, int64_t groups,
                                  const int32_t* offsets, const uint16_t* x, int64_t ld_x, const uint16_t* w,
                                  const uint16_t* bias, uint16_t* h, int64_t ld_h, void* pre, uint8_t* extra,
                                  void* work, int64_t work_bytes) {
  glu_status st = check_gated_shape(act, w_layout, save, M, N, K, groups, offsets != nullptr);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  if (((uintptr_t)offsets & 3u) != 0) return GLU_ERR_ALIGN;
  if ((st = check_matrix(x, M, K, ld_x)) != GLU_OK) return st;
  if ((st = check_matrix(w, groups * 2 * N, K, K)) != GLU_OK) return st;
  if ((st = check_matrix(h, M, N, ld_h)) != GLU_OK) return st;
  if ((st = check_kept(save, pre, extra)) != GLU_OK) return st;
  if (!aligned16(bias) || !aligned16(work)) return GLU_ERR_ALIGN;
  const int64_t need = glu::gated_linear_work_bytes(save, M, N, K, groups, offsets != nullptr);
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  const Operand X = mat(K ? x : nullptr, M, K, ld_x, 2), W = mat(K ? w : nullptr, groups * 2 * N, K, K, 2),
                B = mat(bias, groups, 2 * N, 2 * N, 2), H = mat(h, M, N, ld_h, 2), P = kept(save, pre, M, N),
                S = kept_extra(save, extra, M, N), O = mat(offsets, 1, groups + 1, groups + 1, 4),
                WS = mat(need ? work : nullptr, 1, need, need, 1);
  if (any_overflow({X, W, B, H, P, S, O, WS})) return GLU_ERR_SHAPE;
  return check_no_overlap({H, P, S, WS}, {X, W, B, O});
}

glu_status glu_gated_linear(int act, int w_layout, int save, int64_t M, int64_t N, int64_t K, int64_t groups,
                            const int32_t* offsets, const uint16_t* x, int64_t ld_x, const uint16_t* w,
                            const uint16_t* bias, uint16_t* h, int64_t ld_h, void* pre, uint8_t* extra, void* work,
                            int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_gated_linear(act, w_layout, save, M, N, K, groups, offsets, x, ld_x, w, bias, h, ld_h,
                                               pre, extra, work, work_bytes);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  const glu::GatedLinearArgs a{act, w_layout, save, M, N, K, groups, offsets, x, ld_x, w, bias, h, ld_h, pre, extra,
                               (float*)work};
  return status_of(glu::launch_gated_linear(a, (hipStream_t)stream));
}

int64_t glu_gated_linear_bwd_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, int grouped, int with_bias) {
  if (check_gated_shape(GLU_SWIGLU, GLU_SPLIT, GLU_SAVE_BF16, M, N, K, groups, grouped != 0) != GLU_OK) return -1;
  return glu::gated_linear_bwd_work_bytes(M, N, K, groups, grouped != 0, with_bias != 0);
}

glu_status glu_check_gated_linear_bwd(int act, int w_layout, int save, int64_t M, int64_t N, int64_t K, int64_t groups,
                                      const int32_t* offsets, const uint16_t* dh, int64_t ld_dh, const uint16_t* x,
                                      int64_t ld_x, const uint16_t* w, const void* pre, const uint8_t* extra,
                                      uint16_t* dx, int64_t ld_dx, uint16_t* dw, uint16_t* dbias, uint16_t* h,
                                      int64_t ld_h, void* work, int64_t work_bytes) {
  glu_status st = check_gated_shape(act, w_layout, save, M, N, K, groups, offsets != nullptr);
  if (st != GLU_OK) return st;
  if (save == GLU_SAVE_NONE) return GLU_ERR_ARG;
  if (((uintptr_t)offsets & 3u) != 0) return GLU_ERR_ALIGN;
  if ((st = check_matrix(dh, M, N, ld_dh)) != GLU_OK) return st;
  if (M > 0 && N > 0) {
    if (pre == nullptr || (extra == nullptr && save == GLU_SAVE_MXFP8)) return GLU_ERR_NULL;
    if (!aligned16(pre) || !aligned16(extra)) return GLU_ERR_ALIGN;
  }
  if (dx != nullptr) {
    if ((st = check_matrix(w, groups * 2 * N, K, K)) != GLU_OK) return st;
    if ((st = check_matrix(dx, M, K, ld_dx)) != GLU_OK) return st;
  }
  if (dw != nullptr && (st = check_matrix(x, M, K, ld_x)) != GLU_OK) return st;
  if (h != nullptr && (st = check_matrix(h, M, N, ld_h)) != GLU_OK) return st;
  if (!aligned16(dw) || !aligned16(dbias) || !aligned16(work)) return GLU_ERR_ALIGN;
  const int64_t need = glu::gated_linear_bwd_work_bytes(M, N, K, groups, offsets != nullptr, dbias != nullptr);
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  const bool some = M > 0 && N > 0, sum = K > 0;
  const Operand DH = mat(some ? dh : nullptr, M, N, ld_dh, 2), X = mat(dw && M && sum ? x : nullptr, M, K, ld_x, 2),
                W = mat(dx && N && sum ? w : nullptr, groups * 2 * N, K, K, 2),
                P = kept(save, some ? pre : nullptr, M, N), S = kept_extra(save, some ? extra : nullptr, M, N),
                O = mat(offsets, 1, groups + 1, groups + 1, 4), DX = mat(M && sum ? dx : nullptr, M, K, ld_dx, 2),
                DW = mat(N && sum ? dw : nullptr, groups * 2 * N, K, K, 2),
                DB = mat(N ? dbias : nullptr, groups, 2 * N, 2 * N, 2), H = mat(some ? h : nullptr, M, N, ld_h, 2),
                WS = mat(need ? work : nullptr, 1, need, need, 1);
  if (any_overflow({DH, X, W, P, S, O, DX, DW, DB, H, WS})) return GLU_ERR_SHAPE;
  return check_no_overlap({DX, DW, DB, H, WS}, {DH, X, W, P, S, O});
}

glu_status glu_gated_linear_bwd(int act, int w_layout, int save, int64_t M, int64_t N, int64_t K, int64_t groups,
                                const int32_t* offsets, const uint16_t* dh, int64_t ld_dh, const uint16_t* x,
                                int64_t ld_x, const uint16_t* w, const void* pre, const uint8_t* extra, uint16_t* dx,
                                int64_t ld_dx, uint16_t* dw, uint16_t* dbias, uint16_t* h, int64_t ld_h, void* work,
                                int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_gated_linear_bwd(act, w_layout, save, M, N, K, groups, offsets, dh, ld_dh, x, ld_x, w,
                                                   pre, extra, dx, ld_dx, dw, dbias, h, ld_h, work, work_bytes);
  if (st != GLU_OK) return st;
  // what has no elements is not launched for; with M == 0, dw and dbias are still written (zero)
  const glu::GatedLinearBwdArgs a{act, w_layout, save, M, N, K, groups, offsets, dh, ld_dh, x, ld_x, w, pre, extra,
                                  M && K ? dx : nullptr, ld_dx, N && K ? dw : nullptr, N ? dbias : nullptr,
                                  M && N ? h : nullptr, ld_h, (uint8_t*)work};
  if (a.dx == nullptr && a.dw == nullptr && a.db == nullptr && a.h == nullptr) return GLU_OK;
  return status_of(glu::launch_gated_linear_bwd(a, (hipStream_t)stream));
}

// ---- checkpoints -----------------------------------------------------------------------------

int64_t glu_ckpt_scale_bytes(int64_t M, int64_t N) {
  return check_ckpt_shape(GLU_SWIGLU, GLU_SPLIT, M, N) == GLU_OK ? M * scale_columns(N) : -1;
}

glu_status glu_check_fwd_ckpt(int act, int layout, int64_t M, int64_t N, const uint16_t* gate, const uint16_t* up,
                              int64_t ld_in, uint16_t* h, int64_t ld_h, uint8_t* q, uint8_t* s) {
  glu_status st = check_ckpt_shape(act, layout, M, N);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  const bool paired = layout == GLU_PAIRED;
  if (gate == nullptr || q == nullptr || s == nullptr || (!paired && up == nullptr)) return GLU_ERR_NULL;
  if (paired && up != nullptr) return GLU_ERR_ARG;
  const int64_t cols = paired ? 2 * N : N;
  if ((st = check_rows(gate, cols, ld_in)) != GLU_OK) return st;
  if (h != nullptr && (st = check_rows(h, N, ld_h)) != GLU_OK) return st;
  if (!aligned16(up) || !aligned16(q) || !aligned16(s)) return GLU_ERR_ALIGN;
  const Operand G = mat(gate, M, cols, ld_in, 2), U = mat(up, M, N, ld_in, 2), H = mat(h, M, N, ld_h, 2),
                Q = kept(GLU_SAVE_MXFP8, q, M, N), S = kept_extra(GLU_SAVE_MXFP8, s, M, N);
  if (any_overflow({G, U, H, Q, S})) return GLU_ERR_SHAPE;
  return check_no_overlap({H, Q, S}, {G, U});
}

glu_status glu_fwd_ckpt(int act, int layout, int64_t M, int64_t N, const uint16_t* gate, const uint16_t* up,
                        int64_t ld_in, uint16_t* h, int64_t ld_h, uint8_t* q, uint8_t* s, void* stream) {
  const glu_status st = glu_check_fwd_ckpt(act, layout, M, N, gate, up, ld_in, h, ld_h, q, s);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  return status_of(glu::launch_ckpt_fwd({act, layout, M, N, gate, up, ld_in, h, ld_h, q, s}, (hipStream_t)stream));
}

glu_status glu_check_bwd_ckpt(int act, int layout, int64_t M, int64_t N, const uint8_t* q, const uint8_t* s,
                              const uint16_t* dh, int64_t ld_dh, uint16_t* d, int64_t ld_d, uint16_t* h, int64_t ld_h) {
  glu_status st = check_ckpt_shape(act, layout, M, N);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  if (q == nullptr || s == nullptr || dh == nullptr || d == nullptr) return GLU_ERR_NULL;
  if ((st = check_rows(dh, N, ld_dh)) != GLU_OK || (st = check_rows(d, 2 * N, ld_d)) != GLU_OK) return st;
  if (h != nullptr && (st = check_rows(h, N, ld_h)) != GLU_OK) return st;
  if (!aligned16(q) || !aligned16(s)) return GLU_ERR_ALIGN;
  const Operand Q = kept(GLU_SAVE_MXFP8, q, M, N), S = kept_extra(GLU_SAVE_MXFP8, s, M, N), DH = mat(dh, M, N, ld_dh, 2),
                DD = mat(d, M, 2 * N, ld_d, 2), H = mat(h, M, N, ld_h, 2);
  if (any_overflow({Q, S, DH, DD, H})) return GLU_ERR_SHAPE;
  return check_no_overlap({DD, H}, {Q, S, DH});
}

glu_status glu_bwd_ckpt(int act, int layout, int64_t M, int64_t N, const uint8_t* q, const uint8_t* s,
                        const uint16_t* dh, int64_t ld_dh, uint16_t* d, int64_t ld_d, uint16_t* h, int64_t ld_h,
                        void* stream) {
  const glu_status st = glu_check_bwd_ckpt(act, layout, M, N, q, s, dh, ld_dh, d, ld_d, h, ld_h);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  return status_of(glu::launch_glu_grad({act, layout, M, N, 1, nullptr, nullptr, q, s, dh, ld_dh, d, ld_d, h, ld_h,
                                         nullptr, 0},
                                        (hipStream_t)stream));
}

}  // extern "C"
