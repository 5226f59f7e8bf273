// C-ABI entry points of 8-bit floating point with a scale for each block of 128: host-side validation,
// then the launches on the caller's stream.  As in api.cpp, every check runs before any HIP call
// and the glu_check_* exports run the same checks without a device.
#include "../../include/glu_mx.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "fp8_launch.h"

namespace {

using glu::aligned16;
using glu::any_overflow;
using glu::check_no_overlap;
using glu::fp8_blocks;
using glu::fp8_padded;
using glu::mat;
using glu::Operand;
using glu::status_of;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxQuantWidth = (int64_t)1 << 28;   // one workgroup per 256 columns
constexpr int64_t kMaxWidth = (int64_t)1 << 20;        // N of a product, and K where W is quantized by blocks
constexpr int64_t kMaxRowSum = (int64_t)1 << 22;       // K by rows, the rows of x in W's gradient: 256 code rows stay
                                                       // within 32-bit offsets

// Outputs of a quantizer: the pointers that go with the flags.
glu_status check_directions(int flags, const uint8_t* q_row, const float* s_row, const uint8_t* q_col, const float* s_col) {
  if ((flags & GLU_ROWWISE) ? q_row == nullptr || s_row == nullptr : q_row != nullptr || s_row != nullptr)
    return (flags & GLU_ROWWISE) ? GLU_ERR_NULL : GLU_ERR_ARG;
  if ((flags & GLU_COLWISE) ? q_col == nullptr || s_col == nullptr : q_col != nullptr || s_col != nullptr)
    return (flags & GLU_COLWISE) ? GLU_ERR_NULL : GLU_ERR_ARG;
  return aligned16(q_row) && aligned16(s_row) && aligned16(q_col) && aligned16(s_col) ? GLU_OK : GLU_ERR_ALIGN;
}

// A quantizer of [M, N], or of the GLU of such operands (paired: one of 2 N columns; up then NULL).
glu_status check_quant(bool glu_of, bool paired, int flags, int64_t M, int64_t N, const uint16_t* gate, const uint16_t* up,
                       int64_t ld_in, uint8_t* q_row, float* s_row, uint8_t* q_col, float* s_col) {
  if (flags == 0 || (flags & ~(GLU_ROWWISE | GLU_COLWISE)) != 0) return GLU_ERR_ARG;
  if (M < 0 || N < 0 || N % 8 != 0 || M > kMaxRows || N > kMaxQuantWidth) return GLU_ERR_SHAPE;
  if (M == 0 || N == 0) return GLU_OK;
  if (gate == nullptr || (glu_of && !paired && up == nullptr)) return GLU_ERR_NULL;
  if (paired && up != nullptr) return GLU_ERR_ARG;
  const int64_t cols = paired ? 2 * N : N;
  if (ld_in < cols || ld_in % 8 != 0) return GLU_ERR_STRIDE;
  if (!aligned16(gate) || !aligned16(up)) return GLU_ERR_ALIGN;
  const glu_status st = check_directions(flags, q_row, s_row, q_col, s_col);
  if (st != GLU_OK) return st;
  const Operand G = mat(gate, M, cols, ld_in, 2), U = mat(up, M, N, ld_in, 2),
                QR = mat(q_row, M, fp8_padded(N), fp8_padded(N), 1), SR = mat(s_row, fp8_blocks(N), M, M, 4),
                QC = mat(q_col, N, fp8_padded(M), fp8_padded(M), 1), SC = mat(s_col, fp8_blocks(M), N, N, 4);
  if (any_overflow({G, U, QR, SR, QC, SC})) return GLU_ERR_SHAPE;
  return check_no_overlap({QR, SR, QC, SC}, {G, U});
}

glu_status check_fp8_shape(int w_scales, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped) {
  if (w_scales != GLU_FP8_W_BLOCK && w_scales != GLU_FP8_W_ROW) return GLU_ERR_ARG;
  if (M < 0 || N < 0 || K < 0 || groups < 1 || M > kMaxRows || groups > glu::kMaxExperts) return GLU_ERR_SHAPE;
  if (N % 8 != 0 || K % 16 != 0 || N > kMaxWidth) return GLU_ERR_SHAPE;
  if (K > (w_scales == GLU_FP8_W_BLOCK ? kMaxWidth : kMaxRowSum)) return GLU_ERR_SHAPE;
  return grouped || groups == 1 ? GLU_OK : GLU_ERR_NULL;
}

// A BF16 matrix of the product: 16-byte rows.
glu_status check_matrix(const void* p, int64_t cols, int64_t ld) {
  if (ld < cols || ld % 8 != 0 || ld > glu::kMaxLinearStride) return GLU_ERR_STRIDE;
  return aligned16(p) ? GLU_OK : GLU_ERR_ALIGN;
}

}  // namespace

extern "C" {

glu_status glu_check_quant_fp8(int flags, int64_t M, int64_t N, const uint16_t* x, int64_t ld_x, uint8_t* q_row,
                               float* s_row, uint8_t* q_col, float* s_col) {
  return check_quant(false, false, flags, M, N, x, nullptr, ld_x, q_row, s_row, q_col, s_col);
}

glu_status glu_quant_fp8(int flags, int64_t M, int64_t N, const uint16_t* x, int64_t ld_x, uint8_t* q_row, float* s_row,
                         uint8_t* q_col, float* s_col, void* stream) {
  const glu_status st = glu_check_quant_fp8(flags, M, N, x, ld_x, q_row, s_row, q_col, s_col);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  return status_of(
      glu::launch_fp8_quant({-1, GLU_SPLIT, M, N, x, nullptr, ld_x, q_row, s_row, q_col, s_col}, (hipStream_t)stream));
}

glu_status glu_check_fwd_fp8(int act, int layout, int flags, int64_t M, int64_t N, const uint16_t* gate,
                             const uint16_t* up, int64_t ld_in, uint8_t* q_row, float* s_row, uint8_t* q_col,
                             float* s_col) {
  if (act < GLU_SWIGLU || act > GLU_RELU2 || (layout != GLU_SPLIT && layout != GLU_PAIRED)) return GLU_ERR_ARG;
  return check_quant(true, layout == GLU_PAIRED, flags, M, N, gate, up, ld_in, q_row, s_row, q_col, s_col);
}

glu_status glu_fwd_fp8(int act, int layout, int flags, int64_t M, int64_t N, const uint16_t* gate, const uint16_t* up,
                       int64_t ld_in, uint8_t* q_row, float* s_row, uint8_t* q_col, float* s_col, void* stream) {
  const glu_status st = glu_check_fwd_fp8(act, layout, flags, M, N, gate, up, ld_in, q_row, s_row, q_col, s_col);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  return status_of(
      glu::launch_fp8_quant({act, layout, M, N, gate, up, ld_in, q_row, s_row, q_col, s_col}, (hipStream_t)stream));
}

glu_status glu_check_quant_fp8_weight(int64_t groups, int64_t N, int64_t K, const uint16_t* w, uint8_t* q, float* s,
                                      uint8_t* qt, float* st) {
  if (groups < 0 || groups > glu::kMaxExperts || N < 0 || K < 0 || N % 8 != 0 || K % 8 != 0) return GLU_ERR_SHAPE;
  if (N > kMaxQuantWidth || K > kMaxQuantWidth) return GLU_ERR_SHAPE;
  if (groups == 0 || N == 0 || K == 0) return GLU_OK;
  if (w == nullptr || q == nullptr || s == nullptr || (qt == nullptr) != (st == nullptr)) return GLU_ERR_NULL;
  for (const void* p : {(const void*)w, (const void*)q, (const void*)s, (const void*)qt, (const void*)st})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  const int64_t nb = fp8_blocks(N), kb = fp8_blocks(K);
  const Operand W = mat(w, groups * N, K, K, 2), Q = mat(q, groups * N, fp8_padded(K), fp8_padded(K), 1),
                S = mat(s, groups * nb, kb, kb, 4), QT = mat(qt, groups * K, fp8_padded(N), fp8_padded(N), 1),
                ST = mat(st, groups * kb, nb, nb, 4);
  if (any_overflow({W, Q, S, QT, ST})) return GLU_ERR_SHAPE;
  return check_no_overlap({Q, S, QT, ST}, {W});
}

glu_status glu_quant_fp8_weight(int64_t groups, int64_t N, int64_t K, const uint16_t* w, uint8_t* q, float* s, uint8_t* qt,
                                float* st, void* stream) {
  const glu_status check = glu_check_quant_fp8_weight(groups, N, K, w, q, s, qt, st);
  if (check != GLU_OK || groups == 0 || N == 0 || K == 0) return check;
  return status_of(glu::launch_fp8_weight({groups, N, K, w, q, s, qt, st}, (hipStream_t)stream));
}

int64_t glu_linear_fp8_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, int grouped) {
  if (check_fp8_shape(GLU_FP8_W_ROW, M, N, K, groups, grouped != 0) != GLU_OK) return -1;
  return glu::fp8_linear_work_bytes(M, N, K, groups, grouped != 0);
}

glu_status glu_check_linear_fp8(int w_scales, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                                const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                                const uint16_t* bias, const uint16_t* residual, int64_t ld_res, uint16_t* y,
                                int64_t ld_y, void* work, int64_t work_bytes) {
  glu_status st = check_fp8_shape(w_scales, M, N, K, groups, offsets != nullptr);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  if (((uintptr_t)offsets & 3u) != 0) return GLU_ERR_ALIGN;
  if (y == nullptr || (K > 0 && (xq == nullptr || xs == nullptr || wq == nullptr || ws == nullptr))) return GLU_ERR_NULL;
  if ((st = check_matrix(y, N, ld_y)) != GLU_OK) return st;
  if (residual != nullptr && (st = check_matrix(residual, N, ld_res)) != GLU_OK) return st;
  for (const void* p : {(const void*)xq, (const void*)xs, (const void*)wq, (const void*)ws, (const void*)bias, (const void*)work})
    if (!aligned16(p)) return GLU_ERR_ALIGN;
  const int64_t need = glu::fp8_linear_work_bytes(M, N, K, groups, offsets != nullptr);
  if (need > 0 && work == nullptr) return GLU_ERR_NULL;
  if (need > work_bytes) return GLU_ERR_SHAPE;
  const int64_t kb = fp8_blocks(K), wr = w_scales == GLU_FP8_W_BLOCK ? fp8_blocks(N) : N;
  const Operand X = mat(K ? xq : nullptr, M, K, K, 1), XS = mat(K ? xs : nullptr, kb, M, M, 4),
                W = mat(K ? wq : nullptr, groups * N, K, K, 1), WS = mat(K ? ws : nullptr, groups * wr, kb, kb, 4),
                B = mat(bias, groups, N, N, 2), R = mat(residual, M, N, ld_res, 2), Y = mat(y, M, N, ld_y, 2),
                O = mat(offsets, 1, groups + 1, groups + 1, 4), T = mat(need ? work : nullptr, 1, need, need, 1);
  if (any_overflow({X, XS, W, WS, B, R, Y, O, T})) return GLU_ERR_SHAPE;
  return check_no_overlap({Y, T}, {X, XS, W, WS, B, R, O});
}

glu_status glu_linear_fp8(int w_scales, int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                          const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const uint16_t* bias,
                          const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y, void* work,
                          int64_t work_bytes, void* stream) {
  const glu_status st = glu_check_linear_fp8(w_scales, M, N, K, groups, offsets, xq, xs, wq, ws, bias, residual, ld_res, y,
                                             ld_y, work, work_bytes);
  if (st != GLU_OK || M == 0 || N == 0) return st;
  const glu::Fp8LinearArgs a{w_scales, M, N, K, groups, offsets, xq, xs, wq, ws, bias, residual, ld_res, y, ld_y,
                             (float*)work};
  return status_of(glu::launch_fp8_linear(a, (hipStream_t)stream));
}

}  // extern "C"
