// Host-side argument checks shared by the C-ABI translation units: operand extents, overlap,
// alignment, and the status of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/glu_mx.h"

namespace glu {

// Bytes an operand or output of the GEMM kernels may span (32-bit offsets from its base).
constexpr int64_t kOffsetLimit = (int64_t)1 << 31;

// Byte extent of a row-major matrix: ((rows - 1) * ld + cols) * esz, or -1 on overflow.
inline int64_t extent_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t esz) {
  int64_t a, b, c;
  if (__builtin_mul_overflow(rows - 1, ld, &a)) return -1;
  if (__builtin_add_overflow(a, cols, &b)) return -1;
  if (__builtin_mul_overflow(b, esz, &c)) return -1;
  return c;
}

struct Operand {
  uintptr_t base;
  int64_t rows, cols, ld, esz;  // cols and ld in elements
  int64_t bytes;                // extent, -1 on overflow
};

inline Operand mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esz) {
  return Operand{(uintptr_t)p, rows, cols, ld, esz, extent_bytes(rows, cols, ld, esz)};
}

// True when the two operands may share a byte.  Operands with the same byte row stride
// are tested row by row (so [gate | up] halves of one buffer, or [dGate | dUp] outputs, do
// not count as overlapping); otherwise the byte spans are compared, which can only err
// on the side of rejecting.
inline bool overlaps(const Operand& A, const Operand& B) {
  if (A.base == 0 || B.base == 0) return false;
  const uintptr_t ahi = A.base + (uintptr_t)A.bytes, bhi = B.base + (uintptr_t)B.bytes;
  if (!(A.base < bhi && B.base < ahi)) return false;
  const int64_t L = A.ld * A.esz;
  if (L != B.ld * B.esz || L <= 0) return true;
  const int64_t wa = A.cols * A.esz, wb = B.cols * B.esz;
  const int64_t d = (int64_t)(B.base - A.base);  // two's complement difference
  // rows r of A and r' of B meet iff d - k L lies in (-wb, wa) for k = r - r'
  auto floordiv = [](int64_t x, int64_t y) { return x / y - ((x % y != 0) && ((x < 0) != (y < 0))); };
  for (int64_t k = floordiv(d - wa, L); k <= floordiv(d + wb, L) + 1; k++) {
    if (k > A.rows - 1 || k < -(B.rows - 1)) continue;
    const int64_t off = d - k * L;
    if (off > -wb && off < wa) return true;
  }
  return false;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool any_overflow(std::initializer_list<Operand> ops) {
  for (const Operand& o : ops)
    if (o.base != 0 && (o.bytes < 0 || o.base + (uintptr_t)o.bytes < o.base)) return true;
  return false;
}

inline glu_status check_no_overlap(std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (auto i = outs.begin(); i != outs.end(); ++i) {
    for (const Operand& in : ins)
      if (overlaps(*i, in)) return GLU_ERR_OVERLAP;
    for (auto j = i + 1; j != outs.end(); ++j)
      if (overlaps(*i, *j)) return GLU_ERR_OVERLAP;
  }
  return GLU_OK;
}

inline glu_status status_of(hipError_t e) { return e == hipSuccess ? GLU_OK : GLU_ERR_HIP; }

}  // namespace glu
