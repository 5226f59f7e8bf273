// Device helpers shared by the gated projections and the checkpoints: the GLU of several
// elements, and MXFP8 blocks of BF16 pairs held by a few lanes.
#pragma once

#include "glu_device.h"

namespace glu {

// act(g) u of N elements in FP32, the rare ones of the tail again in FP64.
template <int ACT, int N>
__device__ __forceinline__ void glu_of(float (&h)[N], const float (&g)[N], const float (&u)[N]) {
  bool tail = false;
#pragma unroll
  for (int e = 0; e < N; e++) h[e] = glu_fwd_elem<ACT>(g[e], u[e], tail);
  if (tail) {
#pragma unroll
    for (int e = 0; e < N; e++)
      if (fwd_tail_needed<ACT>(g[e], u[e])) h[e] = glu_fwd_tail<ACT>(g[e], u[e]);
  }
}

// Values kept as BF16 with four more bits beside it (12 significant bits in all), so that gradients
// taken at them are not less exact than BF16 gradients are anyway: gate and up in BF16 alone move dx and
// dW by 0.0018 (2-norm, relative), as much as their own rounding does; so kept, by 0.0001.
// With v' the FP32 bits rounded to 12 significant bits, BF16 is v' rounded to 8 (halves away from zero),
// and the nibble, taken as -8 .. 7, is v' less it: the next four bits.  NaN keeps its kind: a NaN that
// comes of BF16 operands has zeros in the low half, which the roundings do not carry out of.
__device__ __forceinline__ uint32_t wide_pair(float a, float b) {   // two BF16
  return __builtin_amdgcn_perm(__float_as_uint(b) + 0x8800u, __float_as_uint(a) + 0x8800u, 0x07060302u);
}
// Four nibbles, the first lowest: bits 15 .. 12 of each value, moved to their places.
__device__ __forceinline__ uint32_t wide_rests(float a, float b, float c, float d) {
  auto bits = [](float v) { return __float_as_uint(v) + 0x800u; };
  return (bits(a) >> 12 & 0xfu) | (bits(b) >> 8 & 0xf0u) | (bits(c) >> 4 & 0xf00u) | (bits(d) & 0xf000u);
}
// The value of BF16 `hi` (in the upper half of a word whose lower half is zero) and nibble I of `rest`.
template <int I>
__device__ __forceinline__ float wide_value(uint32_t hi, uint32_t rest) {
  return __uint_as_float(hi + (uint32_t)((int32_t)(rest << (28 - 4 * I)) >> 28 << 12));
}

// The largest magnitude of packed BF16 pairs, as a BF16 bit pattern.
template <int N>
__device__ __forceinline__ uint32_t top_of(const uint32_t (&p)[N]) {
  uint32_t m = p[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < N; i++) m = pkmax(m, p[i] & 0x7fff7fffu);
  return umax(lo16(m), hi16(m));
}
// The MXFP8 scale byte of a block with that largest magnitude, and the codes of two pairs under it.
__device__ __forceinline__ uint32_t block_scale(uint32_t top) { return top >= 0x7f80u ? 0xffu : mx_scale_byte(top << 16); }
__device__ __forceinline__ uint32_t block_codes(uint32_t p0, uint32_t p1, uint32_t scale) {
  if (scale == 0xffu) return 0x7f7f7f7fu;
  const float s = e8m0_value(scale);
  return fp8x2_scaled<true>(fp8x2_scaled<false>(0u, p0, s), p1, s);
}

}  // namespace glu
