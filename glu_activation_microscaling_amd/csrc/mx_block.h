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
