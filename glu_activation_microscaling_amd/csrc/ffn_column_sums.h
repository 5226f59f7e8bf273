// Joins partial column sums of the linear products' and the gated projections' gradients.
#pragma once

#include "ffn_device.h"

namespace glu {
namespace {

// 64 columns a workgroup, every fourth part a wave.
__global__ __launch_bounds__(256) void k_linear_join(const float* sums, int64_t parts, int64_t n, uint16_t* out) {
  __shared__ float part[4][64];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int64_t i = 64 * (int64_t)blockIdx.x + lane;
  float s = 0.0f;
  if (i < n) {
#pragma unroll 4
    for (int64_t p = wave; p < parts; p += 4) s += sums[p * n + i];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < n)
    out[i] = (uint16_t)pack_bf16((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]), 0.0f);
}

// Sizes of the pieces of a call's scratch memory.
int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

}  // namespace
}  // namespace glu
