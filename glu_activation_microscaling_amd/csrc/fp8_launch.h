// Internal interface between the C-ABI layer (api_fp8.cpp) and the kernels of 8-bit floating
// point with a scale for each block of 128.  Arguments arrive validated.
#pragma once

#include "ffn_launch.h"
#include "ffn_plan.h"

namespace glu {

enum { FP8_W_BLOCK = 0, FP8_W_ROW = 1 };

inline int64_t fp8_padded(int64_t n) { return (n + 15) / 16 * 16; }

struct Fp8QuantArgs {
  int act, layout;           // act < 0: gate is the matrix itself
  int64_t M, N;
  const uint16_t* gate;
  const uint16_t* up;
  int64_t ld_in;
  uint8_t* q_row;            // [M, padded N], or null
  float* s_row;              // [blocks of N, M]
  uint8_t* q_col;            // [N, padded M], or null
  float* s_col;              // [blocks of M, N]
};

struct Fp8WeightArgs {
  int64_t groups, N, K;
  const uint16_t* w;         // [groups, N, K]
  uint8_t* q;                // [groups, N, padded K]
  float* s;                  // [groups, blocks of N, blocks of K]
  uint8_t* qt;               // [groups, K, padded N], or null
  float* st;                 // [groups, blocks of K, blocks of N]
};

struct Fp8LinearArgs {
  int w_scales;              // FP8_W_BLOCK or FP8_W_ROW
  int64_t M, N, K, groups;   // K % 16 == 0
  const int32_t* offsets;
  const uint8_t* xq;         // [M, K]
  const float* xs;           // [blocks of K, M]
  const uint8_t* wq;         // [groups, N, K]
  const float* ws;           // [groups, blocks of N, blocks of K] or [groups, blocks of K, N]
  const uint16_t* bias;      // [groups, N], or null
  const uint16_t* residual;  // [M, N], or null
  int64_t ld_res;
  uint16_t* y;               // [M, N]
  int64_t ld_y;
  float* work;
};

int64_t fp8_linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped);
hipError_t launch_fp8_quant(const Fp8QuantArgs& a, hipStream_t s);
hipError_t launch_fp8_weight(const Fp8WeightArgs& a, hipStream_t s);
hipError_t launch_fp8_linear(const Fp8LinearArgs& a, hipStream_t s);

}  // namespace glu
