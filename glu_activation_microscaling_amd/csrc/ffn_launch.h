// Internal interface between the C-ABI layer (api_ffn.cpp) and the kernels of the operators
// around the GLU: block norms, linear products, expert routing.  Arguments arrive validated.
#pragma once

#include "glu_launch.h"

namespace glu {

enum { NORM_RMS = 0, NORM_LAYER = 1 };
enum { NORM_PRE = 1, NORM_POST = 2, NORM_F32_STREAM = 4, NORM_F32_PARAMS = 8 };   // flags
enum { LIN_NONE = 0, LIN_SILU = 1, LIN_GELU = 2, LIN_GELU_ERF = 3 };

// A per-channel parameter of the norms: [groups, H] (stride H) or one row for all (stride 0).
struct NormParam {
  const void* p;
  int64_t stride;
};

struct NormArgs {
  int kind, flags;
  int64_t M, H, rows_per_group;
  const void* x;             // residual stream, BF16 or FP32
  int64_t ld_x;
  const uint16_t* y;         // block output; null: x' = x
  int64_t ld_y;
  NormParam gate, w_pre, b_pre, w_post;   // w_post.stride is 0
  float res_scale, eps;
  void* x_out;
  int64_t ld_xo;
  uint16_t* h;               // BF16 h, or
  int64_t ld_h;
  uint8_t* q;                // MXFP8 codes [M, H] and scales [M, H/32] of it
  uint8_t* s;
  float* stats;              // [M, 4]: mean and 1/rms (or 1/sigma) of y, then of x'
};

struct NormGradParam {
  const void* p;
  int64_t stride;
  void* d;                   // gradient, in the parameter's type; null: not wanted
};

struct NormBwdArgs {
  int kind, flags;
  int64_t M, H, rows_per_group;
  const void* x;
  int64_t ld_x;
  const uint16_t* y;
  int64_t ld_y;
  const float* stats;
  const void* dx_out;        // null: zero
  int64_t ld_dxo;
  const uint16_t* dh;
  int64_t ld_dh;
  NormGradParam gate, w_pre, b_pre, w_post;
  float res_scale;
  void* dx;
  int64_t ld_dx;
  uint16_t* dy;
  int64_t ld_dy;
  float* work;               // partial column sums
};

// How the backward splits its rows over workgroups (a rule on shapes alone, so that the
// workspace can be sized before the launch).
struct NormBwdPlan {
  uint32_t groups;           // parameter groups
  uint32_t per_group;        // split: workgroups per group
  uint32_t part_rows;        // split: rows a workgroup; else whole groups a workgroup
  uint32_t blocks;           // workgroups = rows of partial sums
  bool split;                // a workgroup takes a part of one group
  unsigned threads;
  int vecs;                  // 8-column chunks per thread
};
NormBwdPlan norm_bwd_plan(int64_t M, int64_t H, int64_t rows_per_group);

constexpr int64_t kMaxNormWidth = 16384;

// ---- expert routing ----------------------------------------------------------------------

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxLinearStride = (int64_t)1 << 21;   // 256 rows stay within 32-bit offsets

struct MoeSortArgs {
  int64_t n;                 // choices, tokens x choices per token
  int experts;
  int id_bytes;              // 4 or 8
  const void* ids;
  int32_t* rows;             // [n]
  int32_t* offsets;          // [experts + 1]
  int32_t* work;             // [moe_sort_blocks(n)][experts] counts, when there is more than one block
};
int64_t moe_sort_blocks(int64_t n);

struct MoePermuteArgs {
  int64_t tokens, choices, row_bytes, ld_x, ld_xs;   // strides in bytes
  int experts;
  const uint8_t* x;
  const int32_t* rows;
  const int32_t* offsets;
  uint8_t* xs;
};

struct MoeCombineArgs {
  int64_t tokens, choices, H;
  const uint16_t* y;
  int64_t ld_y;
  const int32_t* rows;
  const float* weights;      // null: ones
  const uint16_t* residual;  // null: zero
  int64_t ld_res;
  uint16_t* out;
  int64_t ld_out;
};

struct MoeCombineBwdArgs {
  int64_t tokens, choices, H;
  int experts;
  const uint16_t* dout;
  int64_t ld_dout;
  const uint16_t* y;
  int64_t ld_y;
  const int32_t* rows;
  const float* weights;
  const int32_t* offsets;
  uint16_t* dy;
  int64_t ld_dy;
  float* dweights;           // [tokens, choices]
};

hipError_t launch_moe_sort(const MoeSortArgs& a, hipStream_t s);
hipError_t launch_moe_permute(const MoePermuteArgs& a, hipStream_t s);
hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t s);
hipError_t launch_moe_combine_bwd(const MoeCombineBwdArgs& a, hipStream_t s);

// ---- linear products ---------------------------------------------------------------------

struct LinearArgs {
  int act;
  int64_t M, N, K, groups;   // groups: matrices in w
  const int32_t* offsets;    // [groups + 1] rows of each group, or null (one group, all rows)
  const uint16_t* x;         // [M, K]
  int64_t ld_x;
  const uint16_t* w;         // [groups, N, K], contiguous
  const uint16_t* bias;      // [groups, N] or null
  const uint16_t* residual;  // [M, N] or null
  int64_t ld_res;
  uint16_t* y;               // [M, N]
  int64_t ld_y;
  uint16_t* pre;             // [M, N] FP16, contiguous, or null
  float* work;
};

struct LinearBwdArgs {
  int act;
  int64_t M, N, K, groups;
  const int32_t* offsets;
  const uint16_t* dy;        // [M, N]
  int64_t ld_dy;
  const uint16_t* x;         // [M, K]
  int64_t ld_x;
  const uint16_t* w;
  const uint16_t* pre;       // [M, N] FP16, or null (act none)
  uint16_t* dx;              // [M, K], or null
  int64_t ld_dx;
  uint16_t* dw;              // [groups, N, K], or null
  uint16_t* db;              // [groups, N], or null
  uint8_t* work;
};
int64_t linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped);
int64_t linear_bwd_work_bytes(int act, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias);

hipError_t launch_linear(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t s);

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_block_norm_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t s);

}  // namespace glu
