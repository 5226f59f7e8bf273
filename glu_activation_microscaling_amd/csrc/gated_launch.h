// Internal interface between the C-ABI layer (api_gated.cpp) and the kernels of the gated
// projections and of the checkpoints.  Arguments arrive validated.
#pragma once

#include "glu_launch.h"

namespace glu {

enum { SAVE_NONE = 0, SAVE_BF16 = 1, SAVE_MXFP8 = 2 };

constexpr int64_t kMaxGatedWidth = (int64_t)1 << 19;   // N: 2 N is a width of the linear products
constexpr int64_t kMaxCkptWidth = (int64_t)1 << 28;    // one workgroup per 256 columns

struct GatedLinearArgs {
  int act, w_layout, save;
  int64_t M, N, K, groups;
  const int32_t* offsets;    // [groups + 1] rows of each group, or null (one group, all rows)
  const uint16_t* x;         // [M, K]
  int64_t ld_x;
  const uint16_t* w;         // [groups, 2N, K], contiguous, rows in w_layout
  const uint16_t* bias;      // [groups, 2N] in the same order, or null
  uint16_t* h;               // [M, N]
  int64_t ld_h;
  void* pre;                 // [M, 2N] = [gate | up]: BF16 or E4M3 codes
  uint8_t* extra;            // BF16: [M, N], four more bits of each; codes: scales [M, 2 ceil(N/32)]
  float* work;
};

struct GatedLinearBwdArgs {
  int act, w_layout, save;   // SAVE_BF16 or SAVE_MXFP8
  int64_t M, N, K, groups;
  const int32_t* offsets;
  const uint16_t* dh;        // [M, N]
  int64_t ld_dh;
  const uint16_t* x;         // [M, K]
  int64_t ld_x;
  const uint16_t* w;
  const void* pre;
  const uint8_t* extra;      // BF16: may be null
  uint16_t* dx;              // [M, K], or null
  int64_t ld_dx;
  uint16_t* dw;              // [groups, 2N, K], or null
  uint16_t* db;              // [groups, 2N], or null
  uint16_t* h;               // [M, N] formed again, or null
  int64_t ld_h;
  uint8_t* work;
};

// The GLU's gradient from what was kept, and the column sums that give the bias's.
struct GluGradArgs {
  int act, layout;           // layout: of d
  int64_t M, N, groups;
  const int32_t* offsets;    // or null; with sums only
  const uint16_t* pre;       // BF16 [M, 2N], s then null or four more bits of each, [M, N]; or null:
  const uint8_t* q;          // MXFP8 codes [M, 2N] and scales s [M, 2 ceil(N/32)]
  const uint8_t* s;
  const uint16_t* dh;
  int64_t ld_dh;
  uint16_t* d;               // [M, 2N] = [da | db] or interleaved, or null
  int64_t ld_d;
  uint16_t* h;               // [M, N], or null
  int64_t ld_h;
  float* sums;               // [parts, groups, 2N] in d's order, or null
  int64_t parts;             // of the rows, with sums
};

struct CkptArgs {
  int act, layout;
  int64_t M, N;
  const uint16_t* gate;
  const uint16_t* up;
  int64_t ld_in;
  uint16_t* h;               // [M, N], or null
  int64_t ld_h;
  uint8_t* q;                // [M, 2N] = [gate | up]
  uint8_t* s;                // [M, 2 ceil(N/32)]
};

int64_t gated_linear_work_bytes(int save, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped);
int64_t gated_linear_bwd_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias);
hipError_t launch_gated_linear(const GatedLinearArgs& a, hipStream_t s);
hipError_t launch_gated_linear_bwd(const GatedLinearBwdArgs& a, hipStream_t s);
hipError_t launch_glu_grad(GluGradArgs a, hipStream_t s);
hipError_t launch_ckpt_fwd(const CkptArgs& a, hipStream_t s);

}  // namespace glu
