// Linear products with their epilogue, and their gradients, dense or with one matrix per group
// of rows (the experts' products):
//
//   p = x W^T + b;  y = act(p) + residual
//   dp = dy act'(p);  dx = dp W;  dW = dp^T x;  db = sum of dp's rows
//
// x [M, K], W [groups, N, K], both BF16; products on the matrix cores with FP32 sums, bias,
// activation and residual in FP32, one rounding at the store.  Group e holds rows
// offsets[e] .. offsets[e+1] - 1; rows outside every group give zero rows of y and dx.  The
// pre-activation kept for the gradient is FP16, clamped to its range: act' of SiLU and GELU is
// constant beyond it to more digits than BF16 has, and FP16's 11 bits keep act' eight times
// nearer than BF16's 8 would.  dp is rounded to BF16, the type the matrix cores multiply;
// db sums it unrounded.
#include "ffn_column_sums.h"
#include "ffn_product.h"

namespace glu {
namespace {

// ---- dp = dy act'(p) and its column sums -----------------------------------------------------
// Bound by memory.  grid: (256 columns, group, part of the group's rows).  A thread holds 8 columns
// of every eighth row; the eight row sums are joined through LDS, and the parts by k_linear_join in
// a fixed order.  [16384, 7168] with GELU 166 us (4.2 TB/s), [16384, 4096] in 16 groups without an
// activation 37 us (3.6 TB/s).
struct GradArgs {
  int64_t M, N, groups;
  const int32_t* offsets;
  const uint16_t* dy;
  int64_t ld_dy;
  const uint16_t* pre;       // FP16 [M, N]
  uint16_t* dp;              // [M, N], or null
  float* sums;               // [parts, groups, N], or null
};
template <int ACT>
__global__ __launch_bounds__(256) void k_linear_grad(GradArgs a) {
  __shared__ float part[8][32][8];
  const int lc = threadIdx.x & 31, lr = threadIdx.x >> 5;
  const int64_t col = 256 * (int64_t)blockIdx.x + 8 * lc, e = blockIdx.y;
  int64_t r0 = 0, r1 = a.M;
  if (a.offsets != nullptr) {
    r0 = min((int64_t)max(a.offsets[e], 0), a.M);
    r1 = max(r0, min((int64_t)a.offsets[e + 1], a.M));
  }
  const int64_t n = r1 - r0;
  r1 = r0 + n * (blockIdx.z + 1) / gridDim.z;
  r0 = r0 + n * blockIdx.z / gridDim.z;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (col < a.N) {
    constexpr int U = ACT == LIN_NONE ? 4 : 2;   // rows in flight
    for (int64_t row = r0 + lr; row < r1; row += 8 * U) {
      Raw<uint16_t> y[U], p[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int n = row + 8 * u < r1 ? 8 : 0;
        load<false>(y[u], a.dy + (row + 8 * u) * a.ld_dy, (uint32_t)col, n);
        if constexpr (ACT != LIN_NONE) load<false>(p[u], a.pre + (row + 8 * u) * a.N, (uint32_t)col, n);
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        float d[8];
        y[u].get(d);
        if constexpr (ACT != LIN_NONE) {
#pragma unroll
          for (int i = 0; i < 8; i++)
            d[i] *= act_grad<ACT>((float)__builtin_bit_cast(_Float16, (uint16_t)(p[u].a[i / 2] >> (16 * (i & 1)))));
        }
        if (a.dp != nullptr && row + 8 * u < r1) store<false>(a.dp + (row + 8 * u) * a.N, (uint32_t)col, d, 8);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] += d[i];
      }
    }
  }
  if (a.sums == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; i++) part[lr][lc][i] = s[i];
  __syncthreads();
  const int64_t c = 256 * (int64_t)blockIdx.x + threadIdx.x;
  if (c < a.N) {
    float t = 0.0f;
    for (int w = 0; w < 8; w++) t += part[w][threadIdx.x / 8][threadIdx.x % 8];
    a.sums[((int64_t)blockIdx.z * a.groups + e) * a.N + c] = t;
  }
}

// Parts each group's rows are cut into for the column sums: enough workgroups to fill the chip,
// with 64 rows or more of an average group each.
int64_t grad_parts(int64_t M, int64_t N, int64_t groups) {
  if (N == 0) return 1;
  const int64_t tiles = (N + 255) / 256 * groups, want = (1024 + tiles - 1) / tiles;
  const int64_t most = (M / groups + 63) / 64;
  const int64_t p = want < most ? want : most;
  return p < 1 ? 1 : p;
}

// ---- both gradients in one launch ----------------------------------------------------------

// Both gradients of a product without groups, each whole in its own workgroups: dx = dp W in the first ones, filled
// up to a multiple of 8 so that the rest, dW = dp^T x, start on the first XCD too.
template <int WI, int WJ, int TI, int TJ, int NS>
__global__ __launch_bounds__(64 * WI * WJ) void k_gradients(ProductArgs d, uint32_t d_i, uint32_t d_j, ProductArgs w,
                                                            uint32_t w_i, uint32_t w_j) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kProductLds<16 * WI * TI, 16 * WJ * TJ, NS>];
  const uint32_t nd = d_i * d_j, first = (nd + 7u) / 8u * 8u;
  if (blockIdx.x >= first)
    product_tile<WGRAD, LIN_NONE, WI, WJ, TI, TJ, NS>(w, w_i, w_j, 1, blockIdx.x - first, w_i * w_j, smem);
  else if (blockIdx.x < nd)
    product_tile<DGRAD, LIN_NONE, WI, WJ, TI, TJ, NS>(d, d_i, d_j, 1, blockIdx.x, nd, smem);
}

hipError_t launch_gradients(int kind, const ProductArgs& d, const ProductArgs& w, hipStream_t s) {
  auto go = [&](auto KIND) {
    constexpr TileShape t = kShape[decltype(KIND)::value];
    const int64_t j = ceil_div(d.J, t.cols()), di = ceil_div(d.I, t.rows()), wi = ceil_div(w.I, t.rows());
    return launch_kernel(k_gradients<t.wi, t.wj, t.ti, t.tj, t.stages>, dim3((unsigned)((di * j + 7) / 8 * 8 + wi * j)),
                         dim3(64 * t.wi * t.wj), s, d, (uint32_t)di, (uint32_t)j, w, (uint32_t)wi, (uint32_t)j);
  };
  return kind == TILE_128 ? go(std::integral_constant<int, TILE_128>{}) : go(std::integral_constant<int, TILE_256_128>{});
}

}  // namespace

int64_t linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped) {
  return product_work_bytes(FWD, M, N, K, groups, grouped);
}

namespace {
// Scratch memory of the backward: dp, the partial column sums, then the split sums of the two
// products (one after the other in the same place).
struct BwdWork {
  int64_t dp, sums, split;   // bytes
};
BwdWork bwd_work(int act, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias) {
  BwdWork w{};
  w.dp = act == LIN_NONE ? 0 : round16(2 * M * N);
  w.sums = bias ? round16(4 * grad_parts(M, N, groups) * groups * N) : 0;
  const int64_t d = product_work_bytes(DGRAD, M, K, N, groups, grouped);
  const int64_t g = product_work_bytes(WGRAD, N, K, M, groups, grouped);
  w.split = d > g ? d : g;
  return w;
}
}  // namespace

int64_t linear_bwd_work_bytes(int act, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias) {
  const BwdWork w = bwd_work(act, M, N, K, groups, grouped, bias);
  return w.dp + w.sums + w.split;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  const ProductArgs p{a.M, a.N, a.K, a.groups, a.offsets, a.x, a.ld_x, a.w, a.K, a.N * a.K, a.y, a.ld_y, 0,
                      a.bias, a.residual, a.ld_res, a.pre, a.work};
  return with_linear_act(a.act, [&](auto A) { return launch_product<FWD, decltype(A)::value>(p, s); });
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t s) {
  const BwdWork w = bwd_work(a.act, a.M, a.N, a.K, a.groups, a.offsets != nullptr, a.db != nullptr);
  const uint16_t* dp = a.dy;
  int64_t ld_dp = a.ld_dy;
  hipError_t st = hipSuccess;
  if (a.act != LIN_NONE || a.db != nullptr) {
    const int64_t parts = grad_parts(a.M, a.N, a.groups);
    uint16_t* out = a.act == LIN_NONE ? nullptr : (uint16_t*)a.work;
    float* sums = a.db == nullptr ? nullptr : (float*)(a.work + w.dp);
    const GradArgs g{a.M, a.N, a.groups, a.offsets, a.dy, a.ld_dy, a.pre, out, sums};
    const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)a.groups, (unsigned)parts);
    st = with_linear_act(a.act, [&](auto A) {
      return launch_kernel(k_linear_grad<decltype(A)::value>, grid, dim3(256), s, g);
    });
    if (st == hipSuccess && sums != nullptr)
      st = launch_kernel(k_linear_join, dim3((unsigned)((a.groups * a.N + 63) / 64)), dim3(256), s, sums, parts,
                         a.groups * a.N, a.db);
    if (out != nullptr) {
      dp = out;
      ld_dp = a.N;
    }
  }
  float* split = (float*)(a.work + w.dp + w.sums);
  const ProductArgs to_dx{a.M, a.K, a.N, a.groups, a.offsets, dp, ld_dp, a.w, a.K, a.N * a.K, a.dx, a.ld_dx, 0,
                          nullptr, nullptr, 0, nullptr, split};
  const ProductArgs to_dw{a.N, a.K, a.M, a.groups, a.offsets, dp, ld_dp, a.x, a.ld_x, 0, a.dw, a.K, a.N * a.K,
                          nullptr, nullptr, 0, nullptr, split};
  if (st == hipSuccess && a.dx != nullptr && a.dw != nullptr && a.offsets == nullptr) {
    const int kind = plan_gradients(a.M, a.N, a.K);
    if (kind >= 0) return launch_gradients(kind, to_dx, to_dw, s);
  }
  if (st == hipSuccess && a.dx != nullptr) st = launch_product<DGRAD, LIN_NONE>(to_dx, s);
  if (st == hipSuccess && a.dw != nullptr) st = launch_product<WGRAD, LIN_NONE>(to_dw, s);
  return st;
}

}  // namespace glu
