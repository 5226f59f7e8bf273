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
#include "ffn_device.h"
#include "ffn_launch.h"

namespace glu {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// ---- activations ---------------------------------------------------------------------------

template <int ACT>
__device__ __forceinline__ float act_of(float p) {
  if constexpr (ACT == LIN_NONE) return p;
  if constexpr (ACT == LIN_SILU) return p * (1.0f / (1.0f + __builtin_amdgcn_exp2f(-zl2<SWIGLU>(p))));
  if constexpr (ACT == LIN_GELU) return p * (1.0f / (1.0f + __builtin_amdgcn_exp2f(-zl2<GEGLU_TANH>(p))));
  if constexpr (ACT == LIN_GELU_ERF) return p < ERF_TAIL_X ? 0.0f : p * phi_cdf(p);
}
template <int ACT>
__device__ __forceinline__ float act_grad(float p) {
  if constexpr (ACT == LIN_NONE) return 1.0f;
  if constexpr (ACT == LIN_GELU_ERF) {
    float c, d;
    if (p < ERF_TAIL_X) return 0.0f;
    phi_cdf_pdf(p, c, d);
    return __builtin_fmaf(p, d, c);
  }
  if constexpr (ACT == LIN_SILU || ACT == LIN_GELU) {
    constexpr int A = ACT == LIN_SILU ? SWIGLU : GEGLU_TANH;
    const float z = zl2<A>(p), e = __builtin_amdgcn_exp2f(-__builtin_fabsf(z));
    const float s = 1.0f / (1.0f + e), sp = z >= 0.0f ? s : e * s, sn = z >= 0.0f ? e * s : s;
    return sp * __builtin_fmaf(p * sn, dz<A>(p), 1.0f);
  }
}

template <typename F>
hipError_t with_linear_act(int act, F&& f) {
  switch (act) {
    case LIN_SILU: return f(std::integral_constant<int, LIN_SILU>{});
    case LIN_GELU: return f(std::integral_constant<int, LIN_GELU>{});
    case LIN_GELU_ERF: return f(std::integral_constant<int, LIN_GELU_ERF>{});
    default: return f(std::integral_constant<int, LIN_NONE>{});
  }
}

// ---- the product ---------------------------------------------------------------------------
// C[i, j] = sum_k A(i, k) B(j, k).  An operand is stored with k along its rows (element (i, k)
// at i ld + k) or transposed (at k ld + i).
enum { FWD, DGRAD, WGRAD };

struct ProductArgs {
  int64_t I, J, K;           // rows of C, columns of C, length of the sum
  int64_t groups;
  const int32_t* offsets;    // splits I (FWD, DGRAD) or K (WGRAD)
  const uint16_t* a;
  int64_t ld_a;
  const uint16_t* b;
  int64_t ld_b, b_group;     // elements from one group's B to the next
  uint16_t* c;
  int64_t ld_c, c_group;
  const uint16_t* bias;      // [groups, J]
  const uint16_t* residual;
  int64_t ld_res;
  uint16_t* pre;             // [I, J]
};

constexpr int BI = 128, BJ = 128, BK = 32, PAD = 8, PROD_THREADS = 256;

// Finds the group and the row tile of tile number t when groups are cut into tiles of BI rows
// one by one; past the last group, the rows after it are tiled as group `groups`.
struct RowTile {
  int64_t group, i0, i1;
};
__device__ __forceinline__ RowTile find_tile(const int32_t* off, int64_t groups, int64_t I, int64_t t, int64_t size) {
  if (off == nullptr) return {0, t * size, min((t + 1) * size, I)};
  for (int64_t e = 0; e <= groups; e++) {
    const int64_t a = e == 0 ? 0 : min((int64_t)max(off[e], 0), I);
    const int64_t b = e == groups ? I : max(a, min((int64_t)off[e + 1], I));
    const int64_t n = (b - a + size - 1) / size;
    if (t < n) return {e, a + t * size, min(a + (t + 1) * size, b)};
    t -= n;
  }
  return {-1, 0, 0};
}

// Loads a BI x BK tile of an operand into LDS rows of BK elements (k contiguous): 8 elements
// a thread and step along the operand's contiguous dimension.  Rows i0 .. i1 - 1 and k below
// k1 exist; the rest reads zero.
template <bool T>
__device__ __forceinline__ void load_tile(uint16_t (*lds)[BK + PAD], const uint16_t* p, int64_t ld, int64_t i0,
                                          int64_t i1, int64_t k0, int64_t k1) {
  for (int c = threadIdx.x; c < BI * BK / 8; c += PROD_THREADS) {
    u32x4 v = (u32x4)0u;
    if constexpr (!T) {
      const int i = c / (BK / 8), k = c % (BK / 8) * 8;
      if (i0 + i < i1 && k0 + k < k1) v = *reinterpret_cast<const u32x4*>(p + (i0 + i) * ld + k0 + k);
      *reinterpret_cast<u32x4*>(&lds[i][k]) = v;
    } else {
      const int k = c / (BI / 8), i = c % (BI / 8) * 8;
      if (i0 + i < i1 && k0 + k < k1) v = *reinterpret_cast<const u32x4*>(p + (k0 + k) * ld + i0 + i);
#pragma unroll
      for (int j = 0; j < 8; j++) lds[i + j][k] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
    }
  }
}

// grid: (row tiles, column tiles, groups for WGRAD).  Four waves, 64 x 64 of C each.
template <int MODE, int ACT>
__global__ __launch_bounds__(PROD_THREADS) void k_product(ProductArgs a) {
  constexpr bool TA = MODE == WGRAD, TB = MODE != FWD;
  __shared__ __attribute__((aligned(16))) uint16_t sa[BI][BK + PAD], sb[BJ][BK + PAD];
  RowTile t;
  int64_t group, k0 = 0, k1 = a.K;
  if constexpr (MODE == WGRAD) {
    group = blockIdx.z;
    if (a.offsets != nullptr) {
      k0 = min((int64_t)max(a.offsets[group], 0), a.K);
      k1 = max(k0, min((int64_t)a.offsets[group + 1], a.K));
    }
    t = {group, (int64_t)blockIdx.x * BI, min((int64_t)(blockIdx.x + 1) * BI, a.I)};
  } else {
    t = find_tile(a.offsets, a.groups, a.I, blockIdx.x, BI);
    if (t.group < 0) return;
    group = t.group;
    if (group == a.groups) k1 = 0;   // rows of no group
  }
  const int64_t j0 = (int64_t)blockIdx.y * BJ, j1 = min(j0 + BJ, a.J);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int wi = 64 * (wave >> 1), wj = 64 * (wave & 1);
  const uint16_t* B = a.b + group * a.b_group;
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k = k0; k < k1; k += BK) {
    load_tile<TA>(sa, a.a, a.ld_a, t.i0, t.i1, k, k1);
    load_tile<TB>(sb, B, a.ld_b, j0, j1, k, k1);
    __syncthreads();
    v8bf fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; i++) fa[i] = *reinterpret_cast<const v8bf*>(&sa[wi + 16 * i + r][8 * g]);
#pragma unroll
    for (int j = 0; j < 4; j++) fb[j] = *reinterpret_cast<const v8bf*>(&sb[wj + 16 * j + r][8 * g]);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
  // acc[i][j][e] is C at row wi + 16 i + r, column wj + 16 j + 4 g + e of the tile
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t row = t.i0 + wi + 16 * i + r;
    if (row >= t.i1) continue;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t col = j0 + wj + 16 * j + 4 * g;
      if (col >= j1) continue;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = acc[i][j][e];
      if constexpr (MODE == FWD) {
        if (group < a.groups) {
          if (a.bias != nullptr)
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += bf_lo(a.bias[group * a.J + col + e]);
          if (a.pre != nullptr)
#pragma unroll
            for (int e = 0; e < 4; e++)
              a.pre[row * a.J + col + e] =
                  __builtin_bit_cast(uint16_t, (_Float16)__builtin_amdgcn_fmed3f(v[e], -65504.0f, 65504.0f));
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] = act_of<ACT>(v[e]);
          if (a.residual != nullptr)
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += bf_lo(a.residual[row * a.ld_res + col + e]);
        } else if (a.pre != nullptr) {
#pragma unroll
          for (int e = 0; e < 4; e++) a.pre[row * a.J + col + e] = 0;
        }
      }
      uint16_t* c = a.c + (MODE == WGRAD ? group * a.c_group : 0) + row * a.ld_c + col;
      *reinterpret_cast<u32x2*>(c) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
  }
}

// ---- dp = dy act'(p) and its column sums -----------------------------------------------------
// grid: (256 columns, group, part of the group's rows).  A thread holds 8 columns of every
// eighth row; the eight row sums are joined through LDS, and the parts by k_linear_join.
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
    for (int64_t row = r0 + lr; row < r1; row += 8) {
      Raw<uint16_t> q;
      load<false>(q, a.dy + row * a.ld_dy + col, 8);
      float d[8];
      q.get(d);
      if constexpr (ACT != LIN_NONE) {
        load<false>(q, a.pre + row * a.N + col, 8);
#pragma unroll
        for (int i = 0; i < 8; i++)
          d[i] *= act_grad<ACT>((float)__builtin_bit_cast(_Float16, (uint16_t)(q.a[i / 2] >> (16 * (i & 1)))));
      }
      if (a.dp != nullptr) store<false>(a.dp + row * a.N + col, d, 8);
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] += d[i];
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

__global__ __launch_bounds__(256) void k_linear_join(const float* sums, int64_t parts, int64_t n, uint16_t* out) {
  const int64_t i = 256 * (int64_t)blockIdx.x + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int64_t p = 0; p < parts; p++) s += sums[p * n + i];
  out[i] = (uint16_t)pack_bf16(s, 0.0f);
}

// Parts each group's rows are cut into for the column sums: enough workgroups to fill the chip,
// with 64 rows or more of an average group each.
int64_t grad_parts(int64_t M, int64_t N, int64_t groups) {
  const int64_t tiles = (N + 255) / 256 * groups, want = (1024 + tiles - 1) / tiles;
  const int64_t most = (M / groups + 63) / 64;
  const int64_t p = want < most ? want : most;
  return p < 1 ? 1 : p;
}

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

}  // namespace

int64_t linear_work_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

int64_t linear_bwd_work_bytes(int act, int64_t M, int64_t N, int64_t, int64_t groups, bool bias) {
  int64_t b = act == LIN_NONE ? 0 : round16(2 * M * N);
  if (bias) b += 4 * grad_parts(M, N, groups) * groups * N;
  return b;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  ProductArgs p{a.M, a.N, a.K, a.groups, a.offsets, a.x, a.ld_x, a.w, a.K, a.N * a.K, a.y, a.ld_y, 0,
                a.bias, a.residual, a.ld_res, a.pre};
  const int64_t ti = (a.M + BI - 1) / BI + (a.offsets != nullptr ? a.groups : 0);
  const dim3 grid((unsigned)ti, (unsigned)((a.N + BJ - 1) / BJ));
  return with_linear_act(a.act, [&](auto A) {
    return launch_kernel(k_product<FWD, decltype(A)::value>, grid, dim3(PROD_THREADS), s, p);
  });
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t s) {
  const uint16_t* dp = a.dy;
  int64_t ld_dp = a.ld_dy;
  hipError_t st = hipSuccess;
  if (a.act != LIN_NONE || a.db != nullptr) {
    const int64_t parts = grad_parts(a.M, a.N, a.groups);
    uint16_t* out = a.act == LIN_NONE ? nullptr : (uint16_t*)a.work;
    float* sums = a.db == nullptr ? nullptr : (float*)(a.work + (out ? round16(2 * a.M * a.N) : 0));
    const GradArgs g{a.M, a.N, a.groups, a.offsets, a.dy, a.ld_dy, a.pre, out, sums};
    const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)a.groups, (unsigned)parts);
    st = with_linear_act(a.act, [&](auto A) {
      return launch_kernel(k_linear_grad<decltype(A)::value>, grid, dim3(256), s, g);
    });
    if (st == hipSuccess && sums != nullptr)
      st = launch_kernel(k_linear_join, dim3((unsigned)((a.groups * a.N + 255) / 256)), dim3(256), s, sums, parts,
                         a.groups * a.N, a.db);
    if (out != nullptr) {
      dp = out;
      ld_dp = a.N;
    }
  }
  if (st == hipSuccess && a.dx != nullptr) {
    ProductArgs p{a.M, a.K, a.N, a.groups, a.offsets, dp, ld_dp, a.w, a.K, a.N * a.K, a.dx, a.ld_dx, 0,
                  nullptr, nullptr, 0, nullptr};
    const int64_t ti = (a.M + BI - 1) / BI + (a.offsets != nullptr ? a.groups : 0);
    st = launch_kernel(k_product<DGRAD, LIN_NONE>, dim3((unsigned)ti, (unsigned)((a.K + BJ - 1) / BJ)),
                       dim3(PROD_THREADS), s, p);
  }
  if (st == hipSuccess && a.dw != nullptr) {
    ProductArgs p{a.N, a.K, a.M, a.groups, a.offsets, dp, ld_dp, a.x, a.ld_x, 0, a.dw, a.K, a.N * a.K,
                  nullptr, nullptr, 0, nullptr};
    st = launch_kernel(k_product<WGRAD, LIN_NONE>,
                       dim3((unsigned)((a.N + BI - 1) / BI), (unsigned)((a.K + BJ - 1) / BJ), (unsigned)a.groups),
                       dim3(PROD_THREADS), s, p);
  }
  return st;
}

}  // namespace glu
