// Gated projections: both products of a gated linear unit, its activation and its product in one
// kernel, dense or with one matrix per group of rows, and their gradients:
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u
//   da = dh u act'(g),  db = dh act(g),  dp = [da | db];  dx = dp W,  dW = dp^T x,  dbias = sum of dp
//
// W [groups, 2N, K] holds Wg above Wu, or their rows in turn.  The sums are the tiled product's
// (ffn_product.h) with gate and up rows of W interleaved by 16 in LDS, so that a lane gets the
// gate and the up value of the same outputs and the pre-activation need not reach memory.  For the
// gradient it is kept as BF16, the type the GLU takes its operands in, with four more bits of each
// value beside it, or as MXFP8 codes of BF16 values; the gradient is that of the GLU at the values
// kept.  dp is rounded to BF16 for the matrix cores; dbias sums it unrounded.
#include "ffn_column_sums.h"
#include "ffn_product.h"
#include "gated_launch.h"

namespace glu {
namespace {

// ---- finishing what the tiles do not ---------------------------------------------------------

// N consecutive gates and ups of one row (sums) -> h and, as BF16, what is kept.  N is 4 or 8.
template <int ACT, int N>
__device__ __forceinline__ void finish_gated(const GatedArgs& a, int64_t group, int64_t row, int64_t n, float (&g)[N],
                                             float (&u)[N], uint32_t (&G)[N / 2], uint32_t (&U)[N / 2]) {
#pragma unroll
  for (int q = 0; q < N / 4; q++) {
    float bg[4], bu[4];
    load_gated_bias(bg, bu, a, group, n + 4 * q);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      g[4 * q + e] += bg[e];
      u[4 * q + e] += bu[e];
    }
  }
  float h[N];
  glu_of<ACT>(h, g, u);
  const bool wide = a.pre != nullptr;
#pragma unroll
  for (int e = 0; e < N / 2; e++) {
    G[e] = wide ? wide_pair(g[2 * e], g[2 * e + 1]) : pack_bf16(g[2 * e], g[2 * e + 1]);
    U[e] = wide ? wide_pair(u[2 * e], u[2 * e + 1]) : pack_bf16(u[2 * e], u[2 * e + 1]);
  }
  if (n >= a.J) return;
  *reinterpret_cast<bf16_vec<N>*>(a.c + row * a.ld_c + n) = pack_row(h);
  if (wide) {
    bf16_vec<N> pg, pu;
    uint16_t* rest = reinterpret_cast<uint16_t*>(a.rest + row * a.J + n / 2);
#pragma unroll
    for (int q = 0; q < N / 4; q++) {
      rest[q] = (uint16_t)wide_rests(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]);
      rest[a.J / 4 + q] = (uint16_t)wide_rests(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
    }
#pragma unroll
    for (int e = 0; e < N / 2; e++) {
      pg[e] = G[e];
      pu[e] = U[e];
    }
    *reinterpret_cast<bf16_vec<N>*>(a.pre + row * 2 * a.J + n) = pg;
    *reinterpret_cast<bf16_vec<N>*>(a.pre + row * 2 * a.J + a.J + n) = pu;
  }
}

// Joins the parts of split sums: eight outputs a thread, a row's chunks counted in whole fours, so that
// four neighbouring lanes hold one block of 32.  Bound by its start and
// the parts, which are in the caches: [256, 1024] and [128, 4096] in four parts with codes 5.2 and 5.5 us.
template <int ACT>
__global__ __launch_bounds__(256) void k_gated_join(GatedArgs a, uint32_t splits) {
  const int64_t V = gated_columns(a.J), CP = (a.J + 31) / 32 * 4, all = a.I * CP;
  for (int64_t q0 = 256 * (int64_t)blockIdx.x; q0 < all; q0 += 256 * (int64_t)gridDim.x) {
    const int64_t q = q0 + threadIdx.x;
    const int64_t row = q / CP, n = q < all ? 8 * (q % CP) : 8 * CP;   // 8 CP >= J: nothing to do
    v4f s[4] = {(v4f)0.0f, (v4f)0.0f, (v4f)0.0f, (v4f)0.0f};
    if (n < a.J) {
      const float* src = a.work + row * V + 32 * (n / 16) + n % 16;
      for (uint32_t p = 0; p < splits; p++, src += a.I * V) {
        s[0] += *reinterpret_cast<const v4f*>(src);
        s[1] += *reinterpret_cast<const v4f*>(src + 4);
        s[2] += *reinterpret_cast<const v4f*>(src + 16);
        s[3] += *reinterpret_cast<const v4f*>(src + 20);
      }
    }
    float g[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
    float u[8] = {s[2][0], s[2][1], s[2][2], s[2][3], s[3][0], s[3][1], s[3][2], s[3][3]};
    uint32_t G[4], U[4];
    finish_gated<ACT, 8>(a, 0, row, n, g, u, G, U);
    if (a.codes == nullptr) continue;
    uint32_t m = top_of(G) | top_of(U) << 16;
    m = pkmax(m, dpp<DPP_XOR1>(m));
    m = pkmax(m, dpp<DPP_XOR2>(m));
    const uint32_t sg = block_scale(lo16(m)), su = block_scale(hi16(m));
    if (n >= a.J) continue;
    const int64_t NB = (a.J + 31) / 32;
    uint8_t* c = a.codes + row * 2 * a.J + n;
    *reinterpret_cast<u32x2*>(c) = (u32x2){block_codes(G[0], G[1], sg), block_codes(G[2], G[3], sg)};
    *reinterpret_cast<u32x2*>(c + a.J) = (u32x2){block_codes(U[0], U[1], su), block_codes(U[2], U[3], su)};
    if (n % 32 == 0) {
      uint8_t* sc = a.scales + row * 2 * NB + n / 32;
      sc[0] = (uint8_t)sg;
      sc[NB] = (uint8_t)su;
    }
  }
}

// ---- few rows --------------------------------------------------------------------------------

// Up to 8 rows of one group: a pass over W at memory speed, as the linear products' (k_few_rows): a wave
// takes 8 rows of W of one kind straight from memory into 16 x 16 x 32 tiles whose other halves are
// the same rows 32 elements on.  Of 2 KW waves that share 8 outputs, KW take the gates and KW the ups,
// each kind cutting the sum among them; they meet in LDS.  [1, 2 x 16384, 2048]: 26.5 us (134 MB, 5.1 TB/s).  (The loop
// is that of k_few_rows again: as a function of both, its first loads start in another order, 14.4 us for 14.1 at
// [1, 2048, 16384].)
// grid: tiles of 8 outputs for 2 KW waves
template <int ACT, int KW>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_gated_few(GatedArgs a) {
  __shared__ v4f sums[FEW_WAVES][64];
  constexpr int U = 4, STEPS = 2;   // chunks per stage; tiles per chunk
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = FEW_COLS * ((int64_t)blockIdx.x * (FEW_WAVES / 2 / KW) + wave / (2 * KW));
  const bool up = wave / KW % 2 != 0;
  const uint32_t k1 = (uint32_t)a.K, first = FEW_CHUNK * (wave % KW), stride = FEW_CHUNK * KW;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n0 < a.J && first < k1) {
    const uint32_t r = lane & 7u, mine = 8u * (lane >> 4) + 32u * (lane >> 3 & 1u);   // the lane's row; its elements
    const int64_t step = a.paired ? 2 * a.K : a.K;
    const uint32_t wo = n0 + r < a.J ? 2u * (r * (uint32_t)step + mine) : kOob;
    const uint32_t xo = r < a.I ? 2u * (r * (uint32_t)a.ld_a + mine) : kOob;
    const auto rw = rsrc(uniform(a.b + n0 * step + (!up ? 0 : a.paired ? a.K : a.J * a.K))), rx = rsrc(uniform(a.a));
    v8bf w[2][U][STEPS];
    auto load_w = [&](uint32_t k, int s) {
#pragma unroll
      for (int c = 0; c < U; c++)
#pragma unroll
        for (int u = 0; u < STEPS; u++) {
          const uint32_t kk = k + stride * c + FEW_CHUNK / STEPS * u;
          w[s][c][u] = __builtin_bit_cast(
              v8bf, __builtin_amdgcn_raw_buffer_load_b128(rw, kk + mine < k1 ? wo : kOob, (int)(2u * kk), 0));
        }
    };
    // x of this stage before W of the next: loads return in order, and the products wait for x
    auto step_of = [&](uint32_t k, int s) {
      v8bf x[U][STEPS];
#pragma unroll
      for (int c = 0; c < U; c++)
#pragma unroll
        for (int u = 0; u < STEPS; u++) {
          const uint32_t kk = k + stride * c + FEW_CHUNK / STEPS * u;
          x[c][u] = __builtin_bit_cast(
              v8bf, __builtin_amdgcn_raw_buffer_load_b128(rx, kk + mine < k1 ? xo : kOob, (int)(2u * kk), 0));
        }
      __builtin_amdgcn_sched_barrier(0);
      if (k + stride * U < k1) load_w(k + stride * U, 1 - s);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < U; c++)
#pragma unroll
        for (int u = 0; u < STEPS; u++)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[s][c][u], x[c][u], acc, 0, 0, 0);
    };
    load_w(first, 0);
    for (uint32_t k = first; k < k1; k += 2 * stride * U) {
      step_of(k, 0);
      if (k + stride * U < k1) step_of(k + stride * U, 1);
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave % (2 * KW) != 0 || (lane & 40u) != 0) return;   // results are in rows and columns 0 .. 7 of the tile
  v4f s[2] = {(v4f)0.0f, (v4f)0.0f};
#pragma unroll
  for (int v = 0; v < 2 * KW; v++) s[v / KW] += sums[wave + v][lane] + sums[wave + v][lane + 40];   // and 8 .. 15
  const int64_t row = lane & 15u, n = n0 + 4 * (lane >> 4);
  if (row >= a.I || n >= a.J) return;
  float g[4] = {s[0][0], s[0][1], s[0][2], s[0][3]}, u[4] = {s[1][0], s[1][1], s[1][2], s[1][3]};
  uint32_t G[2], V[2];
  finish_gated<ACT, 4>(a, 0, row, n, g, u, G, V);
}

// ---- launches ----------------------------------------------------------------------------

template <int ACT>
hipError_t launch_gated(const GatedArgs& a, int save, hipStream_t s) {
  const ProductPlan p = plan_gated(save == SAVE_MXFP8, a.I, a.J, a.K, a.groups, a.offsets != nullptr);
  if (p.kind == FEW) {
    auto go = [&](auto KW) {
      return launch_kernel(k_gated_few<ACT, decltype(KW)::value>, dim3((unsigned)p.tiles_j), dim3(64 * FEW_WAVES), s, a);
    };
    return p.share == 1   ? go(std::integral_constant<int, 1>{})
           : p.share == 2 ? go(std::integral_constant<int, 2>{})
                          : go(std::integral_constant<int, 4>{});
  }
  const unsigned n = (unsigned)(p.tiles_i * p.tiles_j * p.splits);
  auto go = [&](auto KIND) {
    constexpr TileShape t = kGatedShape[decltype(KIND)::value];
    return launch_kernel(k_product<GATED, ACT, t.wi, t.wj, t.ti, t.tj, t.stages>, dim3(n), dim3(64 * t.wi * t.wj), s, a,
                         (uint32_t)p.tiles_i, (uint32_t)p.tiles_j, (uint32_t)p.splits);
  };
  const hipError_t e = p.kind == TILE_256       ? go(std::integral_constant<int, TILE_256>{})
                       : p.kind == TILE_256_128 ? go(std::integral_constant<int, TILE_256_128>{})
                       : p.kind == TILE_128     ? go(std::integral_constant<int, TILE_128>{})
                                                : go(std::integral_constant<int, TILE_32>{});
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_kernel(k_gated_join<ACT>, dim3(grid_for(ceil_div(a.I * ((a.J + 31) / 32 * 4), 256), 4096)), dim3(256), s, a,
                       (uint32_t)p.splits);
}

// Parts each group's rows are cut into for the sums of dp's rows: enough workgroups to fill the chip, with
// 16 rows or more of an average group each.  [1021, 1000] with 64 rows or more / 16 or more: the gradient 13.6 /
// 7.6 us, the join of the parts 4.6 / 3.2.
int64_t sum_parts(int64_t M, int64_t N, int64_t groups) {
  if (N == 0) return 1;
  const int64_t tiles = (N + 255) / 256 * groups, want = ceil_div(1024, tiles), most = ceil_div(M / groups, 16);
  const int64_t p = want < most ? want : most;
  return p < 1 ? 1 : p;
}

// Scratch memory of the backward: dp, the partial column sums, then the split sums of the products.
struct GatedBwdWork {
  int64_t dp, sums, split;   // bytes
};
GatedBwdWork gated_bwd_work(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias) {
  GatedBwdWork w{};
  w.dp = round16(4 * M * N);
  w.sums = bias ? round16(8 * sum_parts(M, N, groups) * groups * N) : 0;
  w.split = linear_bwd_work_bytes(LIN_NONE, M, 2 * N, K, groups, grouped, false);
  return w;
}

}  // namespace

int64_t gated_linear_work_bytes(int save, int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped) {
  const ProductPlan p = plan_gated(save == SAVE_MXFP8, M, N, K, groups, grouped);
  return p.splits > 1 ? 4 * p.splits * M * gated_columns(N) : 0;
}

int64_t gated_linear_bwd_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped, bool bias) {
  const GatedBwdWork w = gated_bwd_work(M, N, K, groups, grouped, bias);
  return w.dp + w.sums + w.split;
}

hipError_t launch_gated_linear(const GatedLinearArgs& a, hipStream_t s) {
  GatedArgs p{};
  p.I = a.M;
  p.J = a.N;
  p.K = a.K;
  p.groups = a.groups;
  p.offsets = a.offsets;
  p.a = a.x;
  p.ld_a = a.ld_x;
  p.b = a.w;
  p.ld_b = a.K;
  p.b_group = 2 * a.N * a.K;
  p.c = a.h;
  p.ld_c = a.ld_h;
  p.bias = a.bias;
  p.pre = a.save == SAVE_BF16 ? (uint16_t*)a.pre : nullptr;
  p.work = a.work;
  p.paired = a.w_layout == PAIRED;
  p.rest = a.extra;
  p.codes = a.save == SAVE_MXFP8 ? (uint8_t*)a.pre : nullptr;
  p.scales = a.extra;
  return with_act(a.act, [&](auto A) { return launch_gated<decltype(A)::value>(p, a.save, s); });
}

hipError_t launch_gated_linear_bwd(const GatedLinearBwdArgs& a, hipStream_t s) {
  const GatedBwdWork w = gated_bwd_work(a.M, a.N, a.K, a.groups, a.offsets != nullptr, a.db != nullptr);
  const bool products = a.dx != nullptr || a.dw != nullptr;
  uint16_t* dp = products ? (uint16_t*)a.work : nullptr;
  float* sums = a.db == nullptr ? nullptr : (float*)(a.work + w.dp);
  GluGradArgs g{};
  g.act = a.act;
  g.layout = a.w_layout;
  g.M = a.M;
  g.N = a.N;
  g.groups = sums == nullptr ? 1 : a.groups;
  g.offsets = sums == nullptr ? nullptr : a.offsets;
  g.pre = a.save == SAVE_BF16 ? (const uint16_t*)a.pre : nullptr;
  g.q = (const uint8_t*)a.pre;
  g.s = a.extra;
  g.dh = a.dh;
  g.ld_dh = a.ld_dh;
  g.d = dp;
  g.ld_d = 2 * a.N;
  g.h = a.h;
  g.ld_h = a.ld_h;
  g.sums = sums;
  g.parts = sum_parts(a.M, a.N, g.groups);
  hipError_t st = hipSuccess;
  if (a.N > 0 && (a.M > 0 || sums != nullptr)) st = launch_glu_grad(g, s);
  if (st == hipSuccess && sums != nullptr && a.N > 0)
    st = launch_kernel(k_linear_join, dim3((unsigned)((a.groups * 2 * a.N + 63) / 64)), dim3(256), s, sums, g.parts,
                       a.groups * 2 * a.N, a.db);
  if (st != hipSuccess || !products) return st;
  const LinearBwdArgs p{LIN_NONE, a.M, 2 * a.N, a.K, a.groups, a.offsets, dp, 2 * a.N, a.x, a.ld_x, a.w, nullptr, a.dx,
                        a.ld_dx, a.dw, nullptr, a.work + w.dp + w.sums};
  return launch_linear_bwd(p, s);
}

}  // namespace glu
