// Linear products of E4M3 operands with an FP32 scale for each block of 128 along the sum:
//
//   y[m, n] = sum over blocks b of xs[b, m] ws(b, n) (sum over k in b of xq[m, k] wq[n, k])  + bias + residual
//
// ws is one scale for each 128 x 128 block of W, or one for each row and block (a transposed operand
// quantized along the sum, for gradients).  Dense, or with one matrix per group of rows.
//
// The matrix cores multiply one block at a time (v_mfma_f32_16x16x128_f8f6f4, 128 elements of the
// sum): its result, started from zero, is scaled and added to the sums in FP32 by the vector unit, four
// multiply-adds a 16 x 16 tile, half the time the tile's product takes.  The products of 8 consecutive
// elements are added in a fixed-point window of 14 bits below the largest (see glu_gemm.hip), which moves
// a block's sum by less than the operands' own rounding by three orders of magnitude.
#include "ffn_product.h"
#include "fp8_launch.h"

namespace glu {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr uint32_t CODES = 128;   // codes a step, one line of an operand row and one block of scales

struct Fp8Args : ProductArgs {    // a, b, ld_a, ld_b and K count pairs of codes; work, c, bias, residual as there
  const float* xs;                // [blocks, I]
  const float* ws;                // BLOCK: [groups, blocks of J, blocks]; ROW: [groups, blocks, J]
  int64_t blocks;                 // of the sum
};

__device__ __forceinline__ v4f product128(v8i w, v8i x) {
  // format codes 0: E4M3; no block scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, (v4f)0.0f, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i join16(u32x4 a, u32x4 b) {
  return (v8i){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// WI x WJ waves of TI x TJ tiles of 16 x 16 each, NS stages of one block of the sum in LDS, filled by
// direct copies NS - 1 blocks ahead.  A stage ends with its scales: one for each row of A, then one for
// each row of B.
template <int W_SCALES, int WI, int WJ, int TI, int TJ, int NS>
__global__ __launch_bounds__(64 * WI * WJ) void k_fp8_product(Fp8Args a, uint32_t tiles_i, uint32_t tiles_j,
                                                              uint32_t splits) {
  constexpr int BI = 16 * WI * TI, BJ = 16 * WJ * TJ, WAVES = WI * WJ;
  using OpA = Operand<false, BI, WAVES>;
  using OpB = Operand<false, BJ, WAVES>;
  constexpr uint32_t SA = BI < 64 ? 64 : BI, SROWS = SA + BJ;                  // scales: whole loads of 64 rows
  constexpr int SLOADS = (SROWS / 64 + WAVES - 1) / WAVES, LOADS = OpA::LOADS + OpB::LOADS + SLOADS;
  constexpr uint32_t S_OFF = OpA::BYTES + OpB::BYTES, STAGE = S_OFF + 256u * SLOADS * WAVES;
  static_assert(NS * STAGE <= 160 * 1024);
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * STAGE];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  if (a.offsets != nullptr) {   // the grid allows for more row tiles than there are
    tiles_i = count_tiles(a.offsets, a.groups, a.I, BI);
    if (blockIdx.x >= tiles_i * tiles_j) return;
  }
  const uint32_t per = tiles_i * tiles_j;
  uint32_t b = xcd_run(blockIdx.x, a.offsets != nullptr ? per : gridDim.x);
  const uint32_t part = b / per;
  b -= part * per;
  const uint32_t in_group = GROUP_I * tiles_j, first_i = b / in_group * GROUP_I;
  const uint32_t gi = min(tiles_i - first_i, GROUP_I);
  const uint32_t ti = first_i + b % in_group % gi, tj = b % in_group / gi;
  const RowTile t = find_tile(a.offsets, a.groups, a.I, ti, BI);
  if (t.group < 0) return;
  const int64_t group = t.group;
  const bool none = group == a.groups;   // rows of no group
  uint32_t s0 = 0, s1 = none ? 0u : (uint32_t)a.blocks;   // steps
  if (splits > 1) {
    s0 = part_begin((uint32_t)a.blocks, part, splits);
    s1 = part_begin((uint32_t)a.blocks, part + 1, splits);
  }
  const uint32_t k1 = (uint32_t)a.K;
  const int64_t j0 = (int64_t)tj * BJ, j1 = min(j0 + BJ, a.J);
  const uint32_t wi = wave / WJ, wj = wave % WJ, g = lane >> 4, r = lane & 15u;
  const uint32_t rows = (uint32_t)(t.i1 - t.i0), cols = (uint32_t)(j1 - j0);

  OpA oa;
  OpB ob;
  oa.init(a.a, a.ld_a, t.i0, t.i1, wave, lane);
  ob.init(none ? a.b : a.b + group * a.b_group, a.ld_b, j0, j1, wave, lane);
  Fragments<false, BI, WI, TI> fa;
  Fragments<false, BJ, WJ, TJ> fb;
  fa.init(wi, lane);
  fb.init(wj, lane);
  // scale loads: load q of this wave is rows 64 (wave SLOADS + q) ..
  const int64_t gb = none ? 0 : group;
  const float* const wsb = W_SCALES == FP8_W_BLOCK ? a.ws + (gb * ((a.J + 127) / 128) + j0 / 128) * a.blocks
                                                   : a.ws + gb * a.blocks * a.J + j0;
  uint32_t so[SLOADS];
#pragma unroll
  for (int q = 0; q < SLOADS; q++) {
    const uint32_t at = 64u * (wave * SLOADS + q) + lane;
    if (at < SA) {
      so[q] = at < rows ? 4u * at : kOob;
    } else {
      const uint32_t j = at - SA;
      so[q] = j < cols ? 4u * (W_SCALES == FP8_W_BLOCK ? (uint32_t)((j0 + j) / 128 - j0 / 128) * (uint32_t)a.blocks : j) : kOob;
    }
  }
  auto issue = [&](uint32_t s, uint32_t at) {   // of step s into the stage at byte `at`; past the end zeros
    const bool live = s < s1;
    const uint32_t k = live ? s * (CODES / 2) : k1;
    if (k + BK <= k1) {
#pragma unroll
      for (int q = 0; q < OpA::LOADS; q++) oa.template issue<false>(q, k, k1, smem + at, wave, lane);
#pragma unroll
      for (int q = 0; q < OpB::LOADS; q++) ob.template issue<false>(q, k, k1, smem + at + OpA::BYTES, wave, lane);
    } else {
#pragma unroll
      for (int q = 0; q < OpA::LOADS; q++) oa.template issue<true>(q, k, k1, smem + at, wave, lane);
#pragma unroll
      for (int q = 0; q < OpB::LOADS; q++) ob.template issue<true>(q, k, k1, smem + at + OpA::BYTES, wave, lane);
    }
#pragma unroll
    for (int q = 0; q < SLOADS; q++) {
      const uint32_t first = 64u * (wave * SLOADS + q);
      const float* base = first < SA ? a.xs + (live ? s : 0) * a.I + t.i0
                                     : wsb + (live ? s : 0) * (W_SCALES == FP8_W_BLOCK ? 1 : a.J);
      const auto rs = rsrc(uniform((const uint16_t*)base));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(smem + at + S_OFF + 4u * first), 4,
                                               live && first < SROWS ? so[q] : kOob, 0, 0, 0);
    }
  };

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; i++)
#pragma unroll
    for (int j = 0; j < TJ; j++) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  if (s0 < s1) {
#pragma unroll
    for (int q = 0; q < NS - 1; q++) issue(s0 + q, q * STAGE);
    uint32_t now = 0;
    for (uint32_t s = s0; s < s1; s++) {
      wait_vm<(NS - 2) * LOADS>();
      lds_barrier();   // every wave's loads of this step have landed, and the step before has been read
      issue(s + NS - 1, now == 0 ? (NS - 1) * STAGE : now - STAGE);
      const uint8_t *const pa = smem + now, *const pb = pa + OpA::BYTES;
      const float* const sc = reinterpret_cast<const float*>(pa + S_OFF);
      v8i xb[TJ];
      v4f sw[TJ];
#pragma unroll
      for (int j = 0; j < TJ; j++)
        xb[j] = join16(*reinterpret_cast<const u32x4*>(pb + fb.at[0] + 2048u * j), *reinterpret_cast<const u32x4*>(pb + fb.at[1] + 2048u * j));
      if constexpr (W_SCALES == FP8_W_BLOCK) {
        // a wave's columns are 16 TJ <= 64 of one block, j0 being a multiple of 64 or of the tile
        sw[0] = (v4f)sc[SA + 16 * TJ * wj];
      } else {
#pragma unroll
        for (int j = 0; j < TJ; j++) sw[j] = *reinterpret_cast<const v4f*>(sc + SA + 16 * (TJ * wj + j) + 4 * g);
      }
#pragma unroll
      for (int i = 0; i < TI; i++) {
        const v8i xa = join16(*reinterpret_cast<const u32x4*>(pa + fa.at[0] + 2048u * i), *reinterpret_cast<const u32x4*>(pa + fa.at[1] + 2048u * i));
        const float sx = sc[16 * (TI * wi + i) + r];
#pragma unroll
        for (int j = 0; j < TJ; j++) {
          const v4f p = product128(xb[j], xa);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float f = sx * (W_SCALES == FP8_W_BLOCK ? sw[0][0] : sw[j][e]);
            acc[i][j][e] = __builtin_fmaf(p[e], f, acc[i][j][e]);
          }
        }
      }
      now = now == (NS - 1) * STAGE ? 0u : now + STAGE;
    }
    wait_vm<0>();
    lds_barrier();   // the stages hold the sums next
  }

  if (splits > 1) {
    const auto rw = rsrc(uniform((const uint16_t*)(a.work + ((int64_t)part * a.I + t.i0) * a.J + j0)));
#pragma unroll
    for (int i = 0; i < TI; i++)
#pragma unroll
      for (int j = 0; j < TJ; j++) {
        const uint32_t row = 16u * (TI * wi + i) + r, col = 16u * (TJ * wj + j) + 4u * g;
        put16(__builtin_bit_cast(u32x4, acc[i][j]), rw, row < rows && col < cols ? 4u * (row * (uint32_t)a.J + col) : kOob);
      }
    return;
  }
  // a row tile's sums through the wave's piece of LDS into eight consecutive columns a lane
  constexpr uint32_t PITCH = 16 * TJ + 4, CH = 2 * TJ, ROWS = 64 / CH, PASSES = 16 / ROWS;
  static_assert(WAVES * 16 * PITCH * 4 <= sizeof(smem));
  float* const mine = reinterpret_cast<float*>(smem) + wave * (16 * PITCH);
  const uint32_t cc = 8u * (lane % CH), lrow = lane / CH, col = 16u * TJ * wj + cc;
  const auto rc = rsrc(uniform(a.c + t.i0 * a.ld_c + j0));
  const auto rr = rsrc(uniform(a.residual != nullptr ? a.residual + t.i0 * a.ld_res + j0 : a.c));
  float bias[8];
  load_bf16(bias, !none && col < cols && a.bias != nullptr ? a.bias + group * a.J + j0 + col : nullptr);
#pragma unroll
  for (int i = 0; i < TI; i++) {
#pragma unroll
    for (int j = 0; j < TJ; j++) *reinterpret_cast<v4f*>(mine + r * PITCH + 16 * j + 4 * g) = acc[i][j];
#pragma unroll
    for (uint32_t p = 0; p < PASSES; p++) {
      const float* q = mine + (ROWS * p + lrow) * PITCH + cc;
      const v4f lo = *reinterpret_cast<const v4f*>(q), hi = *reinterpret_cast<const v4f*>(q + 4);
      const uint32_t row = 16u * (TI * wi + i) + ROWS * p + lrow;
      const bool ok = row < rows && col < cols;
      u32x4 res = (u32x4)0u;
      if (a.residual != nullptr && !none)
        res = __builtin_amdgcn_raw_buffer_load_b128(rr, ok ? 2u * (row * (uint32_t)a.ld_res + col) : kOob, 0, 0);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = v[e] + bias[e] + (e % 2 == 0 ? bf_lo(res[e / 2]) : bf_hi(res[e / 2]));
      put16(pack_row(v), rc, ok ? 2u * (row * (uint32_t)a.ld_c + col) : kOob);
    }
  }
}

// ---- few rows --------------------------------------------------------------------------------

// Up to 8 rows of one group: a pass over W at memory speed.  A wave takes 8 rows of W straight from
// memory; rows 8 .. 15 of its 16 x 16 x 128 tiles are the same ones in the next block of the sum, and so
// are columns 8 .. 15 of x: the halves that match are kept, each under its own block's scales.  KW waves
// share the sum, two blocks at a time in turn, and join through LDS.
// grid: column tiles of FEW_COLS FEW_WAVES / KW
template <int W_SCALES, int KW>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_fp8_few(Fp8Args a) {
  __shared__ v4f sums[FEW_WAVES][64];
  constexpr int U = 4;              // pairs of blocks in flight
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = FEW_COLS * ((int64_t)blockIdx.x * (FEW_WAVES / KW) + wave / KW);
  const uint32_t blocks = (uint32_t)a.blocks, first = 2u * (wave % KW), stride = 2u * KW;
  const uint32_t g = lane >> 4, r = lane & 7u, half = lane >> 3 & 1u;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n0 < a.J && first < blocks) {
    const uint32_t K = 2u * (uint32_t)a.K, mine = CODES * half + 16u * g;   // of the lane's first 16 codes; + 64
    const bool wr = n0 + r < a.J, xr = r < a.I;
    const uint32_t wo = r * K + mine, xo = r * K + mine;
    const auto rw = rsrc(uniform(a.b + n0 * a.ld_b)), rx = rsrc(uniform(a.a));
    const auto rxs = rsrc(uniform((const uint16_t*)a.xs));
    // lane (r, half, g): its results are x row r against W rows 4 g .. 4 g + 3 of the 16, so both of one block
    // where g / 2 is half
    const uint32_t own = lane >> 5;   // the block the kept results are of: g / 2
    const bool kept = own == half;
    auto load = [&](__amdgpu_buffer_rsrc_t from, uint32_t o, bool ok, uint32_t k) {
      u32x4 v[2];
#pragma unroll
      for (uint32_t h = 0; h < 2; h++)
        v[h] = __builtin_amdgcn_raw_buffer_load_b128(from, ok && k + mine + 64u * h < K ? o + 64u * h : kOob, (int)k, 0);
      return join16(v[0], v[1]);
    };
    for (uint32_t s = first; s < blocks; s += stride * U) {
      v8i w[U], x[U];
      float sx[U];
      v4f sw[U];
#pragma unroll
      for (int u = 0; u < U; u++) w[u] = load(rw, wo, wr, CODES * (s + stride * u));
#pragma unroll
      for (int u = 0; u < U; u++) {
        x[u] = load(rx, xo, xr, CODES * (s + stride * u));
        const uint32_t blk = s + stride * u + half;
        const bool ok = kept && xr && blk < blocks;
        sx[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rxs, ok ? 4u * (blk * (uint32_t)a.I + r) : kOob, 0, 0));
        sw[u] = (v4f)0.0f;
        if (ok) {
          if constexpr (W_SCALES == FP8_W_BLOCK) {
            sw[u] = (v4f)a.ws[n0 / 128 * blocks + blk];
          } else {
            const int64_t n = n0 + 4 * (g & 1u);
            if (n < a.J) sw[u] = *reinterpret_cast<const v4f*>(a.ws + blk * a.J + n);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const v4f p = product128(w[u], x[u]);
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (kept && s + stride * u + half < blocks) acc[e] = __builtin_fmaf(p[e], sx[u] * sw[u][e], acc[e]);
      }
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave % KW != 0 || (lane & 40u) != 0) return;
  v4f s = (v4f)0.0f;
#pragma unroll
  for (int w = 0; w < KW; w++) s += sums[wave + w][lane] + sums[wave + w][lane + 40];
  const int64_t row = lane & 15u, col = n0 + 4 * (lane >> 4);
  if (row >= a.I || col >= a.J) return;
  float v[4] = {s[0], s[1], s[2], s[3]};
  finish<FWD, LIN_NONE, 4>(a, 0, row, col, v);
}

// ---- which kernel ----------------------------------------------------------------------------

constexpr TileShape kFp8Shape[4] = {{2, 4, 8, 4, 2}, {4, 2, 4, 4, 3}, {2, 4, 4, 2, 3}, {1, 4, 2, 2, 4}};
constexpr double kFp8StepUs[3] = {1.29, 0.85, 0.5}, kFp8TileUs[3] = {15.0, 5.0, 4.0};
constexpr int64_t kFp8LeastPart = 8;   // blocks of a split sum's part

ProductPlan plan_fp8(int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped) {
  ProductPlan p{};
  p.splits = 1;
  if (I == 0 || J == 0) return p;
  const int64_t blocks = fp8_blocks(K);
  if (!grouped && I <= FEW_ROWS) {
    p.kind = FEW;
    const int64_t cols = ceil_div(J, FEW_COLS);
    p.share = 1;
    while (p.share < FEW_WAVES && cols * p.share < 16 * kUnits && blocks >= 4 * p.share) p.share *= 2;
    p.tiles_j = ceil_div(cols * p.share, FEW_WAVES);
    return p;
  }
  if (grouped && I <= kFp8Shape[TILE_32].rows() / 2 * groups) {
    p.kind = TILE_32;
    p.tiles_i = ceil_div(I, kFp8Shape[TILE_32].rows()) + groups + 1;
    p.tiles_j = ceil_div(J, kFp8Shape[TILE_32].cols());
    return p;
  }
  double best = 0.0;
  for (int kind = TILE_256; kind <= TILE_128; kind++) {
    const int64_t ti = ceil_div(I, kFp8Shape[kind].rows()), tj = ceil_div(J, kFp8Shape[kind].cols());
    const int64_t tiles = (ti + (grouped ? groups / 2 : 0)) * tj;
    int64_t splits = 1;
    if (!grouped && kind != TILE_256) {
      const int64_t most = blocks / kFp8LeastPart, want = kUnits / tiles;
      splits = want < most ? want : most;
      if (splits < 1) splits = 1;
    }
    double us = (kFp8TileUs[kind] + kFp8StepUs[kind] * ceil_div(blocks, splits)) * ceil_div(tiles * splits, kUnits);
    if (splits > 1) us += kJoinUs + 8e-6 / kJoinTBps * splits * I * J;
    if (best == 0.0 || us < best) {
      best = us;
      p.kind = kind;
      p.tiles_i = ti + (grouped ? groups + 1 : 0);
      p.tiles_j = tj;
      p.splits = splits;
    }
  }
  return p;
}

template <int W_SCALES>
hipError_t launch_fp8_product(const Fp8Args& a, int64_t codes, hipStream_t s) {
  const ProductPlan p = plan_fp8(a.I, a.J, codes, a.groups, a.offsets != nullptr);
  if (p.kind == FEW) {
    auto go = [&](auto KW) {
      return launch_kernel(k_fp8_few<W_SCALES, decltype(KW)::value>, dim3((unsigned)p.tiles_j), dim3(64 * FEW_WAVES), s, a);
    };
    return p.share == 1   ? go(std::integral_constant<int, 1>{})
           : p.share == 2 ? go(std::integral_constant<int, 2>{})
           : p.share == 4 ? go(std::integral_constant<int, 4>{})
                          : go(std::integral_constant<int, 8>{});
  }
  const unsigned n = (unsigned)(p.tiles_i * p.tiles_j * p.splits);
  auto go = [&](auto KIND) {
    constexpr TileShape t = kFp8Shape[decltype(KIND)::value];
    return launch_kernel(k_fp8_product<W_SCALES, t.wi, t.wj, t.ti, t.tj, t.stages>, dim3(n), dim3(64 * t.wi * t.wj), s, a,
                         (uint32_t)p.tiles_i, (uint32_t)p.tiles_j, (uint32_t)p.splits);
  };
  const hipError_t e = p.kind == TILE_256       ? go(std::integral_constant<int, TILE_256>{})
                       : p.kind == TILE_256_128 ? go(std::integral_constant<int, TILE_256_128>{})
                       : p.kind == TILE_128     ? go(std::integral_constant<int, TILE_128>{})
                                                : go(std::integral_constant<int, TILE_32>{});
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_kernel(k_product_join<FWD, LIN_NONE>, dim3(grid_for(ceil_div(a.I * a.J / 8, 256), 4096)), dim3(256), s, a,
                       (uint32_t)p.splits);
}

}  // namespace

int64_t fp8_linear_work_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool grouped) {
  const ProductPlan p = plan_fp8(M, N, K, groups, grouped);
  return p.splits > 1 ? 4 * p.splits * M * N : 0;
}

hipError_t launch_fp8_linear(const Fp8LinearArgs& a, hipStream_t s) {
  Fp8Args p{};
  p.I = a.M;
  p.J = a.N;
  p.K = a.K / 2;
  p.groups = a.groups;
  p.offsets = a.offsets;
  p.a = (const uint16_t*)a.xq;
  p.ld_a = a.K / 2;
  p.b = (const uint16_t*)a.wq;
  p.ld_b = a.K / 2;
  p.b_group = a.N * (a.K / 2);
  p.c = a.y;
  p.ld_c = a.ld_y;
  p.bias = a.bias;
  p.residual = a.residual;
  p.ld_res = a.ld_res;
  p.work = a.work;
  p.xs = a.xs;
  p.ws = a.ws;
  p.blocks = fp8_blocks(a.K);
  return a.w_scales == FP8_W_BLOCK ? launch_fp8_product<FP8_W_BLOCK>(p, a.K, s) : launch_fp8_product<FP8_W_ROW>(p, a.K, s);
}

}  // namespace glu
