// The tiled matrix product on the BF16 matrix cores that the linear products and the gated
// projections are built from: operands copied straight into LDS, groups of rows found from
// offsets on the device, sums split over workgroups and joined, a kernel for few rows, and the
// rule that picks among them.
#pragma once

#include "ffn_device.h"
#include "ffn_launch.h"
#include "ffn_plan.h"
#include "ffn_split.h"
#include "mx_block.h"

#include <type_traits>

namespace glu {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// ---- activations ---------------------------------------------------------------------------

template <int ACT>
__device__ __forceinline__ float act_of(float p) {
  if constexpr (ACT == LIN_NONE) return p;
  if constexpr (ACT == LIN_SILU) return p * sigmoid_from(exp_neg(zl2<SWIGLU>(p)));
  if constexpr (ACT == LIN_GELU) return p * sigmoid_from(exp_neg(zl2<GEGLU_TANH>(p)));
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
    const float s = __builtin_amdgcn_rcpf(1.0f + e), sp = z >= 0.0f ? s : e * s, sn = z >= 0.0f ? e * s : s;
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
// GATED: C[i, n] = act(gate) * up of two such sums, B's rows in pairs (see GatedOperand).
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
  float* work;               // split sums: [parts, rows of C, J]
};
struct GatedArgs : ProductArgs {   // J outputs from 2 J rows of B; bias [groups, 2 J] in their order
  int paired;                // B's rows are gate0, up0, gate1, ... instead of all gates, then all ups
  uint8_t* rest;             // with pre [I, 2 J] of [gate | up]: four more bits of each value, [I, J] bytes
  uint8_t* codes;            // MXFP8 codes [I, 2 J] of [gate | up], or null; pre is then null
  uint8_t* scales;           // and their scales [I, 2 ceil(J / 32)]
};
// The arguments by the kind of product.  (A kernel's parameter type must not be spelled with a nameless
// enumeration's value: host and device may number nameless types differently, and then the
// host does not find the kernel.)
template <bool IS_GATED>
struct ArgsOf {
  using type = ProductArgs;
};
template <>
struct ArgsOf<true> {
  using type = GatedArgs;
};
// Row segments of grouped products: 0 holds the rows before the first group, e + 1 those of group e,
// groups + 1 those after the last group.  The first and the last are of no group and count as group
// number `groups`.
struct Rows {
  int64_t begin, end;
};
__device__ __forceinline__ Rows segment(const int32_t* off, int64_t groups, int64_t I, int64_t s) {
  const int64_t a = s == 0 ? 0 : min((int64_t)max(off[s - 1], 0), I);
  return {a, s > groups ? I : max(a, min((int64_t)off[s], I))};
}

// Finds the group and the rows of row tile t when each segment's rows are cut into tiles of
// `size`, segment after segment.  group is -1 past the last tile.  64 segments are looked at
// together, one a lane.
struct RowTile {
  int64_t group, i0, i1;
};
// The value of lane `at` (a wave-uniform lane), as a wave-uniform value.
__device__ __forceinline__ int64_t lane_value(int64_t v, int at) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, at), hi = __builtin_amdgcn_readlane((int)(v >> 32), at);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ RowTile find_tile(const int32_t* off, int64_t groups, int64_t I, int64_t t, int64_t size) {
  if (off == nullptr) return {t * size < I ? 0 : -1, t * size, min((t + 1) * size, I)};
  const int lane = threadIdx.x & 63;
  int64_t first = 0;   // tiles of the segments before this batch
  for (int64_t s0 = 0; s0 < groups + 2; s0 += 64) {
    Rows r = {0, 0};
    if (s0 + lane < groups + 2) r = segment(off, groups, I, s0 + lane);
    int64_t n = (r.end - r.begin + size - 1) / size;
    const int64_t own = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(n, d);
      if (lane >= d) n += v;
    }
    const uint64_t hit = __ballot(t < first + n && t >= first + n - own);
    if (hit != 0) {
      const int at = __builtin_ctzll(hit);
      const int64_t i0 = r.begin + (t - (first + n - own)) * size, s = s0 + at;
      return {s == 0 ? groups : s - 1, lane_value(i0, at), lane_value(min(i0 + size, r.end), at)};
    }
    first += lane_value(n, 63);
  }
  return {-1, 0, 0};
}

// Row tiles of all segments.
__device__ __forceinline__ uint32_t count_tiles(const int32_t* off, int64_t groups, int64_t I, int64_t size) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int64_t s = lane; s < groups + 2; s += 64) {
    const Rows r = segment(off, groups, I, s);
    n += (int)((r.end - r.begin + size - 1) / size);
  }
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  return __builtin_amdgcn_readfirstlane(n);
}

// s_waitcnt on the vector-memory counter alone (gfx9 encoding: vmcnt in bits 3:0 and 15:14).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// s_waitcnt lgkmcnt(0) alone.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A pointer that is the same in every lane, held in scalar registers.
__device__ __forceinline__ const uint16_t* uniform(const uint16_t* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (const uint16_t*)((uint64_t)hi << 32 | lo);
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// One operand of a tile: B_ rows of the operand by BK elements of the sum per step, copied
// straight into LDS in blocks of 1 KiB (16 bytes a lane) and read back as 16 x 32 fragments
// (lane r + 16 g: row r, elements 8 g .. 8 g + 7).
//   k along rows (T = false): a row's 128 bytes hold its BK elements; 16-byte chunk c of row R
//     lies at chunk c ^ (R / 2 % 8), so a fragment read touches every LDS bank once.
//   transposed (T = true): an LDS row holds one element of the sum for all B_ rows; its
//     32-byte segment s of element k lies at segment s ^ turn(k), and the fragment is gathered by
//     two transposing reads of 4 elements each.  Such a read takes 256 bytes at a time: two
//     4 x 16 blocks, 8 elements apart, whose rows turn() spreads over all banks.
__device__ __forceinline__ uint32_t turn(uint32_t k) { return (k & 3u) | (k >> 1 & 4u); }

template <bool T, int B_, int WAVES>
struct Operand {
  static constexpr int LOADS = B_ * BK * 2 / 1024 / WAVES;     // 1 KiB blocks per wave and step
  static constexpr uint32_t BYTES = B_ * BK * 2;
  static_assert(LOADS >= 1 && LOADS * WAVES * 1024 == (int)BYTES);
  uint32_t off[LOADS];       // byte offset of the lane's 16 bytes from the tile's base
  uint32_t kk;               // T: the lane's element of the sum in block 0; else its first one
  const uint16_t* base;
  int64_t ld;

  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int64_t i0, int64_t i1, uint32_t wave,
                                       uint32_t lane) {
    ld = ld_;
    if constexpr (!T) {
      base = uniform(p + i0 * ld);
      const uint32_t lrow = lane >> 3;
#pragma unroll
      for (int q = 0; q < LOADS; q++) {
        const uint32_t row = 8u * (wave * LOADS + q) + lrow;
        const uint32_t chunk = (lane & 7u) ^ ((row >> 1) & 7u);
        off[q] = i0 + row < i1 ? 2u * (row * (uint32_t)ld + 8u * chunk) : kOob;
      }
      // the chunk depends on the row through (row / 2) % 8 = 4 (block % 2) + lrow / 2
      kk = 0;
    } else {
      base = uniform(p + i0);
      constexpr uint32_t CH = B_ / 8;                             // chunks per LDS row
#pragma unroll
      for (int q = 0; q < LOADS; q++) {
        const uint32_t k = (wave * LOADS + q) * (64u / CH) + lane / CH;
        const uint32_t chunk = (lane % CH) ^ (2u * turn(k));
        off[q] = i0 + 8u * chunk < i1 ? 2u * (k * (uint32_t)ld + 8u * chunk) : kOob;
      }
      kk = wave * LOADS * (64u / CH) + lane / CH;
    }
  }
  // Starts load q of the step at element k of the sum.  TAIL: elements at and past k1, which are
  // less than a step away, read zero.
  template <bool TAIL>
  __device__ __forceinline__ void issue(int q, uint32_t k, uint32_t k1, uint8_t* lds, uint32_t wave, uint32_t lane) const {
    uint32_t o = off[q];
    if constexpr (TAIL) {
      uint32_t mine;
      if constexpr (!T) {
        const uint32_t row = 8u * (wave * LOADS + q) + (lane >> 3);
        mine = 8u * ((lane & 7u) ^ ((row >> 1) & 7u));
      } else {
        mine = kk + q * (64u / (B_ / 8));
      }
      if (k + mine >= k1) o = kOob;
    }
    const auto r = rsrc(T ? base + k * ld : base + k);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(lds + (wave * LOADS + q) * 1024u), 16, o, 0, 0, 0);
  }
};

// The B operand of a gated product: row R of a tile is the gate (R / 16 even) or up row of output
// 16 (R / 32) + R % 16 of the tile, so a wave's neighbouring 16 x 16 results are the gate and the up
// values of the same outputs in the same lanes.  Gate and up rows may be farther apart than 32-bit
// offsets reach: each half has its base, and an 8-row load is of one half.
template <int B_, int WAVES>
struct GatedOperand {
  static constexpr int LOADS = B_ * BK * 2 / 1024 / WAVES;
  static constexpr uint32_t BYTES = B_ * BK * 2;
  static_assert(LOADS >= 1 && LOADS * WAVES * 1024 == (int)BYTES);
  uint32_t off[LOADS];
  const uint16_t* base[2];

  __device__ __forceinline__ void init(const uint16_t* p, int64_t K, int64_t N, bool paired, int64_t n0, uint32_t wave,
                                       uint32_t lane) {
    const int64_t step = paired ? 2 * K : K;
    base[0] = uniform(p + n0 * step);
    base[1] = uniform(p + n0 * step + (paired ? K : N * K));
#pragma unroll
    for (int q = 0; q < LOADS; q++) {
      const uint32_t row = 8u * (wave * LOADS + q) + (lane >> 3), n = 16u * (row >> 5) + (row & 15u);
      const uint32_t chunk = (lane & 7u) ^ ((row >> 1) & 7u);
      off[q] = n0 + n < N ? 2u * (n * (uint32_t)step + 8u * chunk) : kOob;
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void issue(int q, uint32_t k, uint32_t k1, uint8_t* lds, uint32_t wave, uint32_t lane) const {
    uint32_t o = off[q];
    if constexpr (TAIL) {
      const uint32_t row = 8u * (wave * LOADS + q) + (lane >> 3);
      if (k + 8u * ((lane & 7u) ^ ((row >> 1) & 7u)) >= k1) o = kOob;
    }
    const auto r = rsrc(((wave * LOADS + q) & 2u ? base[1] : base[0]) + k);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(lds + (wave * LOADS + q) * 1024u), 16, o, 0, 0, 0);
  }
};

// Four elements of a 4 x 16 block (per 16 lanes) of 16-bit values in LDS, transposed.  The
// restricted pointer tells the compiler that no copy into LDS that is under way writes here;
// without it every such read would wait for all of them.
__device__ __forceinline__ v4s transposed(const uint8_t* __restrict__ p) {
  typedef __attribute__((address_space(3))) v4s* tr_ptr;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)p);
}

// A lane's fragment addresses of an operand in LDS.  Wave w of W along this operand owns TILES
// tiles of 16 rows: consecutive ones, or, transposed, every W-th one (tile i of the wave is tile
// i W + w).  The lane reads elements k = 8 g + 4 u + q of tile i at segment
//   (i W + w) ^ turn(k) = 8 (i / (8 / W)) + ((i % (8 / W)) W + w) ^ (q + 4 (g % 2)),
// whose first part is a constant of the unrolled code and whose second takes 8 / W values.
template <bool T, int B_, int W, int TILES>
struct Fragments {
  static constexpr int BASES = T ? (8 / W < TILES ? 8 / W : TILES) : 2;
  uint32_t at[BASES];
  static __device__ __forceinline__ uint32_t tile(uint32_t w, int i) { return T ? i * W + w : w * TILES + i; }
  __device__ __forceinline__ void init(uint32_t w, uint32_t lane) {
    const uint32_t g = lane >> 4, r = lane & 15u;
    if constexpr (!T) {
#pragma unroll
      for (uint32_t h = 0; h < 2; h++) at[h] = 128u * (16u * TILES * w + r) + 16u * ((4u * h + g) ^ ((r >> 1) & 7u));
    } else {
      const uint32_t q = r >> 2;
#pragma unroll
      for (uint32_t m = 0; m < BASES; m++)
        at[m] = (8u * g + q) * (2u * B_) + 32u * ((m * W + w) ^ (q + 4u * (g & 1u))) + 8u * (r & 3u);
    }
  }
  __device__ __forceinline__ v8bf read(const uint8_t* lds, int i, int h) const {
    if constexpr (!T) {
      return *reinterpret_cast<const v8bf*>(lds + at[h] + 2048u * i);
    } else {
      const uint8_t* p = lds + at[i % BASES] + 2u * B_ * 32u * h + 256 * (i / (8 / W));
      const v4s lo = transposed(p), hi = transposed(p + 8 * B_);
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Workgroup b of n: those of one XCD (b mod 8) get a contiguous run.
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n) {
  const uint32_t per = n / 8u;
  return b < 8u * per ? (b % 8u) * per + b / 8u : b;
}

constexpr uint32_t GROUP_I = 8;   // row tiles per group of the tile order

// N consecutive BF16 values, widened (zeros for a null pointer).
template <int N>
__device__ __forceinline__ void load_bf16(float (&f)[N], const uint16_t* p) {
  typedef unsigned int vec __attribute__((ext_vector_type(N / 2)));
  vec v = (vec)0u;
  if (p != nullptr) v = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int i = 0; i < N / 2; i++) {
    f[2 * i] = bf_lo(v[i]);
    f[2 * i + 1] = bf_hi(v[i]);
  }
}

template <int N>
using bf16_vec = unsigned int __attribute__((ext_vector_type(N / 2)));

// The saved pre-activation is FP16: 11 significant bits of what the backward evaluates act' at,
// where BF16 has 8; larger values are clamped to its range, where act' is 0 or 1.  The clamp keeps
// NaN (maximum and minimum give NaN where the median of three would give a bound), so that what is
// NaN in y is NaN in the gradients too.
template <int N>
__device__ __forceinline__ bf16_vec<N> pack_pre(const float (&v)[N]) {
  typedef _Float16 half2 __attribute__((ext_vector_type(2)));
  const half2 most = {(_Float16)65504.0f, (_Float16)65504.0f};
  bf16_vec<N> o;
#pragma unroll
  for (int e = 0; e < N / 2; e++) {
    const half2 h = {(_Float16)v[2 * e], (_Float16)v[2 * e + 1]};   // infinite past the range
    o[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_minimum(__builtin_elementwise_maximum(h, -most), most));
  }
  return o;
}
template <int N>
__device__ __forceinline__ bf16_vec<N> pack_row(const float (&v)[N]) {
  bf16_vec<N> o;
#pragma unroll
  for (int e = 0; e < N / 2; e++) o[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
  return o;
}

// Epilogue of N consecutive columns of one row: v holds the sums.
template <int MODE, int ACT, int N>
__device__ __forceinline__ void finish(const ProductArgs& a, int64_t group, int64_t row, int64_t col, float (&v)[N]) {
  if constexpr (MODE == FWD) {
    float bias[N], res[N];
    load_bf16(bias, a.bias != nullptr ? a.bias + group * a.J + col : nullptr);
    load_bf16(res, a.residual != nullptr ? a.residual + row * a.ld_res + col : nullptr);
#pragma unroll
    for (int e = 0; e < N; e++) v[e] += bias[e];
    if (a.pre != nullptr) *reinterpret_cast<bf16_vec<N>*>(a.pre + row * a.J + col) = pack_pre(v);
#pragma unroll
    for (int e = 0; e < N; e++) v[e] = act_of<ACT>(v[e]) + res[e];
  }
  *reinterpret_cast<bf16_vec<N>*>(a.c + (MODE == WGRAD ? group * a.c_group : 0) + row * a.ld_c + col) = pack_row(v);
}

// Stores 16 bytes at an offset of a buffer.  The offset is the lanes' alone: with a scalar offset
// besides, the compiler takes the store to have read its registers when it is issued and may write
// them in the next instruction, and lanes 12 to 15 of 16 then stored what was written.
__device__ __forceinline__ void put16(u32x4 v, __amdgpu_buffer_rsrc_t to, uint32_t offset) {
  __builtin_amdgcn_raw_buffer_store_b128(v, to, offset, 0, 0);
}

// ---- the gated epilogue ----------------------------------------------------------------------

// Four consecutive BF16 values of a bias of gates and ups: gates at n, ups J later, or pairs.
__device__ __forceinline__ void load_gated_bias(float (&g)[4], float (&u)[4], const GatedArgs& a, int64_t group, int64_t n) {
  const uint16_t* b = a.bias == nullptr || n >= a.J ? nullptr : a.bias + group * 2 * a.J;
  if (a.paired) {
    float v[8];
    load_bf16(v, b == nullptr ? nullptr : b + 2 * n);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      g[e] = v[2 * e];
      u[e] = v[2 * e + 1];
    }
  } else {
    load_bf16(g, b == nullptr ? nullptr : b + n);
    load_bf16(u, b == nullptr ? nullptr : b + a.J + n);
  }
}

// Each wave holds 32 outputs (tiles 2 q and 2 q + 1 are gate and up of outputs 16 q ..) of its rows:
// the GLU in registers, then, a row tile at a time, through the wave's piece of LDS into 16-byte
// pieces of rows.  Gate and up are kept for the gradient as BF16 with four more bits (wide_pair) or
// as MXFP8 codes of BF16 values, a block of 32 being the wave's part of a row.
constexpr uint32_t GATED_PITCH = 80, REST_PITCH = 20, GATED_LDS = 3 * 16 * GATED_PITCH + 2 * 16 * REST_PITCH;
template <int ACT, int TI, int TJ, typename FrA>
__device__ __forceinline__ void gated_epilogue(const GatedArgs& a, int64_t group, const RowTile& t, int64_t n0, uint32_t wi,
                                               uint32_t wj, uint32_t lane, uint8_t* mine, v4f (&acc)[TI][TJ]) {
  static_assert(TJ == 4, "a wave's outputs are one MXFP8 block");
  const uint32_t g = lane >> 4, r = lane & 15u, c0 = 32u * wj, ld = (uint32_t)a.ld_c, N = (uint32_t)a.J;
  const uint32_t rows = (uint32_t)(t.i1 - t.i0), NB = (N + 31u) / 32u;
  const uint32_t lrow = lane >> 2, col = c0 + 8u * (lane & 3u);    // of the lane's eight outputs once in rows
  const bool in = n0 + col < a.J, any = n0 + c0 < a.J;
  const auto rh = rsrc(uniform(a.c + t.i0 * a.ld_c + n0));
  const bool has_pre = a.pre != nullptr, has_codes = a.codes != nullptr;
  const auto rp = rsrc(uniform(has_pre ? a.pre + t.i0 * 2 * a.J + n0 : a.c));
  const auto rn = rsrc(uniform((const uint16_t*)(has_pre ? (const void*)(a.rest + t.i0 * a.J + n0 / 2) : a.c)));
  const auto rq = rsrc(uniform((const uint16_t*)(has_codes ? (const void*)(a.codes + t.i0 * 2 * a.J + n0) : a.c)));
  const auto rs = rsrc(uniform((const uint16_t*)(has_codes ? (const void*)(a.scales + t.i0 * 2 * NB + n0 / 32) : a.c)));
  const bool none = group == a.groups;   // rows of no group are zero
  float bg[2][4], bu[2][4];
#pragma unroll
  for (int q = 0; q < 2; q++) {
    if (none) {
#pragma unroll
      for (int e = 0; e < 4; e++) bg[q][e] = bu[q][e] = 0.0f;
    } else {
      load_gated_bias(bg[q], bu[q], a, group, n0 + c0 + 16u * q + 4u * g);
    }
  }
  auto through = [&](uint8_t* at, const uint32_t (&p)[2][2]) {
#pragma unroll
    for (int q = 0; q < 2; q++) *reinterpret_cast<u32x2*>(at + r * GATED_PITCH + 32 * q + 8 * g) = (u32x2){p[q][0], p[q][1]};
    return *reinterpret_cast<const u32x4*>(at + lrow * GATED_PITCH + 16 * (lane & 3u));
  };
  // a loop for each kind of what is kept: instructions are what the epilogue takes its time for ([16384, 2 x 7168,
  // 2048] with choices inside the loop 805 us, with a loop each 786)
  auto finish_rows = [&](auto KEEP) {
    constexpr bool has_pre = decltype(KEEP)::value == 1, has_codes = decltype(KEEP)::value == 2;
#pragma unroll
    for (int i = 0; i < TI; i++) {
      const uint32_t first = 16u * FrA::tile(wi, i), row = first + lrow;
      const bool ok = in && row < rows;
      uint32_t H[2][2], G[2][2] = {}, U[2][2] = {}, ng[2], nu[2];
#pragma unroll
      for (int q = 0; q < 2; q++) {
        float gate[4], up[4], h[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          gate[e] = acc[i][2 * q][e] + bg[q][e];
          up[e] = acc[i][2 * q + 1][e] + bu[q][e];
        }
        glu_of<ACT>(h, gate, up);
#pragma unroll
        for (int e = 0; e < 2; e++) {
          H[q][e] = pack_bf16(h[2 * e], h[2 * e + 1]);
          if constexpr (has_pre) {
            G[q][e] = wide_pair(gate[2 * e], gate[2 * e + 1]);
            U[q][e] = wide_pair(up[2 * e], up[2 * e + 1]);
          } else if constexpr (has_codes) {
            G[q][e] = pack_bf16(gate[2 * e], gate[2 * e + 1]);
            U[q][e] = pack_bf16(up[2 * e], up[2 * e + 1]);
          }
        }
        if constexpr (has_pre) {
          ng[q] = wide_rests(gate[0], gate[1], gate[2], gate[3]);
          nu[q] = wide_rests(up[0], up[1], up[2], up[3]);
        }
      }
      put16(through(mine, H), rh, ok ? 2u * (row * ld + col) : kOob);
      if constexpr (has_pre) {
        put16(through(mine + 16 * GATED_PITCH, G), rp, ok ? 2u * (row * 2u * N + col) : kOob);
        put16(through(mine + 32 * GATED_PITCH, U), rp, ok ? 2u * (row * 2u * N + N + col) : kOob);
        uint8_t* at = mine + 48 * GATED_PITCH;
#pragma unroll
        for (int q = 0; q < 2; q++) {
          *reinterpret_cast<uint16_t*>(at + r * REST_PITCH + 8 * q + 2 * g) = (uint16_t)ng[q];
          *reinterpret_cast<uint16_t*>(at + (16 + r) * REST_PITCH + 8 * q + 2 * g) = (uint16_t)nu[q];
        }
        // (read as vectors, which may alias the 16-bit stores)
        const uint32_t wg = as_u32(*reinterpret_cast<const u16x2*>(at + lrow * REST_PITCH + 4 * (lane & 3u)));
        const uint32_t wu = as_u32(*reinterpret_cast<const u16x2*>(at + (16 + lrow) * REST_PITCH + 4 * (lane & 3u)));
        __builtin_amdgcn_raw_buffer_store_b32(wg, rn, ok ? row * N + col / 2u : kOob, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32(wu, rn, ok ? row * N + N / 2u + col / 2u : kOob, 0, 0);
      }
      if constexpr (has_codes) {
        const uint32_t g4[4] = {G[0][0], G[0][1], G[1][0], G[1][1]}, u4[4] = {U[0][0], U[0][1], U[1][0], U[1][1]};
        uint32_t m = top_of(g4) | top_of(u4) << 16;   // over the row's four lanes
        m = pkmax(m, swz_xor16(m));
        m = pkmax(m, (uint32_t)__builtin_amdgcn_ds_bpermute((int)(4u * (lane ^ 32u)), (int)m));
        const uint32_t sg = block_scale(lo16(m)), su = block_scale(hi16(m));
        uint8_t* at = mine + 16 * GATED_PITCH;
#pragma unroll
        for (int q = 0; q < 2; q++) {
          *reinterpret_cast<uint32_t*>(at + r * 40 + 16 * q + 4 * g) = block_codes(G[q][0], G[q][1], sg);
          *reinterpret_cast<uint32_t*>(at + 640 + r * 40 + 16 * q + 4 * g) = block_codes(U[q][0], U[q][1], su);
        }
        const u32x2 cg = *reinterpret_cast<const u32x2*>(at + lrow * 40 + 8 * (lane & 3u));
        const u32x2 cu = *reinterpret_cast<const u32x2*>(at + 640 + lrow * 40 + 8 * (lane & 3u));
        __builtin_amdgcn_raw_buffer_store_b64(cg, rq, ok ? row * 2u * N + col : kOob, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(cu, rq, ok ? row * 2u * N + N + col : kOob, 0, 0);
        const uint32_t at_s = any && g == 0 && first + r < rows ? (first + r) * 2u * NB + c0 / 32u : kOob;
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)sg, rs, at_s, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)su, rs, at_s == kOob ? kOob : at_s + NB, 0, 0);
      }
    }
  };
  if (has_pre) finish_rows(std::integral_constant<int, 1>{});
  else if (has_codes) finish_rows(std::integral_constant<int, 2>{});
  else finish_rows(std::integral_constant<int, 0>{});
}

// ---- the tiled product -----------------------------------------------------------------------

// WI x WJ waves of TI x TJ tiles of 16 x 16 each: a tile of 16 WI TI rows by 16 WJ TJ columns.
//
// The smaller tiles keep NS LDS stages, each a step of BK elements.  A step's matrix work runs in two
// halves of 32 elements.  While the first half multiplies, the second half's fragments are read;
// then one barrier says both that every wave has read the stage and that the next stage has
// landed; the loads of the step NS further on go into the stage just freed and the next stage's
// first fragments are read while the second half multiplies.  A load so has NS - 1 steps to arrive.
//
// In the largest tile (NS = 2, eight waves) waves 0 .. 3, one a SIMD, read a step's fragments and start
// loads while waves 4 .. 7 multiply, and the other way round; each turn ends with a barrier.  With all
// eight in step, every wave waited for its fragments and for its loads to be taken at the same time (the
// times below 7 % longer, 2 % for the gradient of W).
// The first half reads step s in turn 2 s and multiplies in turn 2 s + 1, the second half one turn later.
// Each half has two turns to see its loads landed:
//   the first half starts in turn 2 s the loads of step s + 1 of its own rows of A and of the low columns
//     of B (both halves have read step s - 1 of those by the end of turn 2 s - 1: two stages);
//   the second half in turn 2 s + 1 those of step s + 1 of its own rows of A, which it reads in turn 2 s + 3,
//     and of step s + 2 of the high columns of B, which the first half reads in turn 2 s + 4: three stages.
// Registers hold B's fragments and half of A's; the others are read while multiplying.
//
// Bound by the matrix cores at large sizes; what is lost there is the start and the end of a tile,
// which nothing overlaps (one workgroup fills a compute unit's LDS).  Measured on an MI355X:
//   256x256  [16384, 7168, 2048] (I, J, K) alone 343 to 362 us (1.4 PFLOP/s), with bias, GELU, residual
//            and saved pre-activation 434 to 456; gradient of x 329 to 343, of W 357 to 378
//            8192^3 711 (1.55 PFLOP/s; 601 on zeros)
//            16 groups, 16384 rows, [4096, 2048]: 257 to 270, gradients 266 to 291 and 274 to 294
//            gated, [16384, 2 x 7168, 2048]: 770 to 842 with gate and up kept (716 for the product alone); 16
//            groups, 16384 rows, [2 x 2048, 2048]: 268 to 326 with them kept as MXFP8; [968, 2 x 16384, 2048] 104 to 113
//   256x128  [968, 2048, 16384] in four parts 59 us (1.1 PFLOP/s), and 7 to join them
//   128x128  [1021, 1000, 2056] in two parts 16.0 us, and 4.4 to join them
//   both gradients of it in one launch of 256x128 tiles 20.5 us (one after the other 14.6 and 13.8)
//   32x128   32 groups, 256 rows, [2048, 2048], W from memory: 49 us (5.5 TB/s); gated, [2 x 2048, 2048], 97 to 102
// Tried and slower at [16384, 7168, 2048] (forward with epilogue, eight waves in step, 500 to 540 us): 128x128 tiles 637;
// 4 waves of 128x128 798; four stages of 32 elements 558; two workgroups of 256x128 and three
// stages of 32 a compute unit 581; workgroups that stay and load the next tile during the
// epilogue 560.  With turns, workgroups that stay and start the next tile's loads before the epilogue
// gain 1 to 4% over 14 rounds of the chip and lose 1 to 2% over 7 or fewer.
//
// `block` of `blocks` is the workgroup's number among those of the product.
template <int BI, int BJ, int NS>
constexpr uint32_t kProductLds = (NS == 2 ? 2 * BI + BJ * 5 / 2 : NS * (BI + BJ)) * BK * 2;   // bytes
template <int MODE, int ACT, int WI, int WJ, int TI, int TJ, int NS>
__device__ __forceinline__ void product_tile(const typename ArgsOf<MODE == 3>::type& a, uint32_t tiles_i, uint32_t tiles_j,
                                             uint32_t splits, uint32_t block, uint32_t blocks, uint8_t* smem) {
  constexpr bool TA = MODE == WGRAD, TB = MODE == DGRAD || MODE == WGRAD;
  constexpr int BI = 16 * WI * TI, BJ = 16 * WJ * TJ, WAVES = WI * WJ;
  constexpr bool TURNS = NS == 2;
  static_assert(!TURNS || (WI == 2 && WJ % 2 == 0 && TI % 2 == 0));
  constexpr int PARTS = TURNS ? 2 : 1;   // of the waves, and of the rows and columns they load
  using OpA = Operand<TA, BI / PARTS, WAVES / PARTS>;
  using OpB = std::conditional_t<MODE == GATED, GatedOperand<BJ / PARTS, WAVES / PARTS>, Operand<TB, BJ / PARTS, WAVES / PARTS>>;
  constexpr uint32_t LDS = kProductLds<BI, BJ, NS>;
  static_assert(LDS == (TURNS ? 4 * OpA::BYTES + 5 * OpB::BYTES : NS * (OpA::BYTES + OpB::BYTES)));
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // this workgroup's tile: contiguous runs per XCD; a run goes down GROUP_I row tiles before the
  // next column tile, so that the workgroups of one XCD share operands in its L2
  if (MODE != WGRAD && a.offsets != nullptr) {   // the grid allows for more row tiles than there are
    tiles_i = count_tiles(a.offsets, a.groups, a.I, BI);
    if (block >= tiles_i * tiles_j) return;
  }
  const uint32_t per = tiles_i * tiles_j;
  // WGRAD of groups: their sums differ in length, so each XCD gets a share of every group's tiles
  const bool each = MODE == WGRAD && a.offsets != nullptr;
  uint32_t b = block, outer = each ? b / per : 0u;   // WGRAD: group; with splits: part of the sum
  b = xcd_run(b - outer * per, each ? per : MODE != WGRAD && a.offsets != nullptr ? per : blocks);
  if (!each) {
    outer = b / per;
    b -= outer * per;
  }
  const uint32_t in_group = GROUP_I * tiles_j, first_i = b / in_group * GROUP_I;
  const uint32_t gi = min(tiles_i - first_i, GROUP_I);
  const uint32_t ti = first_i + b % in_group % gi, tj = b % in_group / gi;

  RowTile t;
  int64_t group;
  uint32_t k0 = 0, k1 = (uint32_t)a.K, part = 0;
  if constexpr (MODE == WGRAD) {
    group = outer / splits;
    part = outer % splits;
    if (a.offsets != nullptr) {
      k0 = min((uint32_t)max(a.offsets[group], 0), k1);
      k1 = max(k0, min((uint32_t)max(a.offsets[group + 1], 0), k1));
    }
    t = {group, (int64_t)ti * BI, min((int64_t)(ti + 1) * BI, a.I)};
  } else {
    t = find_tile(a.offsets, a.groups, a.I, ti, BI);
    if (t.group < 0) return;
    group = t.group;
    part = outer;
    if (group == a.groups) k1 = 0;   // rows of no group
  }
  if (splits > 1) {                  // whole steps to each part
    const uint32_t steps = (k1 - k0 + BK - 1) / BK;
    const uint32_t s0 = part_begin(steps, part, splits), s1 = part_begin(steps, part + 1, splits);
    k1 = min(k1, k0 + s1 * BK);
    k0 += s0 * BK;
  }
  const int64_t width = MODE == GATED ? gated_columns(a.J) : a.J;   // columns of the sums
  const int64_t j0 = (int64_t)tj * BJ, j1 = min(j0 + BJ, width);
  const uint32_t wi = wave / WJ, wj = wave % WJ;

  OpA oa;
  OpB ob;
  const uint32_t half = TURNS ? wave / (WAVES / 2) : 0u, mate = TURNS ? wave % (WAVES / 2) : wave;
  oa.init(a.a, a.ld_a, t.i0 + half * (BI / 2), t.i1, mate, lane);
  const bool none = MODE != WGRAD && group == a.groups;   // rows of no group
  if constexpr (MODE == GATED) {
    ob.init(none ? a.b : a.b + group * a.b_group, a.ld_b, a.J, a.paired != 0, j0 / 2 + half * (BJ / 4), mate, lane);
  } else {
    ob.init(a.b + group * a.b_group, a.ld_b, j0 + half * (BJ / 2), j1, mate, lane);
    if (none) ob.base = a.b;
  }
  using FrA = Fragments<TA, BI / PARTS, WI / PARTS, TI>;
  using FrB = Fragments<TB, BJ / PARTS, WJ / PARTS, TJ>;
  FrA fa;
  FrB fb;
  fa.init(TURNS ? 0 : wi, lane);
  fb.init(TURNS ? wj % (WJ / PARTS) : wj, lane);
  // row tile i and column tile j of a wave in the workgroup's tile
  struct Rows {
    static __device__ __forceinline__ uint32_t tile(uint32_t w, int i) { return TURNS ? TI * w + i : FrA::tile(w, i); }
  };
  struct Cols {
    static __device__ __forceinline__ uint32_t tile(uint32_t w, int j) {
      return TURNS ? w / (WJ / PARTS) * (BJ / 32) + FrB::tile(w % (WJ / PARTS), j) : FrB::tile(w, j);
    }
  };

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; i++)
#pragma unroll
    for (int j = 0; j < TJ; j++) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  v8bf xa[2][TI], xb[2][TJ];
  auto multiply = [&](int h) {
#pragma unroll
    for (int i = 0; i < TI; i++)
#pragma unroll
      for (int j = 0; j < TJ; j++)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[h][j], xa[h][i], acc[i][j], 0, 0, 0);
  };
  // The scheduler's groups: a fragment read to every few products, so that neither the matrix
  // cores nor LDS wait for a burst of the other.
  constexpr int READS = TI * (TA ? 2 : 1) + TJ * (TB ? 2 : 1), PRODUCTS = TI * TJ;
  constexpr int LOADS = OpA::LOADS + OpB::LOADS;
  enum { G_MFMA = 0x8, G_VMEM = 0x10, G_DS_READ = 0x100 };
  // A ring of stages, whose present one starts at byte `now`.  Every step starts the loads of one
  // step, real or not, so that the count of loads under way is known.
  constexpr uint32_t STAGE = OpA::BYTES + OpB::BYTES;
  uint32_t now = 0;
  auto issue_at = [&](uint32_t k, uint32_t at, auto TAIL) {
#pragma unroll
    for (int q = 0; q < OpA::LOADS; q++) oa.template issue<decltype(TAIL)::value>(q, k, k1, smem + at, wave, lane);
#pragma unroll
    for (int q = 0; q < OpB::LOADS; q++)
      ob.template issue<decltype(TAIL)::value>(q, k, k1, smem + at + OpA::BYTES, wave, lane);
  };
  auto read_at = [&](uint32_t at, int h) {
#pragma unroll
    for (int i = 0; i < TI; i++) xa[h][i] = fa.read(smem + at, i, h);
#pragma unroll
    for (int j = 0; j < TJ; j++) xb[h][j] = fb.read(smem + at + OpA::BYTES, j, h);
  };
  auto ring_step = [&](auto&& feed) {
    const uint32_t next = now == (NS - 1) * STAGE ? 0u : now + STAGE;
    read_at(now, 1);
    multiply(0);
#pragma unroll
    for (int q = 0; q < READS; q++) {
      __builtin_amdgcn_sched_group_barrier(G_DS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(G_MFMA, PRODUCTS / READS, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<(NS - 2) * LOADS>();
    lds_barrier();
    feed(now);
    read_at(next, 0);
    multiply(1);
#pragma unroll
    for (int q = 0; q < LOADS; q++) {
      __builtin_amdgcn_sched_group_barrier(G_VMEM, 1, 0);
      __builtin_amdgcn_sched_group_barrier(G_MFMA, 1, 0);
    }
#pragma unroll
    for (int q = 0; q < READS; q++) {
      __builtin_amdgcn_sched_group_barrier(G_DS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(G_MFMA, (PRODUCTS - LOADS) / READS > 1 ? (PRODUCTS - LOADS) / READS : 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();
    now = next;
  };

  if constexpr (NS > 2) {
    if (k0 < k1) {
      // The steps are taken in turn from step `turn` on, those before it last.  Workgroups that all
      // read the same columns of many rows meet in few memory channels when the rows are a power of
      // two apart; each XCD and group starts elsewhere (within an XCD the workgroups stay together,
      // for what they share in its L2).  32 groups of [8, 2048] x [2048, 2048]: 65 -> 50 us.  A
      // partial step is the last one, unless every step may be partial (ANY).  Gradients without groups
      // begin at the beginning, so that their bits do not depend on the tile size, which in turn may depend on
      // whether the other gradient is formed too; of 26 shapes none took longer so.
      constexpr bool ANY = BI <= 32;
      const uint32_t steps = (k1 - k0 + BK - 1) / BK, whole = (k1 - k0) / BK;
      const bool turned = (ANY || whole == steps) && ((MODE != DGRAD && MODE != WGRAD) || a.offsets != nullptr);
      const uint32_t turn = turned ? (3u * (block % 8u) + (uint32_t)group) % steps : 0u;
      uint32_t k = k0 + turn * BK, left = steps;
      auto advance = [&] { k = k + BK < k1 ? k + BK : k0; };
      auto feed = [&](uint32_t at) {
        issue_at(left > 0 ? k : k1, at, std::true_type{});
        left -= left > 0;
        advance();
      };
      auto feed_whole = [&](uint32_t at) {
        issue_at(k, at, std::false_type{});
        advance();
      };
#pragma unroll
      for (uint32_t q = 0; q < NS; q++) feed(q * STAGE);
      wait_vm<(NS - 1) * LOADS>();
      lds_barrier();
      read_at(0, 0);
      wait_lds();
      uint32_t s = 0;
      if (!ANY || whole == steps)
        for (; s + NS < whole; s++) ring_step(feed_whole);
      left = left > 0 ? steps - s - NS : 0;
      for (; s < steps; s++) ring_step(feed);
      wait_vm<0>();   // the stages hold the sums next
      lds_barrier();
    }
  } else if (k0 < k1) {
    // A: two stages of both halves' rows; B's low columns: two, high columns: three
    constexpr uint32_t B_LOW = 4 * OpA::BYTES, B_HIGH = B_LOW + 2 * OpB::BYTES;
    auto load = [&](const auto& op, uint32_t k, uint8_t* to, auto TAIL) {
#pragma unroll
      for (int q = 0; q < std::decay_t<decltype(op)>::LOADS; q++)
        op.template issue<decltype(TAIL)::value>(q, k, k1, to, mate, lane);
    };
    constexpr std::true_type any{};
    constexpr std::false_type whole{};
    load(oa, k0, smem + half * OpA::BYTES, any);
    if (half == 0) {
      load(ob, k0, smem + B_LOW, any);
    } else {
      load(ob, k0, smem + B_HIGH, any);
      load(ob, min(k0 + BK, k1), smem + B_HIGH + OpB::BYTES, any);
    }
    wait_vm<0>();
    lds_barrier();
    auto turns = [&](auto SECOND) {
      constexpr bool second = decltype(SECOND)::value;
      if (second) lds_barrier();
      uint32_t third = 0;   // the step's stage of B's high columns
      auto step = [&](uint32_t k, uint32_t odd, auto TAIL) {
        const uint8_t *const pa = smem + odd * (2 * OpA::BYTES) + half * OpA::BYTES;
        const uint8_t *const pb = smem + (wj < WJ / 2 ? B_LOW + odd * OpB::BYTES : B_HIGH + third * OpB::BYTES);
        v8bf ya[2][TI / 2], yb[2][TJ];
#pragma unroll
        for (int j = 0; j < TJ; j++)
#pragma unroll
          for (int h = 0; h < 2; h++) yb[h][j] = fb.read(pb, j, h);
#pragma unroll
        for (int i = 0; i < TI / 2; i++)
#pragma unroll
          for (int h = 0; h < 2; h++) ya[h][i] = fa.read(pa, i, h);
        __builtin_amdgcn_sched_barrier(0);   // these reads come back while the loads are started
        const uint32_t k_a = min(k + BK, k1), k_b = second ? min(k + 2 * BK, k1) : k_a;   // of the loads
        uint8_t* const to_a = smem + (odd ^ 1u) * (2 * OpA::BYTES) + half * OpA::BYTES;
        uint8_t* const to_b =
            smem + (second ? B_HIGH + (third == 0 ? 2u : third - 1u) * OpB::BYTES : B_LOW + (odd ^ 1u) * OpB::BYTES);
        load(oa, k_a, to_a, TAIL);
        load(ob, k_b, to_b, TAIL);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < TI; i++) {
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int j = 0; j < TJ; j++)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(yb[h][j], ya[h][i % (TI / 2)], acc[i][j], 0, 0, 0);
          if (i < TI / 2) {
#pragma unroll
            for (int h = 0; h < 2; h++) ya[h][i] = fa.read(pa, TI / 2 + i, h);
          }
        }
        // the products stay in this turn
#pragma unroll
        for (int i = 0; i < TI; i++)
#pragma unroll
          for (int j = 0; j < TJ; j++) asm volatile("" : "+v"(acc[i][j]));
#pragma unroll
        for (int i = 0; i < TI / 2; i++) {   // the fragments just done with give way to those of the high rows
          __builtin_amdgcn_sched_group_barrier(G_MFMA, 2 * TJ, 0);
          __builtin_amdgcn_sched_group_barrier(G_DS_READ, TA ? 4 : 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(G_MFMA, TI * TJ, 0);
        __builtin_amdgcn_s_setprio(0);
        wait_vm<0>();
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        third = third == 2 ? 0u : third + 1u;
      };
      uint32_t k = k0;
      for (; k + 4 * BK <= k1; k += 2 * BK) {
        step(k, 0, whole);
        step(k + BK, 1, whole);
      }
      for (uint32_t odd = 0; k < k1; k += BK, odd ^= 1u) step(k, odd, any);
      if (!second) lds_barrier();
    };
    if (half != 0) turns(std::true_type{});
    else turns(std::false_type{});
    wait_vm<0>();   // the stages hold the sums next
    lds_barrier();
  }

  // acc[i][j][e] is C at row r of its row tile and column 4 g + e of its column tile.  Rows and
  // columns past the tile's are given an offset that the buffer's bounds drop.
  const uint32_t g = lane >> 4, r = lane & 15u;
  const uint32_t rows = (uint32_t)(t.i1 - t.i0), cols = (uint32_t)(j1 - j0);
  if (splits > 1) {
    const int64_t at = (MODE == WGRAD ? part * a.groups + group : (int64_t)part) * a.I + t.i0;
    const auto rw = rsrc(uniform((const uint16_t*)(a.work + at * width + j0)));
#pragma unroll
    for (int i = 0; i < TI; i++) {
      const uint32_t first = 16u * Rows::tile(wi, i);
#pragma unroll
      for (int j = 0; j < TJ; j++) {
        const uint32_t col = 16u * Cols::tile(wj, j) + 4u * g;
        const uint32_t o = first + r < rows && col < cols ? 4u * ((first + r) * (uint32_t)width + col) : kOob;
        put16(__builtin_bit_cast(u32x4, acc[i][j]), rw, o);
      }
    }
    return;
  }
  if constexpr (MODE == GATED) {
    static_assert(WAVES * GATED_LDS <= LDS);
    gated_epilogue<ACT, TI, TJ, Rows>(a, group, t, j0 / 2, wi, wj, lane, smem + wave * GATED_LDS, acc);
    return;
  }
  // A row tile's 16 x (16 TJ) sums go through the wave's own piece of LDS, so that a lane gets 8
  // consecutive columns of a row: 16-byte loads and stores.  (No wave reads the stages any
  // more: the last step's barrier comes after its last read.)
  constexpr uint32_t PITCH = 16 * TJ + 4, CH = 2 * TJ, ROWS = 64 / CH, PASSES = 16 / ROWS;   // floats; lanes a row
  static_assert(WAVES * 16 * PITCH * 4 <= LDS);
  float* const mine = reinterpret_cast<float*>(smem) + wave * (16 * PITCH);
  const uint32_t cc = 8u * (lane % CH), lrow = lane / CH;
  const uint32_t col = 16u * Cols::tile(wj, cc / 16) + cc % 16u;
  const uint32_t left = col < cols ? rows - min(rows, lrow) : 0u;   // of the lane's rows lrow + 16 tile + ROWS p
  // the place of pass p of row tile i in a matrix whose rows are ld apart
  auto place = [&](uint32_t ld, int i, uint32_t p) {
    const uint32_t first = 16u * Rows::tile(wi, i) + ROWS * p;
    return first < left ? 2u * (lrow * ld + col) + 2u * first * ld : kOob;
  };
  const uint32_t ld_c = (uint32_t)a.ld_c, J = (uint32_t)a.J;
  const auto rc = rsrc(uniform(a.c + (MODE == WGRAD ? group * a.c_group : 0) + t.i0 * a.ld_c + j0));
  const bool has_pre = MODE == FWD && a.pre != nullptr;
  const auto rp = rsrc(uniform(has_pre ? a.pre + t.i0 * a.J + j0 : a.c));
  if (MODE == FWD && none) {   // rows of no group are zero
#pragma unroll
    for (int i = 0; i < TI; i++)
#pragma unroll
      for (uint32_t p = 0; p < PASSES; p++) {
        put16((u32x4)0u, rc, place(ld_c, i, p));
        if (has_pre) put16((u32x4)0u, rp, place(J, i, p));
      }
    return;
  }
  float bias[8];
  u32x4 res[TI][PASSES];
  if constexpr (MODE == FWD) {
    load_bf16(bias, col < cols && a.bias != nullptr ? a.bias + group * a.J + j0 + col : nullptr);
    if (a.residual != nullptr) {
      const uint32_t ld = (uint32_t)a.ld_res;
      const auto rr = rsrc(uniform(a.residual + t.i0 * a.ld_res + j0));
#pragma unroll
      for (int i = 0; i < TI; i++)
#pragma unroll
        for (uint32_t p = 0; p < PASSES; p++)
          res[i][p] = __builtin_amdgcn_raw_buffer_load_b128(rr, place(ld, i, p), 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < TI; i++)
#pragma unroll
        for (uint32_t p = 0; p < PASSES; p++) res[i][p] = (u32x4)0u;
    }
  }
#pragma unroll
  for (int i = 0; i < TI; i++) {
#pragma unroll
    for (int j = 0; j < TJ; j++) *reinterpret_cast<v4f*>(mine + r * PITCH + 16 * j + 4 * g) = acc[i][j];
#pragma unroll
    for (uint32_t p = 0; p < PASSES; p++) {
      const float* q = mine + (ROWS * p + lrow) * PITCH + cc;
      const v4f lo = *reinterpret_cast<const v4f*>(q), hi = *reinterpret_cast<const v4f*>(q + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      if constexpr (MODE == FWD) {
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] += bias[e];
        if (has_pre) put16(pack_pre(v), rp, place(J, i, p));
#pragma unroll
        for (int e = 0; e < 8; e++)
          v[e] = act_of<ACT>(v[e]) + (e % 2 == 0 ? bf_lo(res[i][p][e / 2]) : bf_hi(res[i][p][e / 2]));
      }
      put16(pack_row(v), rc, place(ld_c, i, p));
    }
  }
}

template <int MODE, int ACT, int WI, int WJ, int TI, int TJ, int NS>
__global__ __launch_bounds__(64 * WI * WJ) void k_product(typename ArgsOf<MODE == 3>::type a,
                                                          uint32_t tiles_i, uint32_t tiles_j, uint32_t splits) {
  static_assert(GATED == 3);
  __shared__ __attribute__((aligned(16))) uint8_t smem[kProductLds<16 * WI * TI, 16 * WJ * TJ, NS>];
  product_tile<MODE, ACT, WI, WJ, TI, TJ, NS>(a, tiles_i, tiles_j, splits, blockIdx.x, gridDim.x, smem);
}

// Joins the parts of split sums and finishes them: eight columns a thread, the parts in order.
// Bound by memory (the parts are in the caches): [968, 2048] in four parts 7.3 us.
template <int MODE, int ACT>
__global__ __launch_bounds__(256) void k_product_join(ProductArgs a, uint32_t splits) {
  const int64_t rows = MODE == WGRAD ? a.groups * a.I : a.I, n = rows * a.J / 8;
  for (int64_t q = 256 * (int64_t)blockIdx.x + threadIdx.x; q < n; q += 256 * (int64_t)gridDim.x) {
    const int64_t row = q / (a.J / 8), col = 8 * (q % (a.J / 8));
    v4f lo = (v4f)0.0f, hi = (v4f)0.0f;
    for (uint32_t p = 0; p < splits; p++) {
      const v4f* src = reinterpret_cast<const v4f*>(a.work + (p * rows + row) * a.J + col);
      lo += src[0];
      hi += src[1];
    }
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    finish<MODE, ACT, 8>(a, MODE == WGRAD ? row / a.I : 0, MODE == WGRAD ? row % a.I : row, col, v);
  }
}

// ---- few rows --------------------------------------------------------------------------------

// The forward for up to 8 rows of one group: a pass over W at memory speed, with no barrier in it.
// A wave takes 8 rows of W (columns of C) and multiplies them, straight from memory, as 16 x 16 x 32
// tiles against the rows of x; a tile's other 8 rows (and columns, of x) are the same ones 32
// elements on: the products of matching halves add up to the result, the others are dropped, and a
// load takes 128 bytes of a row.  KW waves share the sum, taking chunks of 128 elements in turn, and
// join through LDS, so a call is one launch whatever its extents.  The next chunks of W are in
// flight while the present ones are multiplied.  [1, 2048, 16384]: 13.2 to 14.9 us (4.5 to 5.1 TB/s).
// grid: column tiles of FEW_COLS FEW_WAVES / KW
template <int ACT, int KW>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_few_rows(ProductArgs a) {
  __shared__ v4f sums[FEW_WAVES][64];
  constexpr int U = 4, STEPS = 2;   // chunks per stage; tiles per chunk
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = FEW_COLS * ((int64_t)blockIdx.x * (FEW_WAVES / KW) + wave / KW);
  const uint32_t k1 = (uint32_t)a.K, first = FEW_CHUNK * (wave % KW), stride = FEW_CHUNK * KW;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n0 < a.J && first < k1) {
    const uint32_t r = lane & 7u, mine = 8u * (lane >> 4) + 32u * (lane >> 3 & 1u);   // the lane's row; its elements
    const uint32_t wo = n0 + r < a.J ? 2u * (r * (uint32_t)a.ld_b + mine) : kOob;
    const uint32_t xo = r < a.I ? 2u * (r * (uint32_t)a.ld_a + mine) : kOob;
    const auto rw = rsrc(uniform(a.b + n0 * a.ld_b)), rx = rsrc(uniform(a.a));
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
    auto step = [&](uint32_t k, int s) {
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
      step(k, 0);
      if (k + stride * U < k1) step(k + stride * U, 1);
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave % KW != 0 || (lane & 40u) != 0) return;   // results are in rows and columns 0 .. 7 of the tile
  v4f s = (v4f)0.0f;
#pragma unroll
  for (int w = 0; w < KW; w++) s += sums[wave + w][lane] + sums[wave + w][lane + 40];   // and 8 .. 15
  const int64_t row = lane & 15u, col = n0 + 4 * (lane >> 4);
  if (row >= a.I || col >= a.J) return;
  float v[4] = {s[0], s[1], s[2], s[3]};
  finish<FWD, ACT, 4>(a, 0, row, col, v);
}

// ---- launches ----------------------------------------------------------------------------

int64_t product_work_bytes(int mode, int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped) {
  const ProductPlan p = plan_product(mode, I, J, K, groups, grouped);
  return p.splits > 1 ? 4 * p.splits * (mode == WGRAD ? groups : 1) * I * J : 0;
}

template <int MODE, int ACT>
hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  const ProductPlan p = plan_product(MODE, a.I, a.J, a.K, a.groups, a.offsets != nullptr);
  hipError_t e;
  if (p.kind == FEW) {
    auto go = [&](auto KW) {
      return launch_kernel(k_few_rows<ACT, decltype(KW)::value>, dim3((unsigned)p.tiles_j), dim3(64 * FEW_WAVES), s, a);
    };
    return p.share == 1   ? go(std::integral_constant<int, 1>{})
           : p.share == 2 ? go(std::integral_constant<int, 2>{})
           : p.share == 4 ? go(std::integral_constant<int, 4>{})
                          : go(std::integral_constant<int, 8>{});
  } else {
    const unsigned n = (unsigned)(p.tiles_i * p.tiles_j * p.splits * (MODE == WGRAD ? a.groups : 1));
    auto go = [&](auto KIND) {
      constexpr TileShape t = kShape[decltype(KIND)::value];
      return launch_kernel(k_product<MODE, ACT, t.wi, t.wj, t.ti, t.tj, t.stages>, dim3(n), dim3(64 * t.wi * t.wj), s,
                           a, (uint32_t)p.tiles_i, (uint32_t)p.tiles_j, (uint32_t)p.splits);
    };
    e = p.kind == TILE_256       ? go(std::integral_constant<int, TILE_256>{})
        : p.kind == TILE_256_128 ? go(std::integral_constant<int, TILE_256_128>{})
        : p.kind == TILE_128     ? go(std::integral_constant<int, TILE_128>{})
                                 : go(std::integral_constant<int, MODE == FWD ? TILE_32 : TILE_128>{});
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t octets = (MODE == WGRAD ? a.groups : 1) * a.I * a.J / 8;
  return launch_kernel(k_product_join<MODE, ACT>, dim3(grid_for(ceil_div(octets, 256), 4096)), dim3(256), s, a,
                       (uint32_t)p.splits);
}

}  // namespace
}  // namespace glu
