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
#include "ffn_split.h"

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
  float* work;               // split sums: [parts, rows of C, J]
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

constexpr uint32_t BK = 64;   // elements of the sum per step: one 128-byte line of a row

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

// WI x WJ waves of TI x TJ tiles of 16 x 16 each: a tile of 16 WI TI rows by 16 WJ TJ columns.
//
// NS LDS stages, each a step of BK elements.  A step's matrix work runs in two halves of 32
// elements.  While the first half multiplies, the second half's fragments are read; then one
// barrier says both that every wave has read the stage and that the next stage has landed;
// the loads of the step NS further on go into the stage just freed and the next stage's first
// fragments are read while the second half multiplies.  A load so has NS - 1 steps to arrive.
//
// Bound by the matrix cores at large sizes; what is lost there is the start and the end of a tile,
// which nothing overlaps (one workgroup fills a compute unit's LDS).  Measured on an MI355X:
//   256x256  [16384, 7168, 2048] (I, J, K) alone 364 to 373 us (1.3 PFLOP/s), with bias, GELU, residual
//            and saved pre-activation 488 to 506; gradient of x 377 to 388, of W 408 to 410
//            16 groups, 16384 rows, [4096, 2048]: 290 to 323, gradients 296 to 329 and 296 to 326
//   256x128  [968, 2048, 16384] in four parts 59 us (1.1 PFLOP/s), and 7 to join them
//   128x128  [1021, 1000, 2056] in four parts 14.9 us, and 5.6 to join them
//   32x128   32 groups, 256 rows, [2048, 2048], W from memory: 49 us (5.5 TB/s)
// Tried and slower at [16384, 7168, 2048] (forward with epilogue, 500 to 540 us at the time): 128x128 tiles 637;
// 4 waves of 128x128 798; four stages of 32 elements 558; two workgroups of 256x128 and three
// stages of 32 a compute unit 581; workgroups that stay and load the next tile during the
// epilogue 560.
template <int MODE, int ACT, int WI, int WJ, int TI, int TJ, int NS>
__global__ __launch_bounds__(64 * WI * WJ) void k_product(ProductArgs a, uint32_t tiles_i, uint32_t tiles_j,
                                                          uint32_t splits) {
  constexpr bool TA = MODE == WGRAD, TB = MODE != FWD;
  constexpr int BI = 16 * WI * TI, BJ = 16 * WJ * TJ, WAVES = WI * WJ;
  using OpA = Operand<TA, BI, WAVES>;
  using OpB = Operand<TB, BJ, WAVES>;
  // both stages of A, then both of B: every fragment read's place is within the 16-bit offset
  // of a read instruction from the lane's base
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * (OpA::BYTES + OpB::BYTES)];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // this workgroup's tile: contiguous runs per XCD; a run goes down GROUP_I row tiles before the
  // next column tile, so that the workgroups of one XCD share operands in its L2
  if (MODE != WGRAD && a.offsets != nullptr) {   // the grid allows for more row tiles than there are
    tiles_i = count_tiles(a.offsets, a.groups, a.I, BI);
    if (blockIdx.x >= tiles_i * tiles_j) return;
  }
  const uint32_t per = tiles_i * tiles_j;
  // WGRAD of groups: their sums differ in length, so each XCD gets a share of every group's tiles
  const bool each = MODE == WGRAD && a.offsets != nullptr;
  uint32_t b = blockIdx.x, outer = each ? b / per : 0u;   // WGRAD: group; with splits: part of the sum
  b = xcd_run(b - outer * per, each ? per : MODE != WGRAD && a.offsets != nullptr ? per : gridDim.x);
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
  const int64_t j0 = (int64_t)tj * BJ, j1 = min(j0 + BJ, a.J);
  const uint32_t wi = wave / WJ, wj = wave % WJ;

  OpA oa;
  OpB ob;
  oa.init(a.a, a.ld_a, t.i0, t.i1, wave, lane);
  ob.init(a.b + group * a.b_group, a.ld_b, j0, j1, wave, lane);
  if (MODE != WGRAD && group == a.groups) ob.base = a.b;
  using FrA = Fragments<TA, BI, WI, TI>;
  using FrB = Fragments<TB, BJ, WJ, TJ>;
  FrA fa;
  FrB fb;
  fa.init(wi, lane);
  fb.init(wj, lane);

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; i++)
#pragma unroll
    for (int j = 0; j < TJ; j++) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  uint8_t *const sa = smem, *const sb = smem + 2 * OpA::BYTES;
  auto issue = [&](uint32_t k, int stage) {
#pragma unroll
    for (int q = 0; q < OpA::LOADS; q++) oa.template issue<false>(q, k, k1, sa + stage * OpA::BYTES, wave, lane);
#pragma unroll
    for (int q = 0; q < OpB::LOADS; q++) ob.template issue<false>(q, k, k1, sb + stage * OpB::BYTES, wave, lane);
  };
  auto issue_tail = [&](uint32_t k, int stage) {
#pragma unroll
    for (int q = 0; q < OpA::LOADS; q++) oa.template issue<true>(q, k, k1, sa + stage * OpA::BYTES, wave, lane);
#pragma unroll
    for (int q = 0; q < OpB::LOADS; q++) ob.template issue<true>(q, k, k1, sb + stage * OpB::BYTES, wave, lane);
  };
  auto start = [&](uint32_t k, int stage) {   // the loads of the step at k, if there is one
    if (k + BK <= k1) issue(k, stage);
    else if (k < k1) issue_tail(k, stage);
  };
  v8bf xa[2][TI], xb[2][TJ];
  auto read = [&](int stage, int h) {
#pragma unroll
    for (int i = 0; i < TI; i++) xa[h][i] = fa.read(sa + stage * OpA::BYTES, i, h);
#pragma unroll
    for (int j = 0; j < TJ; j++) xb[h][j] = fb.read(sb + stage * OpB::BYTES, j, h);
  };
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
  auto step = [&](uint32_t k, int stage, auto FULL) {
    read(stage, 1);
    multiply(0);
#pragma unroll
    for (int q = 0; q < READS; q++) {
      __builtin_amdgcn_sched_group_barrier(G_DS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(G_MFMA, PRODUCTS / READS, 0);
    }
    __builtin_amdgcn_sched_barrier(0);   // the products above are not to sink below the wait
    wait_vm<0>();
    lds_barrier();
    if constexpr (decltype(FULL)::value) {   // at least two whole steps follow: no branches
      issue(k + 2 * BK, stage);
      read(1 - stage, 0);
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
    } else {
      start(k + 2 * BK, stage);
      if (k + BK < k1) read(1 - stage, 0);
      multiply(1);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();   // long since arrived; said here so that the loop's head waits for no more
  };

  // More stages: a ring, whose present stage starts at byte `now`.  Every step starts the loads of
  // one step, real or not, so that the count of loads under way is known.
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
      // partial step is the last one, unless every step may be partial (ANY).
      constexpr bool ANY = BI <= 32;
      const uint32_t steps = (k1 - k0 + BK - 1) / BK, whole = (k1 - k0) / BK;
      const uint32_t turn = ANY || whole == steps ? (3u * (blockIdx.x % 8u) + (uint32_t)group) % steps : 0u;
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
    start(k0, 0);
    start(k0 + BK, 1);
    if (k0 + 2 * BK <= k1) wait_vm<LOADS>();   // of the second step's
    else wait_vm<0>();
    lds_barrier();
    read(0, 0);
    wait_lds();
    uint32_t k = k0;
    for (; k + 4 * BK <= k1; k += 2 * BK) {
      step(k, 0, std::true_type{});
      step(k + BK, 1, std::true_type{});
    }
    for (; k < k1; k += 2 * BK) {
      step(k, 0, std::false_type{});
      if (k + BK < k1) step(k + BK, 1, std::false_type{});
    }
  }

  // acc[i][j][e] is C at row r of its row tile and column 4 g + e of its column tile.  Rows and
  // columns past the tile's are given an offset that the buffer's bounds drop.
  const uint32_t g = lane >> 4, r = lane & 15u;
  const uint32_t rows = (uint32_t)(t.i1 - t.i0), cols = (uint32_t)(j1 - j0);
  if (splits > 1) {
    const int64_t at = (MODE == WGRAD ? part * a.groups + group : (int64_t)part) * a.I + t.i0;
    const auto rw = rsrc(uniform((const uint16_t*)(a.work + at * a.J + j0)));
#pragma unroll
    for (int i = 0; i < TI; i++) {
      const uint32_t first = 16u * FrA::tile(wi, i);
#pragma unroll
      for (int j = 0; j < TJ; j++) {
        const uint32_t col = 16u * FrB::tile(wj, j) + 4u * g;
        const uint32_t o = first + r < rows && col < cols ? 4u * ((first + r) * (uint32_t)a.J + col) : kOob;
        put16(__builtin_bit_cast(u32x4, acc[i][j]), rw, o);
      }
    }
    return;
  }
  // A row tile's 16 x (16 TJ) sums go through the wave's own piece of LDS, so that a lane gets 8
  // consecutive columns of a row: 16-byte loads and stores.  (No wave reads the stages any
  // more: the last step's barrier comes after its last read.)
  constexpr uint32_t PITCH = 16 * TJ + 4, CH = 2 * TJ, ROWS = 64 / CH, PASSES = 16 / ROWS;   // floats; lanes a row
  static_assert(WAVES * 16 * PITCH * 4 <= sizeof(smem));
  float* const mine = reinterpret_cast<float*>(smem) + wave * (16 * PITCH);
  const uint32_t cc = 8u * (lane % CH), lrow = lane / CH;
  const uint32_t col = 16u * FrB::tile(wj, cc / 16) + cc % 16u;
  const uint32_t left = col < cols ? rows - min(rows, lrow) : 0u;   // of the lane's rows lrow + 16 tile + ROWS p
  // the place of pass p of row tile i in a matrix whose rows are ld apart
  auto place = [&](uint32_t ld, int i, uint32_t p) {
    const uint32_t first = 16u * FrA::tile(wi, i) + ROWS * p;
    return first < left ? 2u * (lrow * ld + col) + 2u * first * ld : kOob;
  };
  const uint32_t ld_c = (uint32_t)a.ld_c, J = (uint32_t)a.J;
  const auto rc = rsrc(uniform(a.c + (MODE == WGRAD ? group * a.c_group : 0) + t.i0 * a.ld_c + j0));
  const bool has_pre = MODE == FWD && a.pre != nullptr;
  const auto rp = rsrc(uniform(has_pre ? a.pre + t.i0 * a.J + j0 : a.c));
  if (MODE == FWD && group == a.groups) {   // rows of no group are zero
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
constexpr int FEW_WAVES = 8, FEW_ROWS = 8, FEW_COLS = 8, FEW_CHUNK = 128;

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

// ---- which kernel ----------------------------------------------------------------------------

// The tiled kernel's sizes: waves and 16 x 16 tiles a wave along the rows and the columns, LDS
// stages.  The larger the tile, the fewer bytes go into LDS for a product (L1 delivers 64 bytes a
// cycle: half the products' time at 256 x 256) and the more of the chip idles at the end.
//   32 x 128, two workgroups a compute unit: a few rows of each of many groups, a pass over W.
struct TileShape {
  int wi, wj, ti, tj, stages;
  constexpr int rows() const { return 16 * wi * ti; }
  constexpr int cols() const { return 16 * wj * tj; }
};
enum { TILE_256, TILE_256_128, TILE_128, TILE_32, FEW };
constexpr TileShape kShape[4] = {{2, 4, 8, 4, 2}, {4, 2, 4, 4, 3}, {2, 4, 4, 2, 3}, {1, 4, 2, 2, 4}};
struct ProductPlan {
  int kind;
  int64_t share;             // FEW: waves sharing a sum
  int64_t tiles_i, tiles_j, splits;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a tile takes, in microseconds a step of BK elements and for its start and end, from calls of
// one round of workgroups (2048 to 8192 rows, sums of 1024 to 8192 elements), and what joining the
// parts of a split sum takes.  The least total over the first three sizes decides.  Measured for
// [I, J, K], 256x256 / 256x128 / 128x128:
//   [ 1000, 1000, 1000]  24.8 / 15.8 / 11.2      [ 4096, 4096, 1024]  33.2 /  41.6 /  45.7
//   [  968, 2048,16384]   278 / 65.8 / 72.0      [ 4096, 4096, 4096]  99.2 / 113.7 / 136.3
//   [ 2048, 4096, 4096]  87.6 / 58.2 / 69.1      [16384, 2048, 2048]   107 /   126 /   151
// (of 33 such shapes the rule takes the fastest of the three on 32 and is 0.5% behind on one).
constexpr int64_t kUnits = 256;
constexpr double kStepUs[3] = {1.29, 0.85, 0.5}, kTileUs[3] = {15.0, 5.0, 4.0}, kJoinUs = 2.5, kJoinTBps = 8.0;
constexpr int64_t kLeastPart = 512;   // elements of a split sum's part: 256 costs up to 5 us more, and gains 0.5

// A rule on extents alone, so that the scratch memory of split sums can be sized before the
// launch.
ProductPlan plan_product(int mode, int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped) {
  ProductPlan p{};
  p.splits = 1;
  if (I == 0 || J == 0) return p;   // nothing to launch
  if (mode == FWD && !grouped && I <= FEW_ROWS) {
    // [I, 2048, 16384], few rows against 128x128 tiles: 14.7 / 20.7 us for one row, 18.4 / 21.3 for 8
    p.kind = FEW;
    // waves sharing a sum: as few as give 16 waves a compute unit, with four chunks or more each
    const int64_t cols = ceil_div(J, FEW_COLS);
    p.share = 1;
    while (p.share < FEW_WAVES && cols * p.share < 16 * kUnits && K >= 8 * p.share * FEW_CHUNK) p.share *= 2;
    p.tiles_j = ceil_div(cols * p.share, FEW_WAVES);
    return p;
  }
  if (mode == FWD && grouped && I <= kShape[TILE_32].rows() / 2 * groups) {
    // 32 groups of W [2048, 2048], 32x128 against 128x128 tiles: 48.7 / 54 us for 8 rows a group on
    // average, 49.5 / 54 for 16, 58 / 54 for 32 (groups of more than 32 rows read W twice)
    p.kind = TILE_32;
    p.tiles_i = ceil_div(I, kShape[TILE_32].rows()) + groups + 1;
    p.tiles_j = ceil_div(J, kShape[TILE_32].cols());
    return p;
  }
  // groups: each ends inside a tile, half a tile more on average; at most one tile more for each of
  // the groups + 2 segments but one
  const bool cut = grouped && mode != WGRAD;
  const int64_t extra = cut ? groups + 1 : 0, outer = mode == WGRAD ? groups : 1;
  const int64_t steps = ceil_div(mode == WGRAD && grouped ? ceil_div(K, groups) : K, BK);
  double best = 0.0;
  for (int kind = TILE_256; kind <= TILE_128; kind++) {
    const int64_t ti = ceil_div(I, kShape[kind].rows()), tj = ceil_div(J, kShape[kind].cols());
    const int64_t tiles = (ti + (cut ? groups / 2 : 0)) * tj * outer;
    int64_t splits = 1;
    if (!grouped && kind != TILE_256) {
      const int64_t most = K / kLeastPart, want = kUnits / tiles;
      splits = want < most ? want : most;
      if (splits < 1) splits = 1;
    }
    const double round = kTileUs[kind] + kStepUs[kind] * ceil_div(steps, splits);
    double us = round * ceil_div(tiles * splits, kUnits);
    if (splits > 1) us += kJoinUs + 8e-6 / kJoinTBps * splits * I * J;
    if (best == 0.0 || us < best) {
      best = us;
      p.kind = kind;
      p.tiles_i = ti + extra;
      p.tiles_j = tj;
      p.splits = splits;
    }
  }
  return p;
}

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

// Parts each group's rows are cut into for the column sums: enough workgroups to fill the chip,
// with 64 rows or more of an average group each.
int64_t grad_parts(int64_t M, int64_t N, int64_t groups) {
  if (N == 0) return 1;
  const int64_t tiles = (N + 255) / 256 * groups, want = (1024 + tiles - 1) / tiles;
  const int64_t most = (M / groups + 63) / 64;
  const int64_t p = want < most ? want : most;
  return p < 1 ? 1 : p;
}

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

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
  if (st == hipSuccess && a.dx != nullptr) {
    const ProductArgs p{a.M, a.K, a.N, a.groups, a.offsets, dp, ld_dp, a.w, a.K, a.N * a.K, a.dx, a.ld_dx, 0,
                        nullptr, nullptr, 0, nullptr, split};
    st = launch_product<DGRAD, LIN_NONE>(p, s);
  }
  if (st == hipSuccess && a.dw != nullptr) {
    const ProductArgs p{a.N, a.K, a.M, a.groups, a.offsets, dp, ld_dp, a.x, a.ld_x, 0, a.dw, a.K, a.N * a.K,
                        nullptr, nullptr, 0, nullptr, split};
    st = launch_product<WGRAD, LIN_NONE>(p, s);
  }
  return st;
}

}  // namespace glu
