// Quantizers to E4M3 with one FP32 scale for each block of 128: 128 consecutive elements of a row
// (rowwise) or of a column (colwise, codes transposed), or 128 x 128 elements (weights), of a BF16
// matrix or of the GLU of one.
//
//   a = max(largest magnitude of the block, 2^-100);  s = a / 448;  code = E4M3(x 448 / a), the code
//   nearest to the real quotient, ties to even.  A block holding NaN or infinity has s NaN and codes NaN.
//
// 448 / a is one IEEE division a block, and the codes need none: y = x fl(448 / a) is within 2^-23 of
// the quotient, which is either a tie of E4M3 or 1 / (31 * 255) or more from every tie (the quotient
// of two 8-bit numbers times 448 = 7 * 2^6 against a 5-bit number).  Rounding y to 15 bits (2^-15)
// therefore restores the ties and moves no other value onto or across one.
//
// Bound by memory: one pass, reading 2 bytes (GLU: 4) and writing 1 for each direction.  Rowwise
// alone a row's 128 elements are 16 lanes, whose maximum takes four exchanges in registers.  With
// columns a workgroup has a tile of 128 x 128 in registers, 8 x 8 elements a thread: the maxima meet in
// LDS, then the codes go through LDS, transposed, into rows of whole 128-byte lines.
#include "ffn_device.h"
#include "fp8_launch.h"
#include "mx_block.h"

namespace glu {
namespace {

constexpr int PLAIN = -1;   // source: the matrix itself; else an activation code
constexpr float LEAST = 0x1p-100f;

// Eight BF16 values from column j of a row as packed pairs.
template <int SRC, int LAYOUT>
__device__ __forceinline__ u32x4 source8(const uint16_t* gate, const uint16_t* up, int64_t j) {
  if constexpr (SRC == PLAIN) {
    return *reinterpret_cast<const u32x4*>(gate + j);
  } else {
    u32x4 A, B;
    float g[8], u[8], h[8];
    if constexpr (LAYOUT == SPLIT) {
      A = *reinterpret_cast<const u32x4*>(gate + j);
      B = *reinterpret_cast<const u32x4*>(up + j);
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4*>(gate + 2 * j), b = *reinterpret_cast<const u32x4*>(gate + 2 * j + 8);
      A = (u32x4){pair_lo(a[0], a[1]), pair_lo(a[2], a[3]), pair_lo(b[0], b[1]), pair_lo(b[2], b[3])};
      B = (u32x4){pair_hi(a[0], a[1]), pair_hi(a[2], a[3]), pair_hi(b[0], b[1]), pair_hi(b[2], b[3])};
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      g[2 * i] = bf_lo(A[i]);
      g[2 * i + 1] = bf_hi(A[i]);
      u[2 * i] = bf_lo(B[i]);
      u[2 * i + 1] = bf_hi(B[i]);
    }
    glu_of<SRC == PLAIN ? 0 : SRC>(h, g, u);
    return (u32x4){pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7])};
  }
}

// The scale of a block whose largest magnitude has this BF16 bit pattern, and what x is multiplied by.
struct Fp8Scale {
  float s, r;
  bool finite;
};
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
  const float a = __builtin_fmaxf(__uint_as_float(top << 16), LEAST);
  if (top >= 0x7f80u) return {__uint_as_float(0x7fc00000u), 0.0f, false};
  return {a / 448.0f, 448.0f / a, true};
}
// x r rounded to 15 bits.
__device__ __forceinline__ float quotient(float x, float r) {
  return __uint_as_float((__float_as_uint(x * r) + 0x100u) & ~0x1ffu);
}
// Codes of four values.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Fp8Scale& f) {
  const uint32_t v = fp8x2<true>(fp8x2<false>(0u, quotient(a, f.r), quotient(b, f.r)), quotient(c, f.r), quotient(d, f.r));
  return f.finite ? v : 0x7f7f7f7fu;
}
__device__ __forceinline__ u32x2 codes8(u32x4 p, const Fp8Scale& f) {
  return (u32x2){codes4(bf_lo(p[0]), bf_hi(p[0]), bf_lo(p[1]), bf_hi(p[1]), f),
                 codes4(bf_lo(p[2]), bf_hi(p[2]), bf_lo(p[3]), bf_hi(p[3]), f)};
}
// The largest 16-bit pattern over 16 lanes, in each of them (both halves of a word at once).
__device__ __forceinline__ uint32_t row_top(uint32_t m) {
  m = pkmax(m, dpp<0x128>(m));   // rotations by 8, 4, 2 and 1 lanes
  m = pkmax(m, dpp<0x124>(m));
  m = pkmax(m, dpp<0x122>(m));
  return pkmax(m, dpp<0x121>(m));
}

// Rowwise alone.  Of the GLU of [8192, 2048] 16 us (84 MB, 5.2 TB/s), of [968, 16384] paired with tanh-GELU 16
// (79 MB, 4.9 TB/s).  grid: (256 columns, row blocks)
template <int SRC, int LAYOUT>
__global__ __launch_bounds__(256) void k_fp8_row(Fp8QuantArgs a) {
  const int64_t col = 256 * (int64_t)blockIdx.x + 8 * (threadIdx.x & 31), ld_q = (a.N + 15) / 16 * 16;
  for (int64_t row = 8 * (int64_t)blockIdx.y + (threadIdx.x >> 5); row < a.M; row += 8 * (int64_t)gridDim.y) {
    u32x4 p = (u32x4)0u;
    if (col < a.N) p = source8<SRC, LAYOUT>(a.gate + row * a.ld_in, a.up + (LAYOUT == SPLIT ? row * a.ld_in : 0), col);
    const uint32_t w[4] = {p[0], p[1], p[2], p[3]};
    const Fp8Scale f = fp8_scale(row_top(top_of(w)));
    if (col < ld_q) *reinterpret_cast<u32x2*>(a.q_row + row * ld_q + col) = col < a.N ? codes8(p, f) : (u32x2)0u;
    if ((threadIdx.x & 15) == 0 && col < a.N) a.s_row[col / 128 * a.M + row] = f.s;
  }
}

// A tile of 128 x 128: thread (lr, lc) has rows 8 lr .. + 7 and columns 8 lc .. + 7.
//   ROW  codes of each row under the row's scale;  COL  of each column, transposed
//   BLOCK  one scale for the tile, codes as they are and, with COL, transposed
// Rows and columns of [16384, 7168] 108 to 117 us (477 MB, 4.1 to 4.4 TB/s: the tile is loaded, turned and stored one after
// the other, and other workgroups fill the gaps), of [16384, 2048] 35 to 38, weights [7168, 2048] both ways 16 to 17;
// of the GLU of [16384, 7168] 168 to 170 (712 MB, 4.2 TB/s).
struct TileArgs {
  int64_t M, N, ld_in;
  const uint16_t* gate;
  const uint16_t* up;
  uint8_t* q_row;
  float* s_row;
  uint8_t* q_col;
  float* s_col;
  int64_t in_group, row_group, col_group, s_group;   // BLOCK: elements from one matrix to the next
};
// grid: (tiles along N, tiles along M, matrices)
template <int SRC, int LAYOUT, bool ROW, bool COL, bool BLOCK>
__global__ __launch_bounds__(256) void k_fp8_tile(TileArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
  __shared__ __attribute__((aligned(16))) uint32_t tops[4][64];   // column maxima of each wave, two to a word
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, lc = threadIdx.x & 15u, lr = threadIdx.x >> 4;
  const int64_t ld_q = (a.N + 15) / 16 * 16, ld_t = (a.M + 15) / 16 * 16;
  const int64_t n0 = 128 * (int64_t)blockIdx.x, col = n0 + 8 * lc, NB = (a.N + 127) / 128, MB = (a.M + 127) / 128;
  const uint16_t* gate = a.gate + blockIdx.z * a.in_group;
  for (int64_t tm = blockIdx.y; tm < MB; tm += gridDim.y) {
    const int64_t m0 = 128 * tm;
    u32x4 p[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int64_t row = m0 + 8 * lr + i;
      p[i] = (u32x4)0u;
      if (row < a.M && col < a.N)
        p[i] = source8<SRC, LAYOUT>(gate + row * a.ld_in, a.up + (SRC != PLAIN && LAYOUT == SPLIT ? row * a.ld_in : 0), col);
    }
    u32x4 top = (u32x4)0u;   // of the thread's columns
    if constexpr (COL || BLOCK) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
#pragma unroll
        for (int i = 0; i < 8; i++) top[j] = pkmax(top[j], p[i][j] & 0x7fff7fffu);
        top[j] = pkmax(top[j], swz_xor16(top[j]));
        top[j] = pkmax(top[j], (uint32_t)__builtin_amdgcn_ds_bpermute((int)(4u * (lane ^ 32u)), (int)top[j]));
      }
      if (lane < 16) *reinterpret_cast<u32x4*>(&tops[wave][4 * lc]) = top;
      __syncthreads();
      top = (u32x4)0u;
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const u32x4 t = *reinterpret_cast<const u32x4*>(&tops[w][4 * lc]);
#pragma unroll
        for (int j = 0; j < 4; j++) top[j] = pkmax(top[j], t[j]);
      }
    }
    Fp8Scale whole;
    if constexpr (BLOCK) {
      uint32_t m = row_top(pkmax(pkmax(top[0], top[1]), pkmax(top[2], top[3])));
      whole = fp8_scale(umax(lo16(m), hi16(m)));
      if (threadIdx.x == 0) {
        a.s_row[blockIdx.z * a.s_group + tm * NB + blockIdx.x] = whole.s;
        if (COL) a.s_col[blockIdx.z * a.s_group + blockIdx.x * MB + tm] = whole.s;
      }
    }
    if constexpr (ROW || BLOCK) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int64_t row = m0 + 8 * lr + i;
        const uint32_t w[4] = {p[i][0], p[i][1], p[i][2], p[i][3]};
        Fp8Scale f;
        if constexpr (BLOCK) f = whole;
        else f = fp8_scale(row_top(top_of(w)));
        if (row < a.M) {
          uint8_t* q = a.q_row + blockIdx.z * a.row_group + row * ld_q + col;
          if (col < ld_q) *reinterpret_cast<u32x2*>(q) = col < a.N ? codes8(p[i], f) : (u32x2)0u;
          if (ROW && lc == 0) a.s_row[blockIdx.x * a.M + row] = f.s;
        }
      }
    }
    if constexpr (COL) {
      // the thread's 8 codes of a column, rows 8 lr .. + 7, are piece lr of line 8 lc + j, kept at place
      // lr ^ lc of the line so that the lanes of a wave spread over the banks
#pragma unroll
      for (int j = 0; j < 8; j++) {
        Fp8Scale f;
        if constexpr (BLOCK) f = whole;
        else f = fp8_scale(j % 2 ? hi16(top[j / 2]) : lo16(top[j / 2]));
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = j % 2 ? bf_hi(p[i][j / 2]) : bf_lo(p[i][j / 2]);
        u32x2 c = {codes4(v[0], v[1], v[2], v[3], f), codes4(v[4], v[5], v[6], v[7], f)};
        if (!f.finite) {   // rows past the last are padding, zero
          const int64_t left = a.M - m0 - 8 * lr;
#pragma unroll
          for (int i = 0; i < 8; i++)
            if (i >= left) c[i / 4] &= ~(0xffu << (8 * (i % 4)));
        }
        *reinterpret_cast<u32x2*>(turned + 128u * (8u * lc + j) + 8u * (lr ^ lc)) = c;
        if (!BLOCK && lr == 0 && col + j < a.N) a.s_col[tm * a.N + col + j] = f.s;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; k++) {   // 128 lines of 8 pieces of 16 codes
        const uint32_t t = threadIdx.x + 256u * k, line = t >> 3, c = t & 7u, x = line >> 3;
        const u32x4 v = *reinterpret_cast<const u32x4*>(turned + 128u * line + 16u * (c ^ (x >> 1)));
        const int64_t m = m0 + 16 * c;
        if (n0 + line < a.N && m < ld_t)
          *reinterpret_cast<u32x4*>(a.q_col + blockIdx.z * a.col_group + (n0 + line) * ld_t + m) =
              x & 1u ? (u32x4){v[2], v[3], v[0], v[1]} : v;
      }
    }
    __syncthreads();
  }
}

dim3 tile_grid(int64_t M, int64_t N, int64_t matrices) {
  const int64_t m = fp8_blocks(M);
  return dim3((unsigned)fp8_blocks(N), (unsigned)(m < 65535 ? m : 65535), (unsigned)matrices);
}

template <int SRC, int LAYOUT>
hipError_t launch_quant(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.q_col == nullptr)
    return launch_kernel(k_fp8_row<SRC, LAYOUT>, grid_2d((a.N + 255) / 256, (a.M + 7) / 8), dim3(256), s, a);
  const TileArgs t{a.M, a.N, a.ld_in, a.gate, a.up, a.q_row, a.s_row, a.q_col, a.s_col, 0, 0, 0, 0};
  const dim3 grid = tile_grid(a.M, a.N, 1);
  return a.q_row != nullptr ? launch_kernel(k_fp8_tile<SRC, LAYOUT, true, true, false>, grid, dim3(256), s, t)
                            : launch_kernel(k_fp8_tile<SRC, LAYOUT, false, true, false>, grid, dim3(256), s, t);
}

}  // namespace

hipError_t launch_fp8_quant(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.act < 0) return launch_quant<PLAIN, SPLIT>(a, s);
  return with_act(a.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    return a.layout == SPLIT ? launch_quant<ACT, SPLIT>(a, s) : launch_quant<ACT, PAIRED>(a, s);
  });
}

hipError_t launch_fp8_weight(const Fp8WeightArgs& a, hipStream_t s) {
  const TileArgs t{a.N, a.K, a.K, a.w, nullptr, a.q, a.s, a.qt, a.st,
                   a.N * a.K, a.N * fp8_padded(a.K), a.K * fp8_padded(a.N), fp8_blocks(a.N) * fp8_blocks(a.K)};
  const dim3 grid = tile_grid(a.N, a.K, a.groups);
  return a.qt != nullptr ? launch_kernel(k_fp8_tile<PLAIN, SPLIT, false, true, true>, grid, dim3(256), s, t)
                         : launch_kernel(k_fp8_tile<PLAIN, SPLIT, false, false, true>, grid, dim3(256), s, t);
}

}  // namespace glu
