// Checkpoints of the GLU's operands in 8 bits, and the GLU's gradient from what was kept.
//
//   forward   h = act(g) u;  q, s = MXFP8 of g and of u: E4M3 codes with one E8M0 scale per 32
//             consecutive elements of a row, rounded up (RCEIL) from the block's largest magnitude
//   backward  g~, u~ = code 2^e;  da = dh u~ act'(g~), db = dh act(g~), and h~ = act(g~) u~ again
//
// 2.06 bytes kept for each (gate, up) where BF16 takes 4, and h need not be kept.  E4M3 has 4
// significant bits, so g~ and u~ are within 2^-4 of g and u (relative, above the subnormals);
// code 2^e is exact in FP32.  A block holding NaN or infinity is kept as NaN.
//
// Element-wise and bound by memory.  A thread has 8 columns of a row; a block of 32 is the four
// lanes of a quad, so its maximum takes two exchanges in registers.  A row's chunks are counted in
// whole quads (the rest of the last quad holds zeros), so no quad holds two rows.
#include "ffn_device.h"
#include "gated_launch.h"
#include "mx_block.h"

namespace glu {
namespace {

constexpr int ROWS = 8, CHUNKS = 32;   // rows and 8-column chunks a workgroup holds at a time

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(float (&v)[8], u32x4 p) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = bf_lo(p[i]);
    v[2 * i + 1] = bf_hi(p[i]);
  }
}

// Measured at [16384, 7168] with h: 162 to 178 us (969 MB, 5.4 to 6.0 TB/s); [1021, 1000] 5.0, [128, 128] 2.8 to 3.2.
// grid: (256 columns, row blocks)
template <int ACT, int LAYOUT>
__global__ __launch_bounds__(256) void k_ckpt_fwd(CkptArgs a) {
  const int lc = threadIdx.x & 31, lr = threadIdx.x >> 5;
  const int64_t col = 8 * (CHUNKS * (int64_t)blockIdx.x + lc), NB = (a.N + 31) / 32;
  const bool in = col < a.N;
  for (int64_t row = ROWS * (int64_t)blockIdx.y + lr; row < a.M; row += ROWS * (int64_t)gridDim.y) {
    u32x4 G = (u32x4)0u, U = (u32x4)0u;   // eight gates, eight ups
    if (in) {
      if constexpr (LAYOUT == SPLIT) {
        G = *reinterpret_cast<const u32x4*>(a.gate + row * a.ld_in + col);
        U = *reinterpret_cast<const u32x4*>(a.up + row * a.ld_in + col);
      } else {
        const u32x4 A = *reinterpret_cast<const u32x4*>(a.gate + row * a.ld_in + 2 * col);
        const u32x4 B = *reinterpret_cast<const u32x4*>(a.gate + row * a.ld_in + 2 * col + 8);
        G = (u32x4){pair_lo(A[0], A[1]), pair_lo(A[2], A[3]), pair_lo(B[0], B[1]), pair_lo(B[2], B[3])};
        U = (u32x4){pair_hi(A[0], A[1]), pair_hi(A[2], A[3]), pair_hi(B[0], B[1]), pair_hi(B[2], B[3])};
      }
    }
    if (a.h != nullptr && in) {
      float g[8], u[8], h[8];
      unpack8(g, G);
      unpack8(u, U);
      glu_of<ACT>(h, g, u);
      *reinterpret_cast<u32x4*>(a.h + row * a.ld_h + col) = pack8(h);
    }
    const uint32_t gp[4] = {G[0], G[1], G[2], G[3]}, up[4] = {U[0], U[1], U[2], U[3]};
    uint32_t m = top_of(gp) | top_of(up) << 16;
    m = pkmax(m, dpp<DPP_XOR1>(m));
    m = pkmax(m, dpp<DPP_XOR2>(m));
    const uint32_t sg = block_scale(lo16(m)), su = block_scale(hi16(m));
    if (in) {
      uint8_t* q = a.q + row * 2 * a.N + col;
      *reinterpret_cast<u32x2*>(q) = (u32x2){block_codes(G[0], G[1], sg), block_codes(G[2], G[3], sg)};
      *reinterpret_cast<u32x2*>(q + a.N) = (u32x2){block_codes(U[0], U[1], su), block_codes(U[2], U[3], su)};
      if ((lc & 3) == 0) {
        uint8_t* s = a.s + row * 2 * NB + col / 32;
        s[0] = (uint8_t)sg;
        s[NB] = (uint8_t)su;
      }
    }
  }
}

// Eight values from codes and their scale byte.
__device__ __forceinline__ void restore8(float (&v)[8], u32x2 q, uint32_t scale) {
  const float s = e8m0_value(scale);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
    v[4 * i] = lo[0] * s;
    v[4 * i + 1] = lo[1] * s;
    v[4 * i + 2] = hi[0] * s;
    v[4 * i + 3] = hi[1] * s;
  }
}

// Eight values from BF16 and four more bits of each.
__device__ __forceinline__ void widen8(float (&v)[8], u32x4 p, uint32_t rest) {
  v[0] = wide_value<0>(p[0] << 16, rest);
  v[1] = wide_value<1>(p[0] & 0xffff0000u, rest);
  v[2] = wide_value<2>(p[1] << 16, rest);
  v[3] = wide_value<3>(p[1] & 0xffff0000u, rest);
  v[4] = wide_value<4>(p[2] << 16, rest);
  v[5] = wide_value<5>(p[2] & 0xffff0000u, rest);
  v[6] = wide_value<6>(p[3] << 16, rest);
  v[7] = wide_value<7>(p[3] & 0xffff0000u, rest);
}

// Measured at [16384, 7168]: from codes with h 217 to 224 us (1234 MB, 5.5 TB/s), from BF16 and four more bits
// without h 250 to 254 (1292 MB, 5.1 TB/s); [1021, 1000] 6.6, with sums 7.6.
// grid: (256 columns, group, part of the group's rows); with sums and h, group number `groups` is the
// rows of no group, whose h is formed too.
template <int ACT, bool MX, int LAYOUT>
__global__ __launch_bounds__(256) void k_glu_grad(GluGradArgs a) {
  __shared__ float part[ROWS][CHUNKS][17];
  const int lc = threadIdx.x & 31, lr = threadIdx.x >> 5;
  const int64_t col = 8 * (CHUNKS * (int64_t)blockIdx.x + lc), NB = (a.N + 31) / 32;
  const int64_t e = blockIdx.y;
  int64_t r0 = 0, r1 = a.M, skip0 = a.M, skip1 = a.M;   // rows r0 .. r1 - 1 but for skip0 .. skip1 - 1
  if (a.offsets != nullptr) {
    const int64_t b = min((int64_t)max(a.offsets[e < a.groups ? e : 0], 0), a.M);
    const int64_t c = max(b, min((int64_t)a.offsets[e < a.groups ? e + 1 : a.groups], a.M));
    if (e < a.groups) {
      r0 = b;
      r1 = c;
    } else {
      skip0 = b;
      skip1 = c;
    }
  }
  const int64_t n = r1 - r0;
  r1 = r0 + n * (blockIdx.z + 1) / gridDim.z;
  r0 = r0 + n * blockIdx.z / gridDim.z;
  float sg[8] = {}, su[8] = {};
  if (col < a.N) {
    for (int64_t row = r0 + lr; row < r1; row += ROWS) {
      if (row >= skip0 && row < skip1) continue;
      float g[8], u[8], d[8], da[8], db[8];
      if constexpr (MX) {
        const uint8_t* q = a.q + row * 2 * a.N + col;
        const uint8_t* s = a.s + row * 2 * NB + col / 32;
        restore8(g, *reinterpret_cast<const u32x2*>(q), s[0]);
        restore8(u, *reinterpret_cast<const u32x2*>(q + a.N), s[NB]);
      } else {
        const uint16_t* p = a.pre + row * 2 * a.N + col;
        const uint8_t* s = a.s + row * a.N + col / 2;
        uint32_t rg = 0, ru = 0;
        if (a.s != nullptr) {
          rg = *reinterpret_cast<const uint32_t*>(s);
          ru = *reinterpret_cast<const uint32_t*>(s + a.N / 2);
        }
        widen8(g, *reinterpret_cast<const u32x4*>(p), rg);
        widen8(u, *reinterpret_cast<const u32x4*>(p + a.N), ru);
      }
      if (a.d != nullptr || a.sums != nullptr) {
        unpack8(d, *reinterpret_cast<const u32x4*>(a.dh + row * a.ld_dh + col));
        bool tail = false;
#pragma unroll
        for (int i = 0; i < 8; i++) glu_bwd_elem<ACT>(g[i], u[i], d[i], da[i], db[i], tail);
        if (tail) {
#pragma unroll
          for (int i = 0; i < 8; i++)
            if (bwd_tail_needed<ACT>(g[i], u[i], d[i])) glu_bwd_tail<ACT>(g[i], u[i], d[i], da[i], db[i]);
        }
        if (a.d != nullptr) {
          if constexpr (LAYOUT == SPLIT) {
            *reinterpret_cast<u32x4*>(a.d + row * a.ld_d + col) = pack8(da);
            *reinterpret_cast<u32x4*>(a.d + row * a.ld_d + a.N + col) = pack8(db);
          } else {
            uint16_t* o = a.d + row * a.ld_d + 2 * col;
#pragma unroll
            for (int i = 0; i < 2; i++)
              *reinterpret_cast<u32x4*>(o + 8 * i) =
                  (u32x4){pack_bf16(da[4 * i], db[4 * i]), pack_bf16(da[4 * i + 1], db[4 * i + 1]),
                          pack_bf16(da[4 * i + 2], db[4 * i + 2]), pack_bf16(da[4 * i + 3], db[4 * i + 3])};
          }
        }
        if (e < a.groups) {
#pragma unroll
          for (int i = 0; i < 8; i++) {
            sg[i] += da[i];
            su[i] += db[i];
          }
        }
      }
      if (a.h != nullptr) {
        float h[8];
        glu_of<ACT>(h, g, u);
        *reinterpret_cast<u32x4*>(a.h + row * a.ld_h + col) = pack8(h);
      }
    }
  }
  if (a.sums == nullptr || e == a.groups) return;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    part[lr][lc][LAYOUT == SPLIT ? i : 2 * i] = sg[i];
    part[lr][lc][LAYOUT == SPLIT ? 8 + i : 2 * i + 1] = su[i];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < 2; v++) {   // 512 sums: 16 of each chunk
    const int k = threadIdx.x + 256 * v, c = k / 16, i = k % 16;
    const int64_t first = 8 * (CHUNKS * (int64_t)blockIdx.x + c);
    if (first >= a.N) continue;
    float t = 0.0f;
    for (int w = 0; w < ROWS; w++) t += part[w][c][i];
    const int64_t at = LAYOUT == SPLIT ? (i < 8 ? first + i : a.N + first + i - 8) : 2 * first + i;
    a.sums[((int64_t)blockIdx.z * a.groups + e) * 2 * a.N + at] = t;
  }
}

}  // namespace

hipError_t launch_ckpt_fwd(const CkptArgs& a, hipStream_t s) {
  const dim3 grid = grid_2d((a.N + 255) / 256, (a.M + ROWS - 1) / ROWS);
  return with_act(a.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    return a.layout == SPLIT ? launch_kernel(k_ckpt_fwd<ACT, SPLIT>, grid, dim3(256), s, a)
                             : launch_kernel(k_ckpt_fwd<ACT, PAIRED>, grid, dim3(256), s, a);
  });
}

hipError_t launch_glu_grad(GluGradArgs a, hipStream_t s) {
  const bool rest = a.offsets != nullptr && a.h != nullptr;
  if (a.sums == nullptr) {
    // four rows a thread once that fills the chip, else as few as do ([1021, 1000]: 11.4 -> 6.6 us)
    const int64_t tiles = (a.N + 255) / 256 * a.groups, four = (a.M + 4 * ROWS - 1) / (4 * ROWS), one = (a.M + ROWS - 1) / ROWS;
    const int64_t want = (1024 + tiles - 1) / tiles, parts = four > want ? four : one < want ? one : want;
    a.parts = parts < 65535 ? parts : 65535;
  }
  const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)(a.groups + rest), (unsigned)a.parts);
  return with_act(a.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    if (a.pre != nullptr)
      return a.layout == SPLIT ? launch_kernel(k_glu_grad<ACT, false, SPLIT>, grid, dim3(256), s, a)
                               : launch_kernel(k_glu_grad<ACT, false, PAIRED>, grid, dim3(256), s, a);
    return a.layout == SPLIT ? launch_kernel(k_glu_grad<ACT, true, SPLIT>, grid, dim3(256), s, a)
                             : launch_kernel(k_glu_grad<ACT, true, PAIRED>, grid, dim3(256), s, a);
  });
}

}  // namespace glu
