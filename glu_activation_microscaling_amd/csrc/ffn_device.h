// Device helpers of the operators around the GLU: rows in 16-byte vectors at any alignment,
// and sums over a wave or a workgroup.
#pragma once

#include "glu_device.h"

namespace glu {

// A value that is the same in every lane, moved to a scalar register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

struct __attribute__((packed, aligned(2))) Vec16 {
  u32x4 v;
};

// Eight elements as loaded: BF16 in one 16-byte vector, FP32 in two.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 a;
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = bf_lo(a[i]);
      f[2 * i + 1] = bf_hi(a[i]);
    }
  }
};
template <>
struct Raw<float> {
  u32x4 a, b;
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[i] = __uint_as_float(a[i]);
      f[4 + i] = __uint_as_float(b[i]);
    }
  }
};

// A lane offset that the compiler forgets the origin of: the address stays a scalar base plus
// this offset, instead of a 64-bit lane pointer per operand kept across a loop over rows.
__device__ __forceinline__ uint32_t lane_offset(uint32_t o) {
  asm volatile("" : "+v"(o));
  return o;
}

// Loads elements o .. o + n - 1 of p (n <= 0: none, n >= 8: all eight); the others read zero.  With a
// wave-uniform p the address is a scalar base and a 32-bit lane offset.
template <bool RAGGED>
__device__ __forceinline__ void load(Raw<uint16_t>& r, const uint16_t* base, uint32_t o, int n) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + lane_offset(2u * o));
  r.a = (u32x4)0u;
  if (n >= 8) {
    r.a = RAGGED ? reinterpret_cast<const Vec16*>(p)->v : *reinterpret_cast<const u32x4*>(p);
  } else if (RAGGED) {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) r.a[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
  }
}
template <bool RAGGED>
__device__ __forceinline__ void load(Raw<float>& r, const float* base, uint32_t o, int n) {
  const float* p = reinterpret_cast<const float*>(reinterpret_cast<const char*>(base) + lane_offset(4u * o));
  r.a = (u32x4)0u;
  r.b = (u32x4)0u;
  if (n >= 8) {
    if (RAGGED) {
      r.a = reinterpret_cast<const Vec16*>(p)[0].v;
      r.b = reinterpret_cast<const Vec16*>(p)[1].v;
    } else {
      r.a = reinterpret_cast<const u32x4*>(p)[0];
      r.b = reinterpret_cast<const u32x4*>(p)[1];
    }
  } else if (RAGGED) {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) {
        if (i < 4) r.a[i & 3] = __float_as_uint(p[i]);
        else r.b[i & 3] = __float_as_uint(p[i]);
      }
  }
}

template <bool RAGGED>
__device__ __forceinline__ void store(uint16_t* base, uint32_t o, const float (&f)[8], int n) {
  uint16_t* p = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(base) + lane_offset(2u * o));
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  if (n >= 8) {
    if (RAGGED) reinterpret_cast<Vec16*>(p)->v = v;
    else *reinterpret_cast<u32x4*>(p) = v;
  } else if (RAGGED) {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}
template <bool RAGGED>
__device__ __forceinline__ void store(float* base, uint32_t o, const float (&f)[8], int n) {
  float* p = reinterpret_cast<float*>(reinterpret_cast<char*>(base) + lane_offset(4u * o));
  const u32x4 a = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  const u32x4 b = {__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
  if (n >= 8) {
    if (RAGGED) {
      reinterpret_cast<Vec16*>(p)[0].v = a;
      reinterpret_cast<Vec16*>(p)[1].v = b;
    } else {
      reinterpret_cast<u32x4*>(p)[0] = a;
      reinterpret_cast<u32x4*>(p)[1] = b;
    }
  } else if (RAGGED) {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < n) p[i] = f[i];
  }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}
// Sum over the wave's 64 lanes, in every lane: partial sums run up each row of 16 lanes, then
// across the rows, to lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);   // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);   // row_bcast 15, 31
  v = dpp_add<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over 16 lanes, in each of them: rotations by 8, 4, 2 and 1 lanes.
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp<0x128>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x124>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x122>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x121>(__float_as_uint(v)));
  return v;
}

// Sums of N values over the workgroup (up to 16 waves), in every thread.  The two halves of `part`
// are used in turn, so one barrier a call suffices: a half is written again only after the
// barrier of the call in between.  Call clear_parts once before the first sum.
template <int N>
struct BlockParts {
  float v[2][16][N];
};
template <int N>
__device__ __forceinline__ void clear_parts(BlockParts<N>& part) {
  for (unsigned i = threadIdx.x; i < 2 * 16 * N; i += blockDim.x) (&part.v[0][0][0])[i] = 0.0f;
  __syncthreads();
}
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], BlockParts<N>& part, int& turn) {
#pragma unroll
  for (int k = 0; k < N; k++) v[k] = wave_sum(v[k]);
  if (blockDim.x == 64) return;
  if ((threadIdx.x & 63u) == 0) {
#pragma unroll
    for (int k = 0; k < N; k++) part.v[turn][threadIdx.x >> 6][k] = v[k];
  }
  __syncthreads();
  // absent waves hold zero; 16 lanes read a wave's sum each and add up in a ring, so every lane
  // ends with all of it after one read
#pragma unroll
  for (int k = 0; k < N; k++) v[k] = row_sum(part.v[turn][threadIdx.x & 15u][k]);
  turn ^= 1;
}

}  // namespace glu
