// The norms on both sides of a block, fused with its gate and its residual scale, forward and
// backward:
//
//   x' = rho x + g * z,  z = N(y) w_post  (or z = y);   h = N(x') w_pre + b_pre
//   N(v) = v / sqrt(mean(v^2) + eps)  (rms)  or  (v - mean v) / sqrt(var(v) + eps)  (layer)
//
// g, w_pre and b_pre hold one row for all rows of x or one per group of consecutive rows.
// All arithmetic is FP32 on the widened inputs; x' enters the second norm unrounded, and each
// output is rounded once at its store.  Variances are two-pass sums over the row, which stays
// in registers, so a large mean costs no digits.
//
// Backward, with n = N(v), r = 1/sqrt(...): v's gradient is r (dn - n mean(dn n) [- mean(dn)]).
//   dn' = dh w_pre;  D = dx' + N_grad(dn');  dx = rho D;  dg = sum D z;  dw_pre = sum dh n'
//   db_pre = sum dh;  dz = g D;  dw_post = sum dz n;  dy = N_grad(dz w_post)
// x' and n' are formed again from x and y (the same bytes as reading x' would take), so the
// gradients are those of the unrounded x'.
//
// Both passes are bound by memory: they read and write each operand once.  A workgroup holds
// one row, 8 columns (one 16-byte vector of BF16) a thread; rows whose width or stride is no
// multiple of 8 use the same vectors unaligned, with the last chunk taken by elements.
//
// Measured on an MI355X, where a copy of 1 GiB reaches 5.1 TB/s (rms norms on both sides, BF16):
//   forward   [16384, 7168] 183 us (5.1 TB/s), [968, 2048] 5.8 us, [1, 2048] 3.2 us
//   backward  [16384, 7168] 293 us (4.8 TB/s), and 6 us to join the column sums
// and with layer norms, an FP32 stream and rows that are no whole number of vectors, [1021, 8193]:
// forward 35 us, backward 61 us, join 9 us (2.9 and 2.5 TB/s).  There the four waits of a row's
// workgroup for its sums count: 256 workgroups of 9 waves have 4 rows each, and registers leave
// room for one workgroup a compute unit (two, at 96 registers, spill: 20 us slower).
#include "ffn_device.h"
#include "ffn_launch.h"

namespace glu {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// Loads and stores of a row's chunk.  Rows of whole vectors go through buffer instructions: a scalar
// base and one 32-bit lane offset, which for lanes past the row is out of range (such loads
// give zeros, such stores do nothing), so there is no branch and no address to keep per operand.
template <bool RAGGED>
__device__ __forceinline__ void get(Raw<uint16_t>& r, const uint16_t* base, uint32_t o, int n) {
  if constexpr (RAGGED) load<true>(r, base, o, n);
  else r.a = __builtin_amdgcn_raw_buffer_load_b128(rsrc(base), n > 0 ? 2u * o : kOob, 0, 0);
}
template <bool RAGGED>
__device__ __forceinline__ void get(Raw<float>& r, const float* base, uint32_t o, int n) {
  if constexpr (RAGGED) {
    load<true>(r, base, o, n);
  } else {
    const uint32_t at = n > 0 ? 4u * o : kOob;
    r.a = __builtin_amdgcn_raw_buffer_load_b128(rsrc(base), at, 0, 0);
    r.b = __builtin_amdgcn_raw_buffer_load_b128(rsrc(base), at + 16u, 0, 0);
  }
}
template <bool RAGGED>
__device__ __forceinline__ void put(uint16_t* base, uint32_t o, const float (&f)[8], int n) {
  if constexpr (RAGGED) {
    store<true>(base, o, f, n);
  } else {
    const u32x4 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc(base), n > 0 ? 2u * o : kOob, 0, 0);
  }
}
template <bool RAGGED>
__device__ __forceinline__ void put(float* base, uint32_t o, const float (&f)[8], int n) {
  if constexpr (RAGGED) {
    store<true>(base, o, f, n);
  } else {
    const uint32_t at = n > 0 ? 4u * o : kOob;
    __builtin_amdgcn_raw_buffer_store_b128((u32x4){__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                                   __float_as_uint(f[3])}, rsrc(base), at, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128((u32x4){__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                                   __float_as_uint(f[7])}, rsrc(base), at + 16u, 0, 0);
  }
}

// Eight values of a parameter (BF16 or FP32 by a wave-uniform flag) at element row + o.
template <bool RAGGED>
__device__ __forceinline__ void load_param(float (&f)[8], const void* p, int64_t row, uint32_t o, int n,
                                           bool f32) {
  if (f32) {
    Raw<float> r;
    get<RAGGED>(r, (const float*)p + row, o, n);
    r.get(f);
  } else {
    Raw<uint16_t> r;
    get<RAGGED>(r, (const uint16_t*)p + row, o, n);
    r.get(f);
  }
}

// Whether element i of a chunk with n elements left is in the row (all 8 or none, unless ragged).
template <bool RAGGED>
__device__ __forceinline__ bool inside(int i, int n) {
  return RAGGED ? i < n : n > 0;
}

// Rows of an operand in flight: loaded a row ahead of their use.
template <typename X, int V, bool RAGGED>
__device__ __forceinline__ void load_row(Raw<X> (&r)[V], const X* p, const uint32_t (&col)[V], const int (&n)[V]) {
#pragma unroll
  for (int v = 0; v < V; v++) get<RAGGED>(r[v], p, col[v], n[v]);
}

// A parameter row, or `fill` where there is none.
template <int V, bool RAGGED>
__device__ __forceinline__ void param_row(float (&f)[V][8], const void* p, int64_t at, const uint32_t (&col)[V],
                                          const int (&n)[V], bool f32, float fill) {
#pragma unroll
  for (int v = 0; v < V; v++) {
    if (p != nullptr) {
      load_param<RAGGED>(f[v], p, at, col[v], n[v], f32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) f[v][i] = fill;
    }
  }
}

// Forward.  A workgroup takes consecutive rows; the next row's x and y are loaded while a row is
// worked on, and with 8 columns a thread the parameters stay in registers until the group changes
// (gate w_post as one factor: g z = (g w_post) n); with 16 they are loaded for every row, which
// keeps the registers below 128 (16 waves a compute unit).  The rms form without the mean's work
// took [16384, 7168] from 228 to 183 us.
template <typename X, int V, bool RAGGED, bool MX, bool LAYER>
__global__ __launch_bounds__(1024) void k_block_norm(NormArgs a, uint32_t rows) {
  __shared__ BlockParts<1> part;
  int turn = 0;
  clear_parts(part);
  const int H = (int)a.H;
  const bool pf32 = a.flags & NORM_F32_PARAMS, post = a.flags & NORM_POST;
  const bool pre = a.flags & NORM_PRE, has_y = a.y != nullptr;
  const float invH = 1.0f / (float)H;
  uint32_t col[V];
  int n[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    col[v] = 8u * (threadIdx.x + blockDim.x * v);
    n[v] = H - (int)col[v];
  }
  const uint32_t r0 = blockIdx.x * rows, r1 = min(r0 + rows, (uint32_t)a.M);
  const X* const px = (const X*)a.x;

  // v := v - mean (layer) with the elements outside the row kept zero; returns 1/sqrt(...)
  float mean = 0.0f;
  auto normalize = [&](float (&f)[V][8]) {
    mean = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 8; i++) s[0] += f[v][i];
      block_sum(s, part, turn);
      mean = s[0] * invH;
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 8; i++) f[v][i] = inside<RAGGED>(i, n[v]) ? f[v][i] - mean : 0.0f;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 8; i++) q[0] = __builtin_fmaf(f[v][i], f[v][i], q[0]);
    block_sum(q, part, turn);
    return 1.0f / __builtin_sqrtf(__builtin_fmaf(q[0], invH, a.eps));
  };

  Raw<X> nx[V];
  Raw<uint16_t> ny[V];
  if (r0 < r1) {
    load_row<X, V, RAGGED>(nx, px + (int64_t)r0 * a.ld_x, col, n);
    if (has_y) load_row<uint16_t, V, RAGGED>(ny, a.y + (int64_t)r0 * a.ld_y, col, n);
  }
  constexpr bool HOLD = V == 1;
  float gw[V][8], wq[V][8], wb[V][8];
  uint32_t next = r0, grp = 0;   // first row of the next group; the group
  auto load_gw = [&] {
    param_row<V, RAGGED>(gw, a.gate.p, grp * a.gate.stride, col, n, pf32, 1.0f);
    if (a.w_post.p != nullptr) {
      param_row<V, RAGGED>(wq, a.w_post.p, 0, col, n, pf32, 1.0f);
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 8; i++) gw[v][i] *= wq[v][i];
    }
  };
  auto load_wb = [&] {
    param_row<V, RAGGED>(wq, a.w_pre.p, grp * a.w_pre.stride, col, n, pf32, 1.0f);
    param_row<V, RAGGED>(wb, a.b_pre.p, grp * a.b_pre.stride, col, n, pf32, 0.0f);
  };
  for (uint32_t row = r0; row < r1; row++) {
    if (row == next) {
      const uint32_t per = (uint32_t)a.rows_per_group;
      grp = uniform(row / per);
      next = (grp + 1) * per;
      if (HOLD) {
        load_gw();
        load_wb();
      }
    }
    float xo[V][8], z[V][8];
#pragma unroll
    for (int v = 0; v < V; v++) {
      nx[v].get(xo[v]);
      if (has_y) ny[v].get(z[v]);
    }
    if (row + 1 < r1) {
      load_row<X, V, RAGGED>(nx, px + (int64_t)(row + 1) * a.ld_x, col, n);
      if (has_y) load_row<uint16_t, V, RAGGED>(ny, a.y + (int64_t)(row + 1) * a.ld_y, col, n);
    }
    float st[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (has_y) {
      float r = 1.0f;
      if (!HOLD) load_gw();
      if (post) {
        r = normalize(z);
        st[0] = mean;
        st[1] = r;
      }
#pragma unroll
      for (int v = 0; v < V; v++) {
#pragma unroll
        for (int i = 0; i < 8; i++) xo[v][i] = __builtin_fmaf(gw[v][i], z[v][i] * r, a.res_scale * xo[v][i]);
        put<RAGGED>((X*)a.x_out + (int64_t)row * a.ld_xo, col[v], xo[v], n[v]);
      }
    }
    if (pre) {
      if (!HOLD) load_wb();
      const float r = normalize(xo);
      st[2] = mean;
      st[3] = r;
#pragma unroll
      for (int v = 0; v < V; v++) {
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; i++) h[i] = __builtin_fmaf(xo[v][i], r * wq[v][i], wb[v][i]);
        if constexpr (MX) {
          // an MXFP8 block is the 32 columns of four neighbouring lanes (H is a multiple of
          // 32, so a block is inside the row or outside it); rounded to BF16 first, as every
          // quantizer of the library sees it
          uint32_t p[4], m = 0;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            p[i] = pack_bf16(h[2 * i], h[2 * i + 1]);
            m = pkmax(m, p[i] & 0x7fff7fffu);
          }
          m = umax(lo16(m), hi16(m));
          m = umax(m, dpp<DPP_XOR1>(m));
          m = umax(m, dpp<DPP_XOR2>(m));
          const bool nonfinite = m >= 0x7f80u;
          const uint32_t sb = nonfinite ? 0xffu : mx_scale_byte(m << 16);
          const float sc = e8m0_value(sb);
          uint32_t c0 = fp8x2_scaled<true>(fp8x2_scaled<false>(0u, p[0], sc), p[1], sc);
          uint32_t c1 = fp8x2_scaled<true>(fp8x2_scaled<false>(0u, p[2], sc), p[3], sc);
          if (nonfinite) c0 = c1 = 0x7f7f7f7fu;
          if (n[v] > 0) {
            *reinterpret_cast<u32x2*>(a.q + (int64_t)row * a.H + col[v]) = (u32x2){c0, c1};
            if ((threadIdx.x & 3u) == 0) a.s[(int64_t)row * (a.H / 32) + col[v] / 32] = (uint8_t)sb;
          }
        } else {
          put<RAGGED>(a.h + (int64_t)row * a.ld_h, col[v], h, n[v]);
        }
      }
    }
    if (threadIdx.x == 0)
      *reinterpret_cast<u32x4*>(a.stats + 4 * (int64_t)row) =
          (u32x4){__float_as_uint(st[0]), __float_as_uint(st[1]), __float_as_uint(st[2]), __float_as_uint(st[3])};
  }
}

// Partial column sums a workgroup keeps: gate, w_pre, b_pre, w_post.
enum { P_GATE, P_WPRE, P_BPRE, P_WPOST, P_COUNT };

// Backward.  A workgroup takes rows of one group (or several whole groups), loads a row ahead,
// and keeps the column sums of its rows.  Gate and w_post need one sum between them:
// S = sum D n gives dg = w_post S and dw_post = g S (summed over groups where the gate is
// grouped).
//   SUMS: 2 (S, w_pre), 3 (b_pre too), 4 (and w_post over several groups with gates of their own).
//   AHEAD: the next row is loaded while a row is worked on.
//   ACC_BYTES: LDS for the column sums, where registers are short (16 columns a thread); 0 keeps
//     them in registers.
// The partial sums go to scratch memory, one row a workgroup and parameter (about 16 waves a
// compute unit, so few rows of them: 22 MB against 1.4 GB of operands at [16384, 7168]), and are
// joined in the order of the workgroups: no atomics, the same bits every time.
template <typename X, int V, bool RAGGED, bool LAYER, int SUMS, bool AHEAD, int ACC_BYTES, int MAXT>
__global__ __launch_bounds__(MAXT) void k_block_norm_bwd(NormBwdArgs a, NormBwdPlan plan) {
  constexpr bool LDS = ACC_BYTES > 0;
  // rms: one sum over the row at a time; layer: two (with the mean of the gradient)
  constexpr int ROW_SUMS = LAYER ? 2 : 1;
  __shared__ BlockParts<ROW_SUMS> part;
  __shared__ v4f in_lds[LDS ? ACC_BYTES / 16 : 1];
  int turn = 0;
  clear_parts(part);
  const int H = (int)a.H;
  const bool pf32 = a.flags & NORM_F32_PARAMS;
  const bool post = a.flags & NORM_POST, pre = a.flags & NORM_PRE, has_y = a.y != nullptr;
  const bool sums_y = a.gate.d != nullptr || a.w_post.d != nullptr;
  const float invH = 1.0f / (float)H;
  uint32_t col[V];
  int n[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    col[v] = 8u * (threadIdx.x + blockDim.x * v);
    n[v] = H - (int)col[v];
  }
  const uint32_t blk = blockIdx.x, per = (uint32_t)a.rows_per_group;
  // one group's rows cut into per_group parts of part_rows rows, or part_rows whole groups
  const bool split = plan.split;
  uint32_t g0, g1, r0, r1;
  if (split) {
    g0 = uniform(blk / plan.per_group);
    g1 = g0 + 1;
    r0 = g0 * per + min((blk - g0 * plan.per_group) * plan.part_rows, per);
    r1 = min(r0 + plan.part_rows, g1 * per);
  } else {
    g0 = min(blk * plan.part_rows, plan.groups);
    g1 = min(g0 + plan.part_rows, plan.groups);
    r0 = g0 * per;
    r1 = g1 * per;
  }

  float acc[LDS ? 1 : SUMS][V][8];
  // sum `which` of this thread's columns; in LDS each thread reaches only its own
  const unsigned half = V * blockDim.x;
  auto slot = [&](int which, int v) { return in_lds + 2 * half * which + blockDim.x * v + threadIdx.x; };
  auto add = [&](int which, int v, const float (&f)[8]) {
    if constexpr (LDS) {
      v4f* p = slot(which, v);
      p[0] += (v4f){f[0], f[1], f[2], f[3]};
      p[half] += (v4f){f[4], f[5], f[6], f[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) acc[which][v][i] += f[i];
    }
  };
  auto add_products = [&](int which, int v, const float (&f)[8], const float (&h)[8]) {
    if constexpr (LDS) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; i++) t[i] = f[i] * h[i];
      add(which, v, t);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) acc[which][v][i] = __builtin_fmaf(f[i], h[i], acc[which][v][i]);
    }
  };
  auto take = [&](int which, int v, float (&f)[8]) {
    if constexpr (LDS) {
      const v4f lo = slot(which, v)[0], hi = slot(which, v)[half];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        f[i] = lo[i];
        f[4 + i] = hi[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) f[i] = acc[which][v][i];
    }
  };
  auto clear = [&](int which, int v) {
    if constexpr (LDS) {
      slot(which, v)[0] = slot(which, v)[half] = (v4f)0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) acc[which][v][i] = 0.0f;
    }
  };
#pragma unroll
  for (int w = 0; w < SUMS; w++)
#pragma unroll
    for (int v = 0; v < V; v++) clear(w, v);

  Raw<X> lx[V], ld[V];
  Raw<uint16_t> ly[V], lh[V];
  auto start = [&](uint32_t r) {
    const int64_t row = r;
    load_row<X, V, RAGGED>(lx, (const X*)a.x + row * a.ld_x, col, n);
    if (has_y) load_row<uint16_t, V, RAGGED>(ly, a.y + row * a.ld_y, col, n);
    if (a.dx_out != nullptr) load_row<X, V, RAGGED>(ld, (const X*)a.dx_out + row * a.ld_dxo, col, n);
    if (pre) load_row<uint16_t, V, RAGGED>(lh, a.dh + row * a.ld_dh, col, n);
  };
  if (AHEAD && r0 < r1) start(r0);

  for (uint32_t g = g0, row = r0; g < g1; g++) {
    float gw[V][8], wq[V][8];   // gate w_post, and w_pre, of this group
    param_row<V, RAGGED>(gw, a.gate.p, g * a.gate.stride, col, n, pf32, 1.0f);
    if (a.w_post.p != nullptr) {
      param_row<V, RAGGED>(wq, a.w_post.p, 0, col, n, pf32, 1.0f);
#pragma unroll
      for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < 8; i++) gw[v][i] *= wq[v][i];
    }
    param_row<V, RAGGED>(wq, a.w_pre.p, g * a.w_pre.stride, col, n, pf32, 1.0f);
    const uint32_t end = split ? r1 : (g + 1) * per;
    for (; row < end; row++) {
      if constexpr (!AHEAD) start(row);
      const float* st = a.stats + 4 * (int64_t)row;
      const float my = st[0], ry = post ? st[1] : 1.0f, mx = st[2], rx = st[3];
      float ny[V][8], D[V][8], nx[V][8], dh[V][8];
#pragma unroll
      for (int v = 0; v < V; v++) {
        lx[v].get(nx[v]);
        if (has_y) ly[v].get(ny[v]);
        if (a.dx_out != nullptr) {
          ld[v].get(D[v]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; i++) D[v][i] = 0.0f;
        }
        if (pre) lh[v].get(dh[v]);
      }
      if (AHEAD && row + 1 < r1) start(row + 1);
      // Lanes past the row hold zeros throughout in the rms form; in the layer form the mean they
      // lose makes them nonzero, so they are cleared where a sum over the row would see them.
      if (has_y) {
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            if (post) {
              if constexpr (LAYER) ny[v][i] = inside<RAGGED>(i, n[v]) ? (ny[v][i] - my) * ry : 0.0f;
              else ny[v][i] *= ry;
            }
            nx[v][i] = __builtin_fmaf(gw[v][i], ny[v][i], a.res_scale * nx[v][i]);
          }
      }
      if (pre) {
        float s[ROW_SUMS] = {};
#pragma unroll
        for (int v = 0; v < V; v++) {
          if constexpr (SUMS > 2) add(2, v, dh[v]);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            if constexpr (LAYER) nx[v][i] = inside<RAGGED>(i, n[v]) ? (nx[v][i] - mx) * rx : 0.0f;
            else nx[v][i] *= rx;
          }
          add_products(1, v, dh[v], nx[v]);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            dh[v][i] *= wq[v][i];
            s[0] = __builtin_fmaf(dh[v][i], nx[v][i], s[0]);
            if constexpr (LAYER) s[1] += dh[v][i];
          }
        }
        block_sum(s, part, turn);
        const float c0 = s[0] * invH, c1 = LAYER ? s[ROW_SUMS - 1] * invH : 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const float d = LAYER ? dh[v][i] - c1 : dh[v][i];
            D[v][i] = __builtin_fmaf(rx, __builtin_fmaf(-c0, nx[v][i], d), D[v][i]);
          }
      }
#pragma unroll
      for (int v = 0; v < V; v++) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = a.res_scale * D[v][i];
        put<RAGGED>((X*)a.dx + (int64_t)row * a.ld_dx, col[v], d, n[v]);
      }
      if (has_y) {
        float s[ROW_SUMS] = {};
#pragma unroll
        for (int v = 0; v < V; v++) {
          if (sums_y) add_products(0, v, D[v], ny[v]);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            D[v][i] *= gw[v][i];
            if constexpr (LAYER) {
              if (!inside<RAGGED>(i, n[v])) D[v][i] = 0.0f;
              s[1] += D[v][i];
            }
            s[0] = __builtin_fmaf(D[v][i], ny[v][i], s[0]);
          }
        }
        float c0 = 0.0f, c1 = 0.0f;
        if (post) {
          block_sum(s, part, turn);
          c0 = s[0] * invH;
          c1 = LAYER ? s[ROW_SUMS - 1] * invH : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; i++) d[i] = ry * __builtin_fmaf(-c0, ny[v][i], LAYER ? D[v][i] - c1 : D[v][i]);
          put<RAGGED>(a.dy + (int64_t)row * a.ld_dy, col[v], d, n[v]);
        }
      }
    }
    // The group's rows here are done.  Where whole groups are taken, the gradients of grouped
    // parameters go out now and their sums start again; everything else goes to this workgroup's
    // row of partial sums after its last group.
    const bool own_gate = !split && a.gate.stride != 0;   // S is one group's
#pragma unroll
    for (int v = 0; v < V; v++) {
      auto give = [&](const NormGradParam& p, int which, const float (&f)[8]) {
        if (!split && p.stride != 0) {
          if (pf32) put<RAGGED>((float*)p.d + g * p.stride, col[v], f, n[v]);
          else put<RAGGED>((uint16_t*)p.d + g * p.stride, col[v], f, n[v]);
        } else if (g + 1 == g1) {
          put<RAGGED>(a.work + (int64_t)(which * plan.blocks + blk) * a.H, col[v], f, n[v]);
        }
      };
      auto times_S = [&](const NormGradParam& p, int64_t at, float (&f)[8]) {   // f = p S
        take(0, v, f);
        if (p.p == nullptr) return;
        float w[8];
        load_param<RAGGED>(w, p.p, at, col[v], n[v], pf32);
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] *= w[i];
      };
      float f[8];
      if (a.w_post.d != nullptr && (own_gate || g + 1 == g1)) {
        times_S(a.gate, g * a.gate.stride, f);
        if constexpr (SUMS > 3) {
          if (own_gate) {
            add(3, v, f);
            take(3, v, f);
          }
        }
        give(a.w_post, P_WPOST, f);
      }
      if (a.gate.d != nullptr && (own_gate || g + 1 == g1)) {
        times_S(a.w_post, 0, f);
        give(a.gate, P_GATE, f);
      }
      if (own_gate) clear(0, v);
      if (a.w_pre.d != nullptr) {
        take(1, v, f);
        give(a.w_pre, P_WPRE, f);
        if (!split && a.w_pre.stride != 0) clear(1, v);
      }
      if constexpr (SUMS > 2) {
        if (a.b_pre.d != nullptr) {
          take(2, v, f);
          give(a.b_pre, P_BPRE, f);
          if (!split && a.b_pre.stride != 0) clear(2, v);
        }
      }
    }
  }
}

// Joins the partial column sums, in a fixed order: 64 columns a workgroup, 16 waves over the
// partial rows, eight loads each in flight (13 -> 9 us for four sums of 8193 columns).  grid: (columns / 64, parameter, group).
constexpr int JOIN_WAVES = 16;
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_block_norm_join(NormBwdArgs a, NormBwdPlan plan) {
  __shared__ float sums[JOIN_WAVES][64];
  const NormGradParam p = blockIdx.y == P_GATE ? a.gate : blockIdx.y == P_WPRE ? a.w_pre
                          : blockIdx.y == P_BPRE ? a.b_pre : a.w_post;
  const bool split = plan.split;
  const bool grouped = p.stride != 0;
  if (p.d == nullptr || (!split && grouped) || (!grouped && blockIdx.z > 0)) return;
  const int64_t b0 = grouped ? (int64_t)blockIdx.z * plan.per_group : 0;
  const int64_t b1 = grouped ? b0 + plan.per_group : plan.blocks;
  const unsigned lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int64_t c = 64 * (int64_t)blockIdx.x + lane;
  const float* src = a.work + (int64_t)blockIdx.y * plan.blocks * a.H + c;
  float s = 0.0f;
  if (c < a.H) {
#pragma unroll 8
    for (int64_t b = b0 + wave; b < b1; b += JOIN_WAVES) s += src[b * a.H];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.H) {
    for (int w = 1; w < JOIN_WAVES; w++) s += sums[w][lane];
    const int64_t o = (int64_t)blockIdx.z * p.stride + c;
    if (a.flags & NORM_F32_PARAMS) ((float*)p.d)[o] = s;
    else ((uint16_t*)p.d)[o] = (uint16_t)pack_bf16(s, 0.0f);
  }
}

// 8 columns a thread up to 8192 columns, 16 above: a row is one workgroup's, of at most 1024 threads.
void threads_for(int64_t H, unsigned& threads, int& vecs) {
  vecs = H <= 8192 ? 1 : 2;
  threads = (unsigned)((H + 512 * vecs - 1) / (512 * vecs) * 64);
}

bool ragged(int64_t H, std::initializer_list<int64_t> strides) {
  bool r = H % 8 != 0;
  for (int64_t ld : strides) r |= ld % 8 != 0;
  return r;
}

}  // namespace

NormBwdPlan norm_bwd_plan(int64_t M, int64_t H, int64_t rows_per_group) {
  NormBwdPlan p{};
  threads_for(H, p.threads, p.vecs);
  p.groups = (uint32_t)(M / rows_per_group);
  // about 16 waves on each of the 256 compute units
  const int64_t want = 256 * (p.threads >= 1024 ? 1 : 1024 / p.threads);
  p.split = p.groups < want;
  if (p.split) {
    const int64_t most = (rows_per_group + 3) / 4;   // four rows or more a workgroup
    int64_t parts = (want + p.groups - 1) / p.groups;
    parts = parts < most ? parts : most;
    p.part_rows = (uint32_t)((rows_per_group + parts - 1) / parts);
    p.per_group = (uint32_t)((rows_per_group + p.part_rows - 1) / p.part_rows);
    p.blocks = p.groups * p.per_group;
  } else {
    p.part_rows = (uint32_t)((p.groups + want - 1) / want);
    p.per_group = 1;
    p.blocks = (uint32_t)((p.groups + p.part_rows - 1) / p.part_rows);
  }
  return p;
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  unsigned threads;
  int vecs;
  threads_for(a.H, threads, vecs);
  // as many workgroups as the kernel's registers leave room for on the 256 compute units
  const unsigned waves = vecs == 2 ? 16 : (a.flags & NORM_F32_STREAM) ? 20 : 28;
  const int64_t want = 256 * (waves * 64 > threads ? waves * 64 / threads : 1);
  const uint32_t rows = (uint32_t)((a.M + want - 1) / want);
  const dim3 grid((unsigned)((a.M + rows - 1) / rows));
  const bool rag = ragged(a.H, {a.ld_x, a.y ? a.ld_y : 0, a.y ? a.ld_xo : 0, a.h ? a.ld_h : 0});
  auto go = [&](auto X, auto V, auto R, auto Q) {
    return a.kind == NORM_LAYER
               ? launch_kernel(k_block_norm<decltype(X), decltype(V)::value, decltype(R)::value, decltype(Q)::value, true>,
                               grid, dim3(threads), s, a, rows)
               : launch_kernel(k_block_norm<decltype(X), decltype(V)::value, decltype(R)::value, decltype(Q)::value, false>,
                               grid, dim3(threads), s, a, rows);
  };
  auto with_v = [&](auto X, auto R, auto Q) {
    return vecs == 1 ? go(X, std::integral_constant<int, 1>{}, R, Q) : go(X, std::integral_constant<int, 2>{}, R, Q);
  };
  auto with_x = [&](auto X) {
    if (a.q != nullptr) return with_v(X, std::false_type{}, std::true_type{});
    return rag ? with_v(X, std::true_type{}, std::false_type{}) : with_v(X, std::false_type{}, std::false_type{});
  };
  return a.flags & NORM_F32_STREAM ? with_x(float{}) : with_x(uint16_t{});
}

hipError_t launch_block_norm_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t s) {
  auto join = [&](const NormBwdPlan& plan) {
    if (!a.gate.d && !a.w_pre.d && !a.b_pre.d && !a.w_post.d) return hipSuccess;
    return launch_kernel(k_block_norm_join, dim3((unsigned)((a.H + 63) / 64), P_COUNT, plan.split ? plan.groups : 1u),
                         dim3(64 * JOIN_WAVES), s, a, plan);
  };
  // no rows: sums over no partial rows
  if (a.M == 0) return join(NormBwdPlan{(uint32_t)groups, 0, 0, 0, true, 0, 0});
  const NormBwdPlan plan = norm_bwd_plan(a.M, a.H, a.rows_per_group);
  const bool rag = ragged(a.H, {a.ld_x, a.y ? a.ld_y : 0, a.dx_out ? a.ld_dxo : 0, a.dh ? a.ld_dh : 0, a.ld_dx,
                                a.y ? a.ld_dy : 0});
  const int sums = !plan.split && a.gate.stride != 0 && a.w_post.d ? 4 : a.b_pre.d ? 3 : 2;
  auto go = [&](auto X, auto V, auto R, auto S, auto AHEAD, auto BYTES, auto T) {
    auto of = [&](auto L) {
      return launch_kernel(k_block_norm_bwd<decltype(X), decltype(V)::value, decltype(R)::value, decltype(L)::value,
                                            decltype(S)::value, decltype(AHEAD)::value, decltype(BYTES)::value,
                                            decltype(T)::value>,
                           dim3(plan.blocks), dim3(plan.threads), s, a, plan);
    };
    return a.kind == NORM_LAYER ? of(std::true_type{}) : of(std::false_type{});
  };
#define GLU_I(n) std::integral_constant<int, n>{}
  auto with_v = [&](auto X, auto R) {
    const auto yes = std::true_type{};
    const auto no = std::false_type{};
    if (plan.vecs == 1) {
      return sums == 2   ? go(X, GLU_I(1), R, GLU_I(2), yes, GLU_I(0), GLU_I(1024))
             : sums == 3 ? go(X, GLU_I(1), R, GLU_I(3), yes, GLU_I(0), GLU_I(1024))
                         : go(X, GLU_I(1), R, GLU_I(4), yes, GLU_I(0), GLU_I(1024));
    }
    // 16 columns a thread: 64 bytes of LDS a thread and sum; past 768 threads a workgroup's
    // registers leave no room to load ahead
    if (sums == 2 && plan.threads <= 768) return go(X, GLU_I(2), R, GLU_I(2), yes, GLU_I(2 * 64 * 768), GLU_I(768));
    if (sums == 2) return go(X, GLU_I(2), R, GLU_I(2), no, GLU_I(2 * 64 * 1024), GLU_I(1024));
    if (sums == 3 && plan.threads <= 768) return go(X, GLU_I(2), R, GLU_I(3), yes, GLU_I(3 * 64 * 768), GLU_I(768));
    return go(X, GLU_I(2), R, GLU_I(4), no, GLU_I(0), GLU_I(1024));
  };
#undef GLU_I
  auto with_x = [&](auto X) { return rag ? with_v(X, std::true_type{}) : with_v(X, std::false_type{}); };
  const hipError_t e = a.flags & NORM_F32_STREAM ? with_x(float{}) : with_x(uint16_t{});
  return e == hipSuccess ? join(plan) : e;
}

}  // namespace glu
