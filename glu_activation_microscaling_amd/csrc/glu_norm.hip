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
#include "ffn_device.h"
#include "ffn_launch.h"

namespace glu {
namespace {

// Eight values of a parameter (BF16 or FP32 by a wave-uniform flag) at element offset o.
template <bool RAGGED>
__device__ __forceinline__ void load_param(float (&f)[8], const void* p, int64_t o, int n, bool f32) {
  if (f32) {
    Raw<float> r;
    load<RAGGED>(r, (const float*)p + o, n);
    r.get(f);
  } else {
    Raw<uint16_t> r;
    load<RAGGED>(r, (const uint16_t*)p + o, n);
    r.get(f);
  }
}

template <typename X, int V, bool RAGGED, bool MX, int MAXT>
__global__ __launch_bounds__(MAXT) void k_block_norm(NormArgs a) {
  __shared__ float part[2][16][1];
  int turn = 0;
  const int64_t row = blockIdx.x, grp = row / a.rows_per_group;
  const int H = (int)a.H;
  const bool pf32 = a.flags & NORM_F32_PARAMS, layer = a.kind == NORM_LAYER;
  const float invH = 1.0f / (float)H;
  int col[V], n[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    col[v] = 8 * (int)(threadIdx.x + blockDim.x * v);
    n[v] = H - col[v];
  }

  // v := v - mean (layer) with the elements outside the row kept zero; returns 1/sqrt(...)
  float mean = 0.0f;
  auto normalize = [&](float (&f)[V][8]) {
    mean = 0.0f;
    if (layer) {
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
        for (int i = 0; i < 8; i++) f[v][i] = i < n[v] ? f[v][i] - mean : 0.0f;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 8; i++) q[0] = __builtin_fmaf(f[v][i], f[v][i], q[0]);
    block_sum(q, part, turn);
    return 1.0f / __builtin_sqrtf(__builtin_fmaf(q[0], invH, a.eps));
  };

  float xo[V][8];
  float st[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const X* px = (const X*)a.x + row * a.ld_x;
  if (a.y == nullptr) {
#pragma unroll
    for (int v = 0; v < V; v++) {
      Raw<X> rx;
      load<RAGGED>(rx, px + col[v], n[v]);
      rx.get(xo[v]);
    }
  } else {
    Raw<X> rx[V];
    float z[V][8];
    const uint16_t* py = a.y + row * a.ld_y;
#pragma unroll
    for (int v = 0; v < V; v++) {
      Raw<uint16_t> ry;
      load<RAGGED>(ry, py + col[v], n[v]);
      load<RAGGED>(rx[v], px + col[v], n[v]);
      ry.get(z[v]);
    }
    if (a.flags & NORM_POST) {
      const float r = normalize(z);
      st[0] = mean;
      st[1] = r;
#pragma unroll
      for (int v = 0; v < V; v++) {
        float w[8];
        if (a.w_post.p != nullptr) load_param<RAGGED>(w, a.w_post.p, col[v], n[v], pf32);
#pragma unroll
        for (int i = 0; i < 8; i++) z[v][i] = a.w_post.p != nullptr ? z[v][i] * r * w[i] : z[v][i] * r;
      }
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
      float x[8], g[8];
      rx[v].get(x);
      if (a.gate.p != nullptr) {
        load_param<RAGGED>(g, a.gate.p, grp * a.gate.stride + col[v], n[v], pf32);
#pragma unroll
        for (int i = 0; i < 8; i++) xo[v][i] = __builtin_fmaf(g[i], z[v][i], a.res_scale * x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) xo[v][i] = __builtin_fmaf(a.res_scale, x[i], z[v][i]);
      }
      store<RAGGED>((X*)a.x_out + row * a.ld_xo + col[v], xo[v], n[v]);
    }
  }
  if (a.flags & NORM_PRE) {
    const float r = normalize(xo);
    st[2] = mean;
    st[3] = r;
#pragma unroll
    for (int v = 0; v < V; v++) {
      float w[8], b[8];
      if (a.w_pre.p != nullptr) {
        load_param<RAGGED>(w, a.w_pre.p, grp * a.w_pre.stride + col[v], n[v], pf32);
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] *= r;
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = r;
      }
      if (a.b_pre.p != nullptr) {
        load_param<RAGGED>(b, a.b_pre.p, grp * a.b_pre.stride + col[v], n[v], pf32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) b[i] = 0.0f;
      }
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; i++) h[i] = __builtin_fmaf(xo[v][i], w[i], b[i]);
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
          *reinterpret_cast<u32x2*>(a.q + row * a.H + col[v]) = (u32x2){c0, c1};
          if ((threadIdx.x & 3u) == 0) a.s[row * (a.H / 32) + col[v] / 32] = (uint8_t)sb;
        }
      } else {
        store<RAGGED>(a.h + row * a.ld_h + col[v], h, n[v]);
      }
    }
  }
  if (threadIdx.x == 0)
    *reinterpret_cast<u32x4*>(a.stats + 4 * row) =
        (u32x4){__float_as_uint(st[0]), __float_as_uint(st[1]), __float_as_uint(st[2]), __float_as_uint(st[3])};
}

// Partial column sums a workgroup keeps: gate, w_pre, b_pre, w_post.
enum { P_GATE, P_WPRE, P_BPRE, P_WPOST, P_COUNT };

template <typename X, int V, bool RAGGED, int MAXT>
__global__ __launch_bounds__(MAXT) void k_block_norm_bwd(NormBwdArgs a, NormBwdPlan plan) {
  __shared__ float part[2][16][2];
  int turn = 0;
  const int H = (int)a.H;
  const bool pf32 = a.flags & NORM_F32_PARAMS, layer = a.kind == NORM_LAYER;
  const bool post = a.flags & NORM_POST, pre = a.flags & NORM_PRE, has_y = a.y != nullptr;
  const float invH = 1.0f / (float)H;
  int col[V], n[V];
#pragma unroll
  for (int v = 0; v < V; v++) {
    col[v] = 8 * (int)(threadIdx.x + blockDim.x * v);
    n[v] = H - col[v];
  }
  const int64_t blk = blockIdx.x;
  // whole groups [g0, g1), or one group's rows split over per_group workgroups
  const bool split = plan.groups * plan.per_group == plan.blocks;
  const int64_t g0 = split ? blk / plan.per_group : blk * plan.groups / plan.blocks;
  const int64_t g1 = split ? g0 + 1 : (blk + 1) * plan.groups / plan.blocks;

  float acc[P_COUNT][V][8];
#pragma unroll
  for (int p = 0; p < P_COUNT; p++)
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 8; i++) acc[p][v][i] = 0.0f;

  for (int64_t g = g0; g < g1; g++) {
    int64_t r0 = g * a.rows_per_group, r1 = r0 + a.rows_per_group;
    if (split && plan.per_group > 1) {
      const int64_t i = blk % plan.per_group;
      r1 = r0 + (i + 1) * a.rows_per_group / plan.per_group;
      r0 += i * a.rows_per_group / plan.per_group;
    }
    float gt[V][8], wq[V][8], wp[V][8];   // gate, w_pre, w_post of this group
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
      for (int i = 0; i < 8; i++) gt[v][i] = wq[v][i] = wp[v][i] = 1.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
      if (a.gate.p != nullptr) load_param<RAGGED>(gt[v], a.gate.p, g * a.gate.stride + col[v], n[v], pf32);
      if (a.w_pre.p != nullptr) load_param<RAGGED>(wq[v], a.w_pre.p, g * a.w_pre.stride + col[v], n[v], pf32);
      if (a.w_post.p != nullptr) load_param<RAGGED>(wp[v], a.w_post.p, col[v], n[v], pf32);
    }
    for (int64_t row = r0; row < r1; row++) {
      const float* st = a.stats + 4 * row;
      const float my = st[0], ry = post ? st[1] : 1.0f, mx = st[2], rx = st[3];
      float ny[V][8], D[V][8], nx[V][8], dh[V][8];
#pragma unroll
      for (int v = 0; v < V; v++) {
        Raw<X> q;
        Raw<uint16_t> h;
        load<RAGGED>(q, (const X*)a.x + row * a.ld_x + col[v], n[v]);
        q.get(nx[v]);
        if (has_y) {
          load<RAGGED>(h, a.y + row * a.ld_y + col[v], n[v]);
          h.get(ny[v]);
        }
        if (a.dx_out != nullptr) {
          load<RAGGED>(q, (const X*)a.dx_out + row * a.ld_dxo + col[v], n[v]);
          q.get(D[v]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; i++) D[v][i] = 0.0f;
        }
        if (pre) {
          load<RAGGED>(h, a.dh + row * a.ld_dh + col[v], n[v]);
          h.get(dh[v]);
        }
      }
      if (has_y) {
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            if (post) ny[v][i] = i < n[v] ? (ny[v][i] - my) * ry : 0.0f;
            nx[v][i] = __builtin_fmaf(gt[v][i], ny[v][i] * wp[v][i], a.res_scale * nx[v][i]);
          }
      }
      if (pre) {
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            nx[v][i] = i < n[v] ? (nx[v][i] - mx) * rx : 0.0f;
            acc[P_WPRE][v][i] = __builtin_fmaf(dh[v][i], nx[v][i], acc[P_WPRE][v][i]);
            acc[P_BPRE][v][i] += dh[v][i];
            dh[v][i] *= wq[v][i];
            s[0] = __builtin_fmaf(dh[v][i], nx[v][i], s[0]);
            s[1] += dh[v][i];
          }
        block_sum(s, part, turn);
        const float c0 = s[0] * invH, c1 = layer ? s[1] * invH : 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++)
            D[v][i] = __builtin_fmaf(rx, dh[v][i] - __builtin_fmaf(nx[v][i], c0, c1), D[v][i]);
      }
#pragma unroll
      for (int v = 0; v < V; v++) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = a.res_scale * D[v][i];
        store<RAGGED>((X*)a.dx + row * a.ld_dx + col[v], d, n[v]);
      }
      if (has_y) {
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            if (i < n[v]) acc[P_GATE][v][i] = __builtin_fmaf(D[v][i], ny[v][i] * wp[v][i], acc[P_GATE][v][i]);
            D[v][i] *= gt[v][i];
            acc[P_WPOST][v][i] = __builtin_fmaf(D[v][i], ny[v][i], acc[P_WPOST][v][i]);
            D[v][i] *= wp[v][i];
            if (i < n[v]) {
              s[0] = __builtin_fmaf(D[v][i], ny[v][i], s[0]);
              s[1] += D[v][i];
            }
          }
        float c0 = 0.0f, c1 = 0.0f;
        if (post) {
          block_sum(s, part, turn);
          c0 = s[0] * invH;
          c1 = layer ? s[1] * invH : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; i++) d[i] = ry * (D[v][i] - __builtin_fmaf(ny[v][i], c0, c1));
          store<RAGGED>(a.dy + row * a.ld_dy + col[v], d, n[v]);
        }
      }
    }
    // a whole group of a grouped parameter is done: its gradient goes out at once
    if (!split) {
      auto flush = [&](const NormGradParam& p, float (&s)[V][8]) {
        if (p.stride == 0) return;
#pragma unroll
        for (int v = 0; v < V; v++) {
          if (p.d != nullptr) {
            if (pf32) store<RAGGED>((float*)p.d + g * p.stride + col[v], s[v], n[v]);
            else store<RAGGED>((uint16_t*)p.d + g * p.stride + col[v], s[v], n[v]);
          }
#pragma unroll
          for (int i = 0; i < 8; i++) s[v][i] = 0.0f;
        }
      };
      flush(a.gate, acc[P_GATE]);
      flush(a.w_pre, acc[P_WPRE]);
      flush(a.b_pre, acc[P_BPRE]);
    }
  }
  auto keep = [&](const NormGradParam& p, float (&s)[V][8], int which) {
    if (p.d == nullptr || (!split && p.stride != 0)) return;
#pragma unroll
    for (int v = 0; v < V; v++)
      store<RAGGED>(a.work + (which * plan.blocks + blk) * a.H + col[v], s[v], n[v]);
  };
  keep(a.gate, acc[P_GATE], P_GATE);
  keep(a.w_pre, acc[P_WPRE], P_WPRE);
  keep(a.b_pre, acc[P_BPRE], P_BPRE);
  keep(a.w_post, acc[P_WPOST], P_WPOST);
}

// Joins the partial column sums, in the order of the workgroups: 64 columns a workgroup, 16
// waves over the partial rows.  grid: (columns / 64, parameter, group).
constexpr int JOIN_WAVES = 16;
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_block_norm_join(NormBwdArgs a, NormBwdPlan plan) {
  __shared__ float sums[JOIN_WAVES][64];
  const NormGradParam p = blockIdx.y == P_GATE ? a.gate : blockIdx.y == P_WPRE ? a.w_pre
                          : blockIdx.y == P_BPRE ? a.b_pre : a.w_post;
  const bool split = plan.groups * plan.per_group == plan.blocks;
  const bool grouped = p.stride != 0;
  if (p.d == nullptr || (!split && grouped) || (!grouped && blockIdx.z > 0)) return;
  const int64_t b0 = grouped ? blockIdx.z * plan.per_group : 0;
  const int64_t b1 = grouped ? b0 + plan.per_group : plan.blocks;
  const unsigned lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const int64_t c = 64 * (int64_t)blockIdx.x + lane;
  const float* src = a.work + blockIdx.y * plan.blocks * a.H + c;
  float s = 0.0f;
  if (c < a.H)
    for (int64_t b = b0 + wave; b < b1; b += JOIN_WAVES) s += src[b * a.H];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.H) {
    for (int w = 1; w < JOIN_WAVES; w++) s += sums[w][lane];
    const int64_t o = (int64_t)blockIdx.z * p.stride + c;
    if (a.flags & NORM_F32_PARAMS) ((float*)p.d)[o] = s;
    else ((uint16_t*)p.d)[o] = (uint16_t)pack_bf16(s, 0.0f);
  }
}

// 8 columns a thread up to 8192 columns, 16 above.
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
  p.groups = M / rows_per_group;
  // about 16 waves on each of the 256 compute units
  const int64_t want = 256 * (p.threads >= 1024 ? 1 : 1024 / p.threads);
  if (p.groups < want) {
    int64_t per = (want + p.groups - 1) / p.groups;
    const int64_t most = (rows_per_group + 3) / 4;   // four rows or more a workgroup
    p.per_group = per < most ? per : most;
    p.blocks = p.groups * p.per_group;
  } else {
    p.per_group = 1;
    p.blocks = want;
  }
  return p;
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  unsigned threads;
  int vecs;
  threads_for(a.H, threads, vecs);
  const bool rag = ragged(a.H, {a.ld_x, a.y ? a.ld_y : 0, a.y ? a.ld_xo : 0, a.h ? a.ld_h : 0});
  auto go = [&](auto X, auto V, auto R, auto Q, auto T) {
    return launch_kernel(k_block_norm<decltype(X), decltype(V)::value, decltype(R)::value, decltype(Q)::value,
                                      decltype(T)::value>,
                         dim3((unsigned)a.M), dim3(threads), s, a);
  };
  auto with_v = [&](auto X, auto R, auto Q) {
    return vecs == 1 ? go(X, std::integral_constant<int, 1>{}, R, Q, std::integral_constant<int, 1024>{})
                     : go(X, std::integral_constant<int, 2>{}, R, Q, std::integral_constant<int, 1024>{});
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
    const bool split = plan.groups * plan.per_group == plan.blocks;
    return launch_kernel(k_block_norm_join,
                         dim3((unsigned)((a.H + 63) / 64), P_COUNT, split ? (unsigned)plan.groups : 1u),
                         dim3(64 * JOIN_WAVES), s, a, plan);
  };
  // no rows: sums over no partial rows
  if (a.M == 0) return join(NormBwdPlan{groups, 0, 0, 0, 0});
  const NormBwdPlan plan = norm_bwd_plan(a.M, a.H, a.rows_per_group);
  const bool rag = ragged(a.H, {a.ld_x, a.y ? a.ld_y : 0, a.dx_out ? a.ld_dxo : 0, a.dh ? a.ld_dh : 0, a.ld_dx,
                                a.y ? a.ld_dy : 0});
  auto go = [&](auto X, auto V, auto R, auto T) {
    return launch_kernel(k_block_norm_bwd<decltype(X), decltype(V)::value, decltype(R)::value, decltype(T)::value>,
                         dim3((unsigned)plan.blocks), dim3(plan.threads), s, a, plan);
  };
  auto with_v = [&](auto X, auto R) {
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    if (plan.vecs == 1) return go(X, I1{}, R, std::integral_constant<int, 1024>{});
    return plan.threads <= 640 ? go(X, I2{}, R, std::integral_constant<int, 640>{})
                               : go(X, I2{}, R, std::integral_constant<int, 1024>{});
  };
  auto with_x = [&](auto X) { return rag ? with_v(X, std::true_type{}) : with_v(X, std::false_type{}); };
  hipError_t e = a.flags & NORM_F32_STREAM ? with_x(float{}) : with_x(uint16_t{});
  return e == hipSuccess ? join(plan) : e;
}

}  // namespace glu
