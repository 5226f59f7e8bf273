// Tokens sorted by expert and back: the places of a stable counting sort, the copy of token
// rows into that order, the weighted sum of the experts' rows back into tokens, and the
// gradients.
//
//   rows[t, j] = offsets[e] + #{(t', j') before (t, j) in reading order with expert e},
//                e = ids[t, j];  -1 where e is not an expert (a dropped choice)
//   xs[rows[t, j]] = x[t];  rows of xs past offsets[E] are zero
//   out[t] = residual[t] + sum_j w[t, j] y[rows[t, j]]  over the choices that are not dropped
//   dy[rows[t, j]] = w[t, j] dout[t];  dw[t, j] = <dout[t], y[rows[t, j]]>
//
// With w = 1 the sum is also the gradient of the copy.  The copy and the gradients go by token,
// so a token's row is read from memory once however many experts take it; every row of xs or dy
// is written by one workgroup alone and sums run in the order of j: no atomics, and the same
// bits every time.
//
// All but the sort are bound by memory.  Measured on an MI355X (a copy of 1 GiB: 5.1 TB/s) for 8192
// tokens, 8 of 64 experts, 7168 columns:
//   sort 5.0 + 6.2 us, copy 186 us (5.7 TB/s, nearly all of it writes), sum 223 to 246 us (4.3 to
//   4.7 TB/s, nearly all of it reads), gradients 394 us (5.1 TB/s)
// and for 4 tokens of 2048 columns 4 us each, which is what a launch takes.
#include "ffn_device.h"
#include "ffn_launch.h"

namespace glu {
namespace {

constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64;

__device__ __forceinline__ int expert_at(const void* ids, int64_t i, int bytes, int experts) {
  const int64_t e = bytes == 8 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
  return e >= 0 && e < experts ? (int)e : -1;
}

__device__ __forceinline__ int64_t sort_begin(int64_t n, int64_t parts, int64_t i) { return n * i / parts; }

// Counts of each expert in each workgroup's part, by integer additions in LDS (whose order does
// not matter).
__global__ __launch_bounds__(SORT_THREADS) void k_moe_count(MoeSortArgs a) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += SORT_THREADS) count[e] = 0;
  __syncthreads();
  const int64_t i0 = sort_begin(a.n, gridDim.x, blockIdx.x), i1 = sort_begin(a.n, gridDim.x, blockIdx.x + 1);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += SORT_THREADS) {
    const int e = expert_at(a.ids, i, a.id_bytes, a.experts);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += SORT_THREADS) a.work[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// Places.  A workgroup takes a contiguous part of the choices and each of its waves a
// contiguous part of that, so a choice's place is the start of its expert, plus the choices
// of that expert in earlier workgroups (from k_moe_count), in earlier waves, and in earlier
// lanes of its own wave (a ballot for each bit of the expert's number finds the lanes that
// share it).  Bound by latency: two passes over a part's numbers.
__global__ __launch_bounds__(SORT_THREADS) void k_moe_place(MoeSortArgs a) {
  __shared__ int next[SORT_WAVES][kMaxExperts];   // counts, then the next place, per wave
  __shared__ int wave_total[SORT_WAVES], sum_all[kMaxExperts], sum_early[kMaxExperts];
  const int E = a.experts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b0 = sort_begin(a.n, gridDim.x, blockIdx.x), b1 = sort_begin(a.n, gridDim.x, blockIdx.x + 1);
  const int64_t i0 = b0 + sort_begin(b1 - b0, SORT_WAVES, wave), i1 = b0 + sort_begin(b1 - b0, SORT_WAVES, wave + 1);
  for (int x = threadIdx.x; x < E; x += SORT_THREADS) {
    for (int w = 0; w < SORT_WAVES; w++) next[w][x] = 0;
    sum_all[x] = sum_early[x] = 0;
  }
  __syncthreads();
  for (int64_t i = i0 + lane; i < i1; i += 64) {
    const int e = expert_at(a.ids, i, a.id_bytes, E);
    if (e >= 0) atomicAdd(&next[wave][e], 1);
  }
  __syncthreads();
  // totals of the experts, and of them what earlier workgroups have; 1024 / E threads an expert
  // share the other workgroups' counts
  const int e = threadIdx.x;
  int total = 0, before = 0;
  if (gridDim.x > 1) {
    const int share = SORT_THREADS / E, part = threadIdx.x / E, x = threadIdx.x % E;
    if (part < share) {
      int all = 0, early = 0;
#pragma unroll 4
      for (unsigned b = part; b < gridDim.x; b += share) {
        const int c = a.work[(int64_t)b * E + x];
        all += c;
        early += b < blockIdx.x ? c : 0;
      }
      atomicAdd(&sum_all[x], all);
      atomicAdd(&sum_early[x], early);
    }
    __syncthreads();
    if (e < E) {
      total = sum_all[e];
      before = sum_early[e];
    }
  } else if (e < E) {
    for (int w = 0; w < SORT_WAVES; w++) total += next[w][e];
  }
  // thread e: the expert's start is the scan of the totals; this workgroup's counts become places
  int scan = total;
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 63) wave_total[wave] = scan;
  __syncthreads();
  int start = scan - total;
  for (int w = 0; w < wave; w++) start += wave_total[w];
  if (e < E) {
    if (blockIdx.x == 0) {
      a.offsets[e] = start;
      if (e == E - 1) a.offsets[E] = start + total;
    }
    int at = start + before;
    for (int w = 0; w < SORT_WAVES; w++) {
      const int c = next[w][e];
      next[w][e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t base = i0; base < i1; base += 64) {
    const int64_t i = base + lane;
    const int id = i < i1 ? expert_at(a.ids, i, a.id_bytes, E) : -1;
    uint64_t same = __ballot(id >= 0);
    for (int bit = 0; (1 << bit) < E; bit++) {
      const uint64_t set = __ballot((id >> bit) & 1);
      same &= (id >> bit) & 1 ? set : ~set;
    }
    int place = -1;
    if (id >= 0) {
      const int first = next[wave][id], ahead = __popcll(same & ((1ull << lane) - 1));
      place = first + ahead;
      if (ahead == 0) next[wave][id] = first + __popcll(same);
    }
    if (i < i1) a.rows[i] = place;
  }
}

struct __attribute__((packed)) Bytes16 {
  u32x4 v;
};

constexpr int MOVE_THREADS = 256;

// Zeroes the rows of `out` past the last expert's that workgroup (t, part) is given: as many
// as a token has choices, so that all of them are covered however many choices were dropped.
__device__ __forceinline__ void zero_tail(uint8_t* out, int64_t ld, int64_t row_bytes, int64_t used, int64_t rows,
                                          int64_t t, int64_t choices, int64_t c0, int64_t c1) {
  for (int64_t j = 0; j < choices; j++) {
    const int64_t r = used + t * choices + j;
    if (r >= rows) return;
    uint8_t* p = out + r * ld;
    for (int64_t c = c0 + 16 * (int64_t)threadIdx.x; c < c1; c += 16 * MOVE_THREADS) {
      if (c + 16 <= row_bytes) {
        reinterpret_cast<Bytes16*>(p + c)->v = (u32x4)0u;
      } else {
        for (int64_t i = c; i < row_bytes; i++) p[i] = 0;
      }
    }
  }
}

// The copy: 16 bytes a lane, read once and written to each of the token's places.  By bytes, so
// one kernel serves every type, FP8 rows included.  grid: (parts of a row of 4 KiB, tokens)
constexpr int64_t MOVE_PART = 16 * MOVE_THREADS;
__global__ __launch_bounds__(MOVE_THREADS) void k_moe_permute(MoePermuteArgs a) {
  const int64_t c0 = MOVE_PART * blockIdx.x, c1 = min(c0 + MOVE_PART, a.row_bytes);
  const int64_t c = c0 + 16 * (int64_t)threadIdx.x;
  const int64_t used = max(a.offsets[a.experts], 0), rows = a.tokens * a.choices;
  for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    if (c < c1) {
      const uint8_t* src = a.x + t * a.ld_x + c;
      if (c + 16 <= a.row_bytes) {
        const u32x4 v = reinterpret_cast<const Bytes16*>(src)->v;
        for (int64_t j = 0; j < a.choices; j++) {
          const int64_t r = a.rows[t * a.choices + j];
          if (r >= 0 && r < rows) reinterpret_cast<Bytes16*>(a.xs + r * a.ld_xs + c)->v = v;
        }
      } else {
        for (int64_t j = 0; j < a.choices; j++) {
          const int64_t r = a.rows[t * a.choices + j];
          if (r >= 0 && r < rows)
            for (int64_t i = 0; i < a.row_bytes - c; i++) a.xs[r * a.ld_xs + c + i] = src[i];
        }
      }
    }
    zero_tail(a.xs, a.ld_xs, a.row_bytes, used, rows, t, a.choices, c0, c1);
  }
}

// The weighted sum: FP32 sums of up to eight rows in flight at a time, in the order of j, rounded
// once.  grid: (parts of 2048 columns, tokens)
constexpr int64_t SUM_PART = 8 * MOVE_THREADS;
constexpr int SUM_CHOICES = 8;
template <bool RAGGED>
__global__ __launch_bounds__(MOVE_THREADS) void k_moe_combine(MoeCombineArgs a) {
  const int64_t c = SUM_PART * blockIdx.x + 8 * (int64_t)threadIdx.x;
  if (c >= a.H) return;
  const int n = (int)min((int64_t)8, a.H - c);
  const int64_t rows = a.tokens * a.choices;
  for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (a.residual != nullptr) {
      Raw<uint16_t> r;
      load<RAGGED>(r, a.residual + t * a.ld_res, (uint32_t)c, n);
      r.get(s);
    }
    for (int64_t j0 = 0; j0 < a.choices; j0 += SUM_CHOICES) {
      // all rows of the batch are in flight before the first is added
      Raw<uint16_t> q[SUM_CHOICES];
      float w[SUM_CHOICES];
#pragma unroll
      for (int j = 0; j < SUM_CHOICES; j++) {
        const int64_t i = t * a.choices + j0 + j;
        const int64_t r = j0 + j < a.choices ? a.rows[i] : -1;
        w[j] = 0.0f;
        q[j].a = (u32x4)0u;
        if (r >= 0 && r < rows) {
          load<RAGGED>(q[j], a.y + r * a.ld_y, (uint32_t)c, n);
          w[j] = a.weights != nullptr ? a.weights[i] : 1.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < SUM_CHOICES; j++) {
        float f[8];
        q[j].get(f);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] = __builtin_fmaf(w[j], f[i], s[i]);
      }
    }
    store<RAGGED>(a.out + t * a.ld_out, (uint32_t)c, s, n);
  }
}

// The gradients: one workgroup a token, so that a token's eight dot products are whole in it and its
// row of dout is read once; eight choices at a time.
constexpr int GRAD_CHOICES = 8;
template <bool RAGGED>
__global__ __launch_bounds__(MOVE_THREADS) void k_moe_combine_bwd(MoeCombineBwdArgs a) {
  __shared__ BlockParts<GRAD_CHOICES> part;
  int turn = 0;
  clear_parts(part);
  const int64_t used = max(a.offsets[a.experts], 0), rows = a.tokens * a.choices;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    for (int64_t j0 = 0; j0 < a.choices; j0 += GRAD_CHOICES) {
      int64_t r[GRAD_CHOICES];
      float w[GRAD_CHOICES], dot[GRAD_CHOICES];
#pragma unroll
      for (int j = 0; j < GRAD_CHOICES; j++) {
        const int64_t i = t * a.choices + j0 + j;
        r[j] = j0 + j < a.choices ? a.rows[i] : -1;
        if (r[j] >= rows) r[j] = -1;
        w[j] = j0 + j < a.choices ? a.weights[i] : 0.0f;
        dot[j] = 0.0f;
      }
      for (int64_t c = 8 * (int64_t)threadIdx.x; c < a.H; c += SUM_PART) {
        const int n = (int)min((int64_t)8, a.H - c);
        Raw<uint16_t> q;
        float g[8];
        load<RAGGED>(q, a.dout + t * a.ld_dout, (uint32_t)c, n);
        q.get(g);
#pragma unroll
        for (int j = 0; j < GRAD_CHOICES; j++) {
          if (r[j] < 0) continue;
          float f[8], d[8];
          load<RAGGED>(q, a.y + r[j] * a.ld_y, (uint32_t)c, n);
          q.get(f);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            dot[j] = __builtin_fmaf(g[i], f[i], dot[j]);
            d[i] = w[j] * g[i];
          }
          store<RAGGED>(a.dy + r[j] * a.ld_dy, (uint32_t)c, d, n);
        }
      }
      block_sum(dot, part, turn);
      if (threadIdx.x == 0) {
#pragma unroll
        for (int j = 0; j < GRAD_CHOICES; j++)
          if (j0 + j < a.choices) a.dweights[t * a.choices + j0 + j] = dot[j];
      }
    }
    zero_tail((uint8_t*)a.dy, 2 * a.ld_dy, 2 * a.H, used, rows, t, a.choices, 0, 2 * a.H);
  }
}

}  // namespace

// Workgroups of the sort: one up to 4096 choices, in one launch, else parts of 1024 choices or more,
// at most 64 (each reads the others' counts).  One part against several, back to back in a graph:
// 2048 choices 4.8 / 6.6 us, 4096 6.5 / 6.7, 8192 10.1 / 6.8, 65536 59 / 7.9.
int64_t moe_sort_blocks(int64_t n) {
  if (n <= 4 * SORT_THREADS) return 1;
  const int64_t b = (n + SORT_THREADS - 1) / SORT_THREADS;
  return b < 64 ? b : 64;
}

hipError_t launch_moe_sort(const MoeSortArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)moe_sort_blocks(a.n);
  if (blocks > 1) {
    const hipError_t e = launch_kernel(k_moe_count, dim3(blocks), dim3(SORT_THREADS), s, a);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(k_moe_place, dim3(blocks), dim3(SORT_THREADS), s, a);
}

hipError_t launch_moe_permute(const MoePermuteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.row_bytes + MOVE_PART - 1) / MOVE_PART), (unsigned)(a.tokens < 65535 ? a.tokens : 65535));
  return launch_kernel(k_moe_permute, grid, dim3(MOVE_THREADS), s, a);
}

hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.H + SUM_PART - 1) / SUM_PART), (unsigned)(a.tokens < 65535 ? a.tokens : 65535));
  const bool rag = a.H % 8 != 0 || a.ld_y % 8 != 0 || a.ld_out % 8 != 0 || (a.residual && a.ld_res % 8 != 0);
  return rag ? launch_kernel(k_moe_combine<true>, grid, dim3(MOVE_THREADS), s, a)
             : launch_kernel(k_moe_combine<false>, grid, dim3(MOVE_THREADS), s, a);
}

hipError_t launch_moe_combine_bwd(const MoeCombineBwdArgs& a, hipStream_t s) {
  const dim3 grid(grid_for(a.tokens, (int64_t)1 << 20));
  const bool rag = a.H % 8 != 0 || a.ld_y % 8 != 0 || a.ld_dout % 8 != 0 || a.ld_dy % 8 != 0;
  return rag ? launch_kernel(k_moe_combine_bwd<true>, grid, dim3(MOVE_THREADS), s, a)
             : launch_kernel(k_moe_combine_bwd<false>, grid, dim3(MOVE_THREADS), s, a);
}

}  // namespace glu
