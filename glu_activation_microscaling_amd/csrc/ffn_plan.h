// Which kernel a product takes: tile sizes and rules on extents alone, so that the scratch memory of split
// sums can be sized before the launch.  Plain C++: the launches use it and a host compiler takes it alone.
#pragma once

#include <stdint.h>

namespace glu {

enum { FWD, DGRAD, WGRAD, GATED };   // forward, gradient of x, gradient of W, gated projection

constexpr uint32_t BK = 64;   // elements of the sum per step: one 128-byte line of a row
// Up to 8 rows of one group: rows, columns a wave, waves a workgroup, elements of a chunk of the sum.
constexpr int FEW_WAVES = 8, FEW_ROWS = 8, FEW_COLS = 8, FEW_CHUNK = 128;

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
  double us;                 // the rule's estimate, of the tiled ones
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kUnits = 256;

// What a tile takes, in microseconds a step of the sum and for its start and end, and what joining the parts of a split
// sum takes.  The least total over the first three sizes decides.
struct ProductCost {
  double step[3];            // while more than half the chip works
  double few[3];             // while at most half of it does
  double tile[3];
  // how much longer a step takes where operand rows start off a 128-byte line, so that a load asks for two lines
  double off_line[3], off_line_few[3];
  double join_us, join_tbps;
  int64_t least;             // elements of a part of the sum
};
// Fitted to the linear products, their gradients and products of groups at each size and count of parts, 181 calls of
// up to eight rounds of workgroups: of them the rule takes the fastest or is within 3% of it but for seven (3 to 8%).
// Measured for [I, J, K], in a graph, 256x256 / 256x128 / 128x128:
//   [ 1000, 1000, 1000]  22.2 / 19.2 / 13.6      [ 4096, 4096, 1024]  31.7 /  40.2 /  45.7
//   [  968, 2048, 4096]  66.2 / 43.8 / 29.9      [ 4096, 4096, 4096]  94.1 / 113.6 / 132.5
//   [ 2048, 4096, 4096]  75.6 / 58.4 / 68.4      [ 6000, 4096, 2048]  91.1 /  93.6 / 111.1
//   gradient of x [2048, 8192, 512]  23.5 / 30.3 / 31.9      of W, 8 groups, 4096 rows, [4096, 2048]  85.6 / 111 / 123
// and in 1 / 2 / 3 / 4 parts, 128x128: [512, 2048, 2048] 16.9 / 19.1 / 19.1 / 20.6, [1021, 1000, 2056] 23.3 / 19.0 / 19.4 /
// 20.2, [1024, 1024, 4096] 28.3 / 22.6 / 20.7 / 21.2.
constexpr ProductCost kLinearCost = {{1.0, 0.76, 0.48}, {0.95, 0.65, 0.40}, {12.0, 7.5, 4.7}, {1.0, 1.1, 1.4}, {1.0, 1.05, 1.2},
                                     4.0, 6.0, 512};

// The number of parts of a sum that takes the least time: one, a power of two or the most, at least cost.least
// elements each and one round of workgroups in all.
struct Parts {
  int64_t splits;
  double us;
};
inline Parts best_parts(const ProductCost& cost, int kind, int64_t tiles, int64_t K, int64_t steps, int64_t outputs, bool whole,
                        bool off_line) {
  const int64_t fit = whole ? 1 : K / cost.least < kUnits / tiles ? K / cost.least : kUnits / tiles, most = fit < 1 ? 1 : fit;
  Parts best{0, 0.0};
  for (int64_t splits = 1;;) {
    const bool half = tiles * splits <= kUnits / 2;
    double step = half ? cost.few[kind] : cost.step[kind];
    if (off_line) step *= half ? cost.off_line_few[kind] : cost.off_line[kind];
    double us = (cost.tile[kind] + step * ceil_div(steps, splits)) * ceil_div(tiles * splits, kUnits);
    if (splits > 1) us += cost.join_us + 8e-6 / cost.join_tbps * splits * outputs;
    if (best.splits == 0 || us < best.us) best = {splits, us};
    if (splits == most) return best;
    splits = 2 * splits < most ? 2 * splits : most;
  }
}

// A rule on extents alone, so that the scratch memory of split sums can be sized before the
// launch.  whole: sums are not cut.
inline ProductPlan plan_one(int mode, int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped, bool whole) {
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
    const Parts parts = best_parts(kLinearCost, kind, tiles, K, steps, I * J, whole || grouped || kind == TILE_256,
                                   mode == FWD && K % BK != 0);
    if (best == 0.0 || parts.us < best) {
      best = parts.us;
      p.kind = kind;
      p.tiles_i = ti + extra;
      p.tiles_j = tj;
      p.splits = parts.splits;
    }
  }
  p.us = best;
  return p;
}

// Both gradients in one launch, for x [M, K] and dp [M, N] without groups, every sum in one piece: when all tiles of
// both run at once and that is estimated to take less than one product after the other.  The parts of a sum must not
// depend on whether the other gradient is formed (they show in the last bits), so a gradient formed alone is not cut
// either where this is taken, and what the two gain together has to be more than what they lose alone.  The
// tiles' kind, or -1.  Measured for [M, N, K], in a graph, one after the other / together: [256, 512, 512] 12.1 / 6.7
// us, [1000, 1000, 1000] 21.2 / 11.7, [1024, 2048, 2048] 30.4 / 26.8, [1021, 2000, 2056] 38.5 / 31.3; where one alone would
// be cut, and it alone cut / whole: [3000, 1000, 1000] 33.3 / 26.2, dW 20.5 / 25.2; [2000, 512, 512] 20.7 / 18.0, dW 13.4 /
// 17.5 (the rule takes the gain for 5.9); not taken [512, 2048, 512], 19.9 / 16.1, dx 12.4 / 17.
constexpr double kLaunchUs = 3.5;   // a launch and the gap before it
inline int plan_gradients(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0) return -1;
  const double apart = plan_one(DGRAD, M, K, N, 1, false, false).us + plan_one(WGRAD, N, K, M, 1, false, false).us;
  const double uncut = plan_one(DGRAD, M, K, N, 1, false, true).us + plan_one(WGRAD, N, K, M, 1, false, true).us;
  double best = apart + kLaunchUs - (uncut - apart);
  int kind = -1;
  for (int k = TILE_256_128; k <= TILE_128; k++) {
    const int64_t rows = kShape[k].rows(), j = ceil_div(K, kShape[k].cols());
    const int64_t tiles = ceil_div(M, rows) * j + ceil_div(N, rows) * j;
    if (tiles > kUnits) continue;
    const ProductCost& c = kLinearCost;
    const double us = c.tile[k] + (tiles <= kUnits / 2 ? c.few[k] : c.step[k]) * ceil_div(M > N ? M : N, BK);
    if (us < best) {
      best = us;
      kind = k;
    }
  }
  return kind;
}

inline ProductPlan plan_product(int mode, int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped) {
  const ProductPlan p = plan_one(mode, I, J, K, groups, grouped, false);
  if (p.splits == 1 || (mode != DGRAD && mode != WGRAD)) return p;
  const int joint = mode == DGRAD ? plan_gradients(I, K, J) : plan_gradients(K, I, J);
  return joint < 0 ? p : plan_one(mode, I, J, K, groups, grouped, true);
}

// ---- gated projections ------------------------------------------------------------------------

// Columns of a gated product's sums: 16 gate and 16 up for each 16 outputs.
constexpr int64_t gated_columns(int64_t J) { return (J + 15) / 16 * 32; }

// The tile sizes of the linear products, each with waves of 64 columns of the sums (32 outputs).  Their loops take the
// linear products' time; a tile's end takes 1 us more, and up to 5 a 256 x 256 tile where gate and up are kept.  Of 79 calls
// as above the rule is 3 to 7% behind on twelve: where three or six parts would be best, and [1021, 2 x 1000, 2056], which
// it leaves whole.  With codes, in a graph, 256x256
// / 256x128 / 128x128: [968, 2 x 1024, 2048] 43.0 / 28.2 / 19.5, [2048, 2 x 2048, 4096] 83.3 / 60.5 / 75.1, [4096, 2 x 2048,
// 1024] 36.4 / 44.7 / 55.4, 16 groups, 8192 rows, [2 x 2048, 1024] 99.3 / 129 / 143; in 1 / 2 / 4 parts, 128x128, [1021, 2 x
// 1000, 2056] 25.7 / 24.4 / 30.8, [128, 2 x 4096, 4096] 30.3 / 24.0 / 22.9.
constexpr TileShape kGatedShape[4] = {{2, 4, 8, 4, 2}, {4, 2, 4, 4, 3}, {4, 2, 2, 4, 3}, {2, 2, 1, 4, 4}};
constexpr ProductCost kGatedCost = {{1.1, 0.76, 0.48}, {0.95, 0.65, 0.40}, {13.5, 8.0, 5.5}, {1.0, 1.1, 1.4}, {1.0, 1.05, 1.2},
                                    4.0, 6.0, 512};

// Codes need whole blocks of 32 outputs, which the few rows' kernel does not have.
inline ProductPlan plan_gated(bool codes, int64_t I, int64_t N, int64_t K, int64_t groups, bool grouped) {
  const int64_t J = gated_columns(N);
  ProductPlan p{};
  p.splits = 1;
  if (I == 0 || N == 0) return p;
  if (!grouped && I <= FEW_ROWS && !codes) {
    p.kind = FEW;
    const int64_t cols = ceil_div(N, FEW_COLS);
    p.share = 1;
    while (p.share < FEW_WAVES / 2 && 2 * cols * p.share < 16 * kUnits && K >= 8 * p.share * FEW_CHUNK) p.share *= 2;
    p.tiles_j = ceil_div(2 * cols * p.share, FEW_WAVES);
    return p;
  }
  if (grouped && I <= kGatedShape[TILE_32].rows() / 2 * groups) {
    p.kind = TILE_32;
    p.tiles_i = ceil_div(I, kGatedShape[TILE_32].rows()) + groups + 1;
    p.tiles_j = ceil_div(J, kGatedShape[TILE_32].cols());
    return p;
  }
  const int64_t extra = grouped ? groups + 1 : 0, steps = ceil_div(K, BK);
  double best = 0.0;
  for (int kind = TILE_256; kind <= TILE_128; kind++) {
    const int64_t ti = ceil_div(I, kGatedShape[kind].rows()), tj = ceil_div(J, kGatedShape[kind].cols());
    const int64_t tiles = (ti + (grouped ? groups / 2 : 0)) * tj;
    const Parts parts = best_parts(kGatedCost, kind, tiles, K, steps, I * J, grouped || kind == TILE_256, K % BK != 0);
    if (best == 0.0 || parts.us < best) {
      best = parts.us;
      p.kind = kind;
      p.tiles_i = ti + extra;
      p.tiles_j = tj;
      p.splits = parts.splits;
    }
  }
  return p;
}

// ---- 8-bit products ----------------------------------------------------------------------------

constexpr int64_t kFp8Block = 128;   // elements of the sum with a scale of their own
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// A step is a block of the sum.  22 calls of one to four rounds at each size and count of parts: the rule takes the
// fastest or is within 1% of it but for two, 7 and 8% behind, where three or six parts would be best.  Measured for
// [I, J, K], in a graph, 256x256 / 256x128 / 128x128 (parts of the sum):
//   [ 1021, 1000, 2048]  24.9 / 20.7 / 14.3              [ 4096, 4096, 4096]  58.7 / 78.1 / 93.3
//   [  968, 2048,16384]  47.7 (8) / 48.2 (4) / 52.2 (2)   [16384, 2048, 2048]  68.0 / 90.8 / 108
//   [ 2048, 4096, 4096]  44.2 / 41.4 / 49.2              [ 6000, 4096, 2048]  58.0 / 65.9 / 79.4
//   [   16, 2048, 2048]  24.1 / 19.4 / 13.1, 128x128 in 2 / 4 / 8 parts 11.1 / 9.7 / 9.7
constexpr TileShape kFp8Shape[4] = {{2, 4, 8, 4, 2}, {4, 2, 4, 4, 3}, {2, 4, 4, 2, 3}, {1, 4, 2, 2, 4}};
constexpr ProductCost kFp8Cost = {{1.40, 1.04, 0.62}, {1.12, 0.98, 0.58}, {7.6, 5.2, 4.8}, {1.0, 1.0, 1.0}, {1.0, 1.0, 1.0},
                                  4.0, 6.5, 512};

inline ProductPlan plan_fp8(int64_t I, int64_t J, int64_t K, int64_t groups, bool grouped) {
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
    const Parts parts = best_parts(kFp8Cost, kind, tiles, K, blocks, I * J, grouped, false);
    if (best == 0.0 || parts.us < best) {
      best = parts.us;
      p.kind = kind;
      p.tiles_i = ti + (grouped ? groups + 1 : 0);
      p.tiles_j = tj;
      p.splits = parts.splits;
    }
  }
  return p;
}

}  // namespace glu
