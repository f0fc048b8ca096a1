// How the feed-forward's products are laid out, tiled, split and paced: plain
// host C++, so that it can be compiled and checked without a device.
#pragma once

#include <stdint.h>

#include <cmath>
#include <initializer_list>

namespace rnnk {

// A product's output is [M, N]; its operands are given by rows of the summed
// dimension's neighbours ("along": [M, K]) or by rows of the outputs'
// neighbours ("across": [K, M]).
enum FeedOp { kFeedIn, kFeedOut, kFeedDh, kFeedDx, kFeedDwIn, kFeedDwOut, kFeedOps };
// Tile and split of one product.
enum FeedTileKind { kTileSmall, kTileBig, kTileDeep };  // 128 x 128, 256 x 256, 128 x 128 with more loads in flight
struct FeedPlan {
  int tile;
  int splits;
};

inline double feed_tiles(const FeedPlan& p, int64_t M, int64_t N, int op) {
  const double rows = p.tile == kTileBig ? 256 : 128, cols = op == kFeedIn ? rows / 2 : rows;
  return std::ceil((double)M / rows) * std::ceil((double)N / cols);
}

// The tile and the split with the shortest expected time: rounds of the
// workgroups that the device holds, times steps, plus the results' way out and
// the partial products' way through memory. dh reads and writes 16 bytes
// a result there (fp32; 12 in bf16), which two workgroups a compute unit hide
// better than one: 32000 x 2816 bf16 422 us in small tiles and 450 in large
// ones, 19334 x 1368 fp32 356 (now 339) and 501; without that traffic large ones
// win (dx of the same in bf16: 411 us, 480 in small ones). The constants are fitted to such
// pairs: a step and a tile's results for each tile, 8 us for the launch that
// adds up and 4 MB/us for the partial products (2 rows, 1424 x 2456 fp32
// training: 286 us with the first products undivided, 141 divided; 799 rows,
// 1032 x 624: 304 and 199). Of all tiles and divisions by up to 16, tried one
// product at a time in fp32 training, the best were 0 to 12% of the whole pass
// faster than the plan's (1361 rows, 1376 x 268: 2%; 400 rows, 1024 x 2816: 3%;
// 700 rows, 534 x 6864: 9%; 3306 rows, 1168 x 160: 12%).
inline FeedPlan feed_plan(int op, int64_t M, int64_t N, int steps, bool bf16_storage, int cus) {
  FeedPlan best{kTileSmall, 1};
  double least = 0.0;
  for (int tile : {kTileSmall, kTileBig, kTileDeep}) {
    FeedPlan p{tile, 1};
    const bool big = tile == kTileBig;
    const double tiles = feed_tiles(p, M, N, op), resident = tile == kTileSmall ? 2.0 * cus : cus;
    // us of a step, with all workgroups that the device holds at work, and of a tile's results
    const double step = bf16_storage ? (big ? 2.0 : tile == kTileDeep ? 0.8 : 1.3) : (big ? 7.6 : tile == kTileDeep ? 2.6 : 3.9);
    const double results = big ? (op == kFeedDh ? 90.0 : 12.0) : 6.0;
    for (int want = 1; want <= 32 && want <= steps; ++want) {
      const int each = (steps + want - 1) / want;
      p.splits = (steps + each - 1) / each;
      if (p.splits != want) continue;
      double us = std::ceil(tiles * want / resident) * (each * step + results);
      if (want > 1) us += 8.0 + (double)want * M * N * (op == kFeedIn ? 16.0 : 8.0) / 4e6;
      if (least == 0.0 || us < least) {
        least = us;
        best = p;
      }
    }
  }
  return best;
}

constexpr int kFeedFewRows = 64;

// The widths as the products see them, and their plans.
struct FeedSizes {
  int64_t m, rows;     // elements of 16 bytes
  int N, F, N_out;
  int Np, Fm, Op, Fp;  // N, F and N_out in whole 16 bytes; F in whole steps of 128 bytes
  FeedSizes(bool bf16_storage, int64_t rows_, int N_, int F_, int N_out_) : m(bf16_storage ? 8 : 4), rows(rows_), N(N_), F(F_), N_out(N_out_) {
    auto up = [](int64_t v, int64_t to) { return (int)((v + to - 1) / to * to); };
    Np = up(N, m);
    Fm = up(F, m);
    Op = up(N_out, m);
    Fp = up(F, 8 * m);
  }
  // Serving takes the few-row kernels up to 64 rows. So does training forward,
  // but with more than 32 rows for weights up to 2^23 numbers each: 64 rows, 1024
  // x 2816, bf16, with the backward pass 79 us in tiles and 69 so, 2048 x 4096 101
  // and 98, 2048 x 5632 116 and 126; 32 rows, 2048 x 8192, 140 and 135, fp32 329
  // and 290.
  bool few(bool train) const {
    if (rows > kFeedFewRows) return false;
    return !train || rows <= 32 || (int64_t)(N > N_out ? N : N_out) * F <= 1 << 23;
  }
  int steps(int64_t k) const { return (int)((k + 8 * m - 1) / (8 * m)); }
  FeedPlan plan(int op, int cus) const {
    const bool bf = m == 8;
    switch (op) {
      case kFeedIn: return feed_plan(op, rows, Fp, steps(Np), bf, cus);
      case kFeedOut: return feed_plan(op, rows, N_out, steps(Fm), bf, cus);
      case kFeedDh: return feed_plan(op, rows, Fp, steps(Op), bf, cus);
      case kFeedDx: return feed_plan(op, rows, N, steps(2 * (int64_t)Fp), bf, cus);
      case kFeedDwIn: return feed_plan(op, 2 * (int64_t)Fp, N, steps(rows), bf, cus);
      default: return feed_plan(op, N_out, F, steps(rows), bf, cus);
    }
  }
};

// Loads that may be on their way where a step t ends (in units of one
// operand's step): those that are newer than what step t + 1 takes. A
// workgroup's loads are issued in the order A 0, B 0, A 1, B 1, ..., over all
// its tiles; with step t go B t + ahead - 1 and A t + ahead, as long as there
// are steps left (more_b, more_a). `whole`: both went from memory straight into
// LDS; what goes through registers has waited for all that was older. `left`:
// steps of this tile behind t, at most as many as the workgroup has left.
constexpr int feed_later(int ahead, bool more_a, bool more_b, bool whole, int left) {
  return !whole            ? 0
         : more_a          ? 2 * ahead - 3
         : more_b          ? 2 * ahead - 4   // the last B: A t + 2, B t + 2 up to A and B t + ahead - 1
         : left > 1        ? 2 * (left - 1)  // nothing more: A t + 2 up to B t + left
                           : 0;
}

}  // namespace rnnk
