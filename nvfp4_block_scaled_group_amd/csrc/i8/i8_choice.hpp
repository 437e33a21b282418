// i8_choice.hpp -- which tiles a product in 8-bit integers takes (host code): a
// model of its time over sizes and routing.
#pragma once
#include <algorithm>
#include <cmath>

#include "i8_common.hpp"

namespace i8 {

enum Epilogue { kOutF32, kOutBf16, kGluSilu, kGluGelu, kParts };
constexpr bool is_glu(Epilogue e) { return e == kGluSilu || e == kGluGelu; }

// Row tiles of BM rows that the routing can need at most.
template <int BM>
inline int64_t row_tiles(const Routing& R, bool dense, int64_t rows) {
  if (dense) return (rows + BM - 1) / BM;
  if (BM <= kTileRows) return rows / BM;
  if (R.d_offs) return std::min<int64_t>(rows / kTileRows, rows / BM + R.num_experts);
  int64_t t = 0;
  for (int e = 0; e < R.num_experts; ++e) t += (R.h_offs[e] - (e ? R.h_offs[e - 1] : 0) + BM - 1) / BM;
  return t;
}

// The tiles a call can take.  Big: 256 x 256, one work-group on a CU.  Mid: 128
// x 128, two of them.  Mid4: 128 x 128 with four stages, one on a CU: for grids
// that do not fill the CUs twice, where a step takes as long as its copies.
constexpr int kMaxParts = 16;
constexpr int64_t kMaxWorkspace = 32 << 20;

// Row tiles of 256 that a call is likely to need, whole ones and those that an
// expert's last 128 rows leave half empty, and the experts that have rows.  The
// host does not know the rows of device routing: half of the experts end so.
struct RowCount {
  double whole, half, experts;
};
inline RowCount row_count(const Routing& R, bool dense, int64_t rows) {
  if (dense) return {(double)((rows + 255) / 256), 0.0, 1.0};
  if (R.d_offs) {
    const double groups = (double)(rows / kTileRows), e = std::min<double>(R.num_experts, groups);
    return {(groups - 0.5 * e) / 2, 0.5 * e, e};
  }
  RowCount c{0.0, 0.0, 0.0};
  for (int e = 0; e < R.num_experts; ++e) {
    const int64_t m = R.h_offs[e] - (e ? R.h_offs[e - 1] : 0);
    c.whole += (double)(m / 256);
    c.half += m % 256 ? 1 : 0;
    c.experts += m ? 1 : 0;
  }
  return c;
}

// Time in us: rounds of work-groups, each a fixed part (start, epilogue) and
// its steps.  Measured (8192 x 8192 x 8192: Big 450, Mid 543, Mid4 604; 512 x
// 7168 x 7168: 67, 50, 43; 128 rows of it: 54, 40, 27; 32768 rows of 64
// experts, 2048 x 7168, fp32: 656, 756, 896; 18560 rows, 448 x 2 x 512: 28, 25).
// A step of a grid that fills the CUs takes longer where few row tiles share an
// expert's weights, which come from memory (gated block 7168 x 2 x 2048, 128 rows
// of each of 32 experts: 214, 195, 203; 256 rows: 261, 336, 349; 512: 449, 586, 635;
// 384: 391, 452, 489; 8192 rows at random among 64: 443, 360, 367).
struct Choice {
  int shape;  // 0 Big, 1 Mid, 2 Mid4
  int parts;
  int64_t per;  // steps of a part
};
template <Epilogue EPI>
Choice choose(int64_t rows, int64_t n, int64_t k, const Routing& R, bool dense, int64_t workspace) {
  constexpr int kDiv = is_glu(EPI) ? 2 : 1;
  auto cols = [&](int bn) { return (n + bn / kDiv - 1) / (bn / kDiv); };
  const int64_t steps = (k + 127) / 128, mid = row_tiles<128>(R, dense, rows) * cols(128);
  const RowCount count = row_count(R, dense, rows);
  const double fixed = EPI == kOutF32 ? 6.5 : 5, big = (count.whole + count.half) * cols(256);
  // what a step takes longer by: `alone` us where nothing is shared and the grid is full
  auto unshared = [&](double alone, double tiles_of_all, double fill) {
    return dense ? 0.0 : alone * count.experts / tiles_of_all * std::min(1.0, fill);
  };
  auto rounds = [](double tiles, int slots) { return std::ceil(tiles / slots); };
  // a half empty tile takes 0.68 of a whole one, and mixed ones end unevenly
  const double mixed = (count.whole + 0.68 * count.half) * cols(256) / kCus + 0.7;
  Choice c{0, 1, steps};
  double best = (count.half > 0 ? std::max(1.0, std::min(rounds(big, kCus), mixed)) : rounds(big, kCus)) *
                (6.5 + (1.75 + unshared(0.45, count.whole + count.half, big / kCus)) * steps);
  auto take = [&](double t, const Choice& o) {
    if (t < best) best = t, c = o;
  };
  // a last round with one work-group on a CU at most takes 0.7 of a full one
  const int64_t rest = mid % (2 * kCus);
  const double row128 = (double)row_tiles<128>(R, dense, rows);
  take((mid / (2 * kCus) + (rest == 0 ? 0.0 : rest <= kCus ? 0.7 : 1.0)) *
           (fixed + (1.06 + unshared(0.6, row128, mid / (2.0 * kCus))) * steps),
       Choice{1, 1, steps});
  auto mid4 = [&](int64_t wgs, int64_t per) {
    const double fill = wgs / (double)kCus;
    return rounds((double)wgs, kCus) * (fixed + (0.43 + 0.12 * std::min(1.0, fill) + unshared(0.27, row128, fill)) * per);
  };
  take(mid4(mid, steps), Choice{2, 1, steps});
  // parts of the contraction, joined by a second launch
  for (int p = 2; p <= kMaxParts && dense; ++p) {
    const int64_t per = (steps + p - 1) / p;
    if (per * (p - 1) >= steps || mid * p > kCus || p * rows * n * 4 > workspace) continue;
    take(mid4(mid * p, per) + 4 + 8e-6 * p * rows * n / 4, Choice{2, p, per});
  }
  return c;
}

}  // namespace i8
