// What a matrix product reads and how it is cut into tiles, by sizes and types:
// plain arithmetic, without the device.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/shardconv.h"

namespace st {

// Bytes that may be read from the first of `rows` rows' scale bytes on, `stride`
// apart, of `blocks` blocks each: behind the last row's words there need not be
// anything (columns of a wider buffer end with it).  Words: scales lie on a grid of
// four bytes, so that the last one's rest is in the same page.
constexpr int scale_span(int rows, int stride, int blocks) { return (rows - 1) * stride + (blocks + 3) / 4 * 4; }

// Contraction steps of a stage: 128 bytes of either operand
inline int stage_steps(int type) { return type == ST_F32 ? 32 : type == ST_BF16 ? 64 : 128; }

struct Shape {                        // tile and what a compute unit holds of it
  int ta, tb, per_cu;
};
// large, middle and small tile.  fp32 (products a ninth as fast, twice the registers per
// fragment) has 128 x 128 for a large one, taken for long contractions alone and there
// with split sums, never with whole ones: weight gradients of many rows (55053 rows,
// 1818 to 1494 channels: 2655 us, with the smaller tiles 3010; 124716 rows, 4312 to
// 1530: 13.5 ms, 14.7).
// (8-bit operands: two of the 128 x 64 tiles fit a compute unit's LDS, not three; the
// third of the workgroups start when others have ended.)
constexpr Shape kShapes[2][3] = {{{256, 256, 1}, {128, 64, 3}, {64, 64, 4}}, {{128, 128, 2}, {128, 64, 3}, {64, 64, 4}}};
inline const Shape& shape_of(int type, int s) { return kShapes[type == ST_F32][s]; }
constexpr int kFewShape = 3;
constexpr int kCus = 256;

struct Choice {
  int shape, splits, per_split;
};
constexpr int kFewRows = 64;
constexpr int kFewWaves = 8;            // waves of a workgroup of few rows

// What the choice between shapes and splits goes by, in microseconds, fitted to
// measured products (96 x 2048 x 8192 to 458752 x 64 x 256, within a fifth of most):
// a stage of one tile alone on a compute unit, a tile's share of a busy one, and
// a tile's start and end.
struct Pace {
  double alone, busy, ends;
};
constexpr Pace kPace[2][3] = {{{1.0, 1.45, 7.0}, {0.48, 0.33, 3.0}, {0.42, 0.22, 2.0}}, {{2.0, 2.0, 7.0}, {1.0, 1.0, 3.0}, {0.55, 0.5, 2.0}}};

// Tile shape and split of the contraction: the least time of the fullest compute
// unit, with the partial sums' way through memory (7 TB/s, 5 us for the join).
// exact: 8-bit operands with an output that is no bf16, which the middle tile alone has:
// its paces are the 8-bit instructions', of which the widened products take almost three
// times as long (16384 x 2048 x 8192: 1076 us, by the paces 404).  cols: the weights are
// read across their rows.
inline Choice choose(int64_t m, int64_t n, int64_t k, int type, bool exact, bool cols) {
  const int kt = stage_steps(type);
  const int64_t stages = (k + kt - 1) / kt;
  if (m <= kFewRows && !cols) {
    // splits where the channels leave compute units idle, of two units a wave at least
    const int64_t blocks = (n + 31) / 32;
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(kCus / blocks, stages / (2 * kFewWaves)));
    const int64_t per = (stages + splits - 1) / splits;
    return Choice{kFewShape, (int)((stages + per - 1) / per), (int)per};
  }
  Choice best{};
  double least = INFINITY;
  for (int s = exact ? 1 : 0; s < (exact ? 2 : 3); ++s) {
    const Shape& h = shape_of(type, s);
    const Pace& p = kPace[type == ST_F32][s];
    const int64_t tiles = (n + h.ta - 1) / h.ta * ((m + h.tb - 1) / h.tb);
    for (int64_t splits = 1; splits <= 512 && splits <= stages; splits = splits < 8 ? splits + 1 : splits * 9 / 8) {
      int64_t per = (stages + splits - 1) / splits;
      if (type == ST_MX8) per = (per + 3) / 4 * 4;       // (scale bytes come for four stages)
      if ((stages + per - 1) / per != splits) continue;
      const double all = (double)tiles * splits, fill = std::min(1.0, all / kCus);
      const int64_t on = (tiles * splits + kCus - 1) / kCus;                 // tiles of the fullest unit
      const double stage = s == 0 && type != ST_F32 ? p.alone + (p.busy - p.alone) * fill : p.busy;
      double t = on <= h.per_cu ? per * std::max(p.alone, on * stage) + p.ends
                                : on * per * stage + (on + h.per_cu - 1) / h.per_cu * p.ends;
      if (splits > 1) t += 5.0 + (double)m * n * splits * 8 / 7.0e6;
      if (t < least) { least = t; best = Choice{s, (int)splits, (int)per}; }
      if (tiles * splits > 8 * kCus) break;
    }
  }
  return best;
}

}  // namespace st
