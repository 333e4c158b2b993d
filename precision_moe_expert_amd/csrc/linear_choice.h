// Which kernel a product of the dense FP8 projection runs: host arithmetic on sizes
// alone.
#pragma once
#include <cstddef>
#include <cstdint>

namespace moe {

struct LinChoice {
  int shape, splits, halved;  // of kLinShapes or LIN_BATCH; ways K is split; last tiles that are done as two halves
};

// Tiles of a product, and what they cost (cycles of a CU, measured at 8192 x
// 7168 x 4096 and smaller calls): a K block of one tile, the rest of a tile; `per`
// workgroups share a CU.
struct LinShape {
  int bm, bn, per;
  float step, rest;
};
constexpr LinShape kLinShapes[] = {
    {256, 256, 1, 2500, 9000}, {128, 256, 1, 1400, 6000}, {128, 128, 2, 1700, 5000}, {64, 128, 2, 1000, 4000},
    {32, 128, 2, 900, 4000},  {32, 64, 2, 600, 4000}};
constexpr int kLinShapeCount = 6;
constexpr int kLinVecShapes = 5;  // without groups, for scales per row on both sides
constexpr int kLinCus = 256;

inline size_t lin_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int lin_tiles(int64_t m, int64_t n, const LinShape& s) {
  return (int)((m + s.bm - 1) / s.bm * ((n + s.bn - 1) / s.bn));
}

// The tile and the ways K is split for a product: the least of what the rounds
// of workgroups cost, and of writing and joining the parts (fp32) where K is
// split.  A last round of 256 x 256 tiles that would leave half of the CUs idle is
// done in halves.
inline LinChoice lin_choose(int64_t m, int64_t n, int kt, bool vec) {
  LinChoice best{0, 1, 0};
  float least = 0.0f;
  for (int i = 0; i < (vec ? kLinVecShapes : kLinShapeCount); ++i) {
    const LinShape& s = kLinShapes[i];
    const int tiles = lin_tiles(m, n, s), slots = kLinCus * s.per;
    for (int sp = 1; sp <= 16 && (sp == 1 || kt / sp >= 2); ++sp) {
      const float join = sp == 1 ? 0.0f : 6000.0f + (float)((double)sp * m * n * 8 / 2000.0);  // about 4 TB/s at 2 GHz
      if (sp > 1 && join >= least) break;
      if (sp > 1 && ((int64_t)sp * m * n * 4 > (64 << 20) || (int64_t)tiles * (sp - 1) >= 2 * slots)) break;
      const int64_t wgs = (int64_t)tiles * sp, full = wgs / slots;
      const int rem = (int)(wgs - full * slots);
      const float one = (float)((kt + sp - 1) / sp) * s.step + s.rest;
      const bool half = i == 0 && sp == 1 && rem > 0 && rem * 2 <= slots;
      // a round that leaves CUs to one workgroup instead of two costs less
      const float last = rem == 0 ? 0.0f : half ? 0.6f * one : s.per == 2 && rem * 2 <= slots ? 0.7f * one : one;
      const float cost = (float)full * one + last + join;
      if (i == 0 && sp == 1 ? true : cost < least) {
        least = cost;
        best = LinChoice{i, sp, half ? rem : 0};
      }
    }
  }
  return best;
}

// Whether a product of quantized rows is k_lin_batch's, on top of lin_is_few's (16 rows
// 2048 x 7168 8.9 us, in tiles 10.5; 7168 x 4096 13.8 and 16.9; 32 rows 4096 x 2048
// 11.6 and 13.3, 1024 x 1024 6.4 and 8.1; 7168 x 576 15.2 and 13.4: long rows of
// codes come from the L2 again for every 16 columns).
constexpr int LIN_BATCH = kLinShapeCount;  // of LinChoice
inline bool lin_is_batch(int64_t m, int kt) { return m <= 16 || (m <= 32 && kt <= 32); }
// 32 columns per workgroup where 16 would make more than one per CU.
inline int lin_batch_cols(int64_t n) { return n <= 16 * kLinCus ? 1 : 2; }

// Whether a product is k_lin_few's, which quantizes the rows in every workgroup and so
// pays for few and short ones (10 rows 2048 x 7168 9.1 us, with a launch that
// quantizes them first 9.1, 12 rows 10.1 and 9.2; 4 and 8 rows 4096 x 2048 7.1 and 8.2,
// 9.6 and 8.6; 3 and 6 rows 7168 x 4096 10.9 and 12.3, 12.5 and 11.8).
inline int lin_few_waves(int kt) { return kt > 32 ? 16 : 8; }
inline bool lin_is_few(int64_t m, int kt) {
  return m <= 16 && (m == 1 ? kt * 132 + 16384 <= 65536 : m * kt <= 176);
}

// Whether both gradients' products go into one launch, given their choices.
inline bool lin_joined(const LinChoice& dx, const LinChoice& dw) {
  return dx.shape == 0 && dx.splits == 1 && dw.shape == 0 && dw.splits == 1;
}
// Of such a launch with na tiles of ka K blocks and then nb of kb, kb <= ka: the last round of
// the shorter tiles, in halves if it would leave half of the CUs idle.
inline int lin_joined_halves(int na, int ka, int nb, int kb) {
  const int rem = (int)(((int64_t)na * ka / kb + nb) % kLinCus);
  return rem * 2 <= kLinCus && rem <= nb ? rem : 0;
}

}  // namespace moe
