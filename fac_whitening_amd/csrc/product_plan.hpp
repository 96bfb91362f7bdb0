// Which form a call of the gated block or of the weight gradient takes, and
// how a product's tiles are shared out.  Plain arithmetic on the host.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/gift.h"
#include "wgrad_levels.hpp"

namespace gift {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether k_glu_tokens makes the block's output: up to 32 rows of x, and up to 64 where the weights are small (tokens
// against tiles, 64 rows bf16: 1536 x 6144 22 and 23 us, 4096 x 16384 111 and 68) or fp32, whose tiles need their
// operands laid out anew (1536 x 6144: 45 and 86; the limit of 2^24 weights lies between the two shapes).
inline bool glu_by_tokens(int dtype, int64_t T, int d, int f) {
  return T <= 32 || (T <= 64 && (dtype == GIFT_FP32 || (int64_t)d * f <= (int64_t)1 << 24));
}
// Hidden units of one of its workgroups, in sixteens: 32 read x half as often.  4096 x 16384 bf16, 16 units against 32:
// 1 token 52 and 57 us, 16 tokens 65 and 61, 32 tokens 79 and 69; with fewer than two workgroups a compute unit the
// smaller ones are quicker.
inline int glu_token_units(int dtype, int64_t T, int f) {
  return dtype != GIFT_FP32 && T > 8 && T <= 32 && ceil_div(f, 32) >= 512 ? 2 : 1;
}
// Whether the tokens' backward form makes dx: few rows, and no output over what it reads again.  (It is
// built for two sets of 16 tokens in 16 bits and for one in fp32.  The tiles behind it, 33 rows bf16 against 32: 1536 x 6144
// 33 and 25 us, 4096 x 16384 72 and 70; fp32, 17 against 16: 88 and 33, 520 and 114.)
inline bool glu_backward_by_tokens(int dtype, int64_t T, bool in_place) {
  return T <= (dtype == GIFT_FP32 ? 16 : 32) && !in_place;
}

enum { kEpiGlu = 0, kEpiStore = 1, kEpiGrad = 2 };   // what a product's tiles become (k_product.hip)

constexpr int kProductGroups = 256;   // compute units of an MI355X

struct ProdPlan {
  int side, deep, nbm, nbn, nst, unit, grid;   // deep: four stages in LDS, one workgroup a compute unit
  int first, split;    // first split tile, split tiles
  size_t bytes;        // of the pieces
};

// A plan in one of three forms (tiles of 256, of 128 with two workgroups a
// compute unit, of 128 with one and four stages in LDS), split at multiples of
// `unit` stages (0: not split), and what it is expected to take, in us.
// Measured on bf16 (direct x direct, transposing x direct, both transposing; 1536
// x 6144 and 4096 x 4096, 128 to 8192 tokens), within a fifth or so, and taken for
// fp32 too, whose stages are the same over six times as many:
//   a stage of a workgroup   256: 1.75 each; 128: 1.0, 1.25, 1.15; deep: 0.6
//   a whole tile written     256: 6, fp32 gradients 14; 128: 2, 4
//   a split                  7 for the launch of the join, pieces written and read at 8 TB/s, outputs written at 6, and
//                            0.15 for each piece of a tile, which the join adds one after another
inline double product_try(ProdPlan& p, int side, int deep, int unit, int most, int epi, bool ax, bool bx, int64_t M, int64_t N, int64_t K, int nseg) {
  p.side = side;
  p.deep = deep;
  p.nbm = (int)ceil_div(M, epi == kEpiGlu ? side / 2 : side);
  p.nbn = (int)ceil_div(N, side);
  p.nst = (int)ceil_div(K, 64);
  p.grid = side == 128 && !deep ? 2 * kProductGroups : kProductGroups;
  const int total = p.nst * nseg;
  p.unit = unit ? unit : total;
  const int64_t tiles = (int64_t)p.nbm * p.nbn;
  if (unit && tiles * most < p.grid) p.grid = (int)tiles * most;
  const WLevel v = wgrad_levels((int)tiles, (int)ceil_div(total, p.unit), p.grid);
  const WSplit w = wgrad_split(v);
  p.first = w.first;
  p.split = w.tiles;
  p.bytes = (size_t)w.pieces * side * side * 4;
  const double stages = (double)v.C * p.unit;
  const bool large = side == 256, grad = epi == kEpiGrad;
  const double stage = large ? 1.75 : deep ? 0.6 : bx ? 1.15 : ax ? 1.25 : 1.0;
  const double whole = (double)(v.C * (int64_t)p.unit / total) * (large ? grad ? 14.0 : 6.0 : grad ? 4.0 : 2.0);
  const double join = 7.0 + 2.0 * (double)p.bytes / 8e6 + 0.15 * (double)ceil_div(p.grid, tiles) +
                      (double)p.split * side * side * (grad ? 4 : 2) / 6e6;
  return stages * stage + whole + (p.split ? join : 0.0);
}

inline ProdPlan product_plan(int epi, bool ax, bool bx, int64_t M, int64_t N, int64_t K, int nseg) {
  ProdPlan best{};
  double least = 0;
  if (K < 1) return best;
  for (int form = 0; form < 3; ++form) {   // 256, 128, 128 deep
    if (form == 2 && (ax || bx)) continue;
    for (int unit = 0; unit <= 8; unit += unit ? unit : 2)
      for (int most = 4; most <= 256; most *= 4) {   // workgroups a tile
        ProdPlan p{};
        const double t = product_try(p, form == 0 ? 256 : 128, form == 2, unit, most, epi, ax, bx, M, N, K, nseg);
        if (best.side == 0 || t < least) {
          best = p;
          least = t;
        }
        if (unit == 0) break;
      }
  }
  return best;
}

}  // namespace gift
