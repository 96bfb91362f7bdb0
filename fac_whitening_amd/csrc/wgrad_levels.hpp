// How the products (k_wgrad.hip, k_product.hip) share their output tiles among
// workgroups.  Plain integer arithmetic, the same on the host, which sizes the
// workspace by it, and on the device.
#pragma once
#include <stdint.h>

namespace gift {

// How G workgroups share R tiles of n units each: in levels, each a set of
// pieces of one length that start at one place of the token axis, so that
// workgroups on one die walk the same tokens at the same time and share them
// through its L2.  With C = ceil(R n / G) units for every workgroup:
//   n >= C: q = n / C workgroups a tile take C units each and are done
//   n <  C: every workgroup takes all n units of C / n tiles
// and what is left of tiles, units, workgroups and C goes through the same
// step again (the Euclidean algorithm on n and C).  Pieces of a level are
// numbered from `base`; piece 0 .. R - 1 of a level is that of its tile.
// Whole tiles have no pieces and take no numbers.
struct WLevel {
  int R, n, W, C;      // tiles, units left of each, workgroups, units left for each
  int from;            // first unit of the pieces
  int tile0;           // first tile
  int base;            // number of the level's first piece
  __host__ __device__ bool done() const { return R == 0 || n == 0; }
  __host__ __device__ bool split() const { return n >= C; }            // pieces of C units, count() a tile
  __host__ __device__ int count() const { return split() ? n / C : C / n; }
  __host__ __device__ int tiles() const {                              // tiles that are finished at this level
    const int64_t t = split() ? R : (int64_t)count() * W;
    return t < R ? (int)t : R;
  }
  __host__ __device__ void next() {
    if (split()) {
      const int q = n / C;
      base += q * R;
      W -= q * R;
      from += q * C;
      n -= q * C;
    } else {
      const int t = tiles();
      if (from > 0) base += t;   // (from == 0: whole tiles)
      C -= count() * n;
      R -= t;
      tile0 += t;
    }
  }
};

// The first level.  Pieces of whole tiles are written to W directly and have
// no number.
__host__ __device__ inline WLevel wgrad_levels(int tiles, int units, int G) {
  WLevel v{};
  v.R = tiles;
  v.n = units;
  v.W = G;
  v.C = (int)(((int64_t)tiles * units + G - 1) / G);
  return v;
}

// Calls piece(tile, first unit, units, number) for the pieces of workgroup g,
// in order.  (The lane-independent values are wave-uniform; `uniform` tells a
// device compiler so.)
template <typename U, typename F>
__host__ __device__ inline void wgrad_walk(WLevel v, int g, U&& uniform, F&& piece) {
  int k = 0;
  while (!v.done()) {
    int tile, from = v.from, units = v.n, number;
    if (v.split()) {
      const int mine = v.count() * v.R;
      if (g >= mine) {
        g -= mine;
        v.next();
        continue;
      }
      const int c = g / v.R;
      tile = g - c * v.R;
      from += c * v.C;
      units = v.C;
      number = v.base + g;
      v.R = 0;   // the last piece
    } else {
      tile = g + k * v.W;
      number = v.base + tile;
      if (k == v.count() || tile >= v.R) {
        k = 0;
        v.next();
        continue;
      }
      ++k;
    }
    piece(uniform(v.tile0 + tile), uniform(from), uniform(units), uniform(number));
  }
}

// Piece p of workgroup g, the p-th that wgrad_walk calls for; false past the
// last.  (For a kernel that asks for one piece at a time.)
__host__ __device__ inline bool wgrad_piece(WLevel v, int g, int p, int& tile, int& from, int& units, int& number) {
  for (; !v.done(); v.next()) {
    from = v.from;
    if (v.split()) {
      const int mine = v.count() * v.R;
      if (g >= mine) {
        g -= mine;
        continue;
      }
      if (p > 0) return false;
      const int c = g / v.R;
      tile = v.tile0 + g - c * v.R;
      from += c * v.C;
      units = v.C;
      number = v.base + g;
    } else {
      const int n = g >= v.R ? 0 : (v.R - g + v.W - 1) / v.W;      // of this level's tiles
      const int mine = n < v.count() ? n : v.count();
      if (p >= mine) {
        p -= mine;
        continue;
      }
      tile = v.tile0 + g + p * v.W;
      units = v.n;
      number = v.base + g + p * v.W;
    }
    return true;
  }
  return false;
}

// Calls add(number, stride, count) for each level's numbered pieces of a split
// tile, in token order: number, number + stride, ...
template <typename F>
__host__ __device__ inline void wgrad_pieces(WLevel v, int tile, F&& add) {
  for (; !v.done(); v.next()) {
    const int r = tile - v.tile0;
    const int count = v.split() ? v.count() : v.from > 0 && r < v.tiles() ? 1 : 0;
    if (count) add(v.base + r, v.R, count);
    if (!v.split() && r < v.tiles()) break;
  }
}

// What the host needs: the first split tile, how many there are, and the
// pieces to keep.
struct WSplit {
  int first, tiles, pieces;
};
inline WSplit wgrad_split(WLevel v) {
  WSplit s{0, 0, 0};
  if (!v.split()) v.next();   // whole tiles
  s.first = v.tile0;
  s.tiles = v.from == 0 && v.n == v.C ? 0 : v.R;
  for (; !v.done(); v.next()) s.pieces = v.base + (v.split() ? v.count() * v.R : v.tiles());
  if (s.tiles == 0) s.pieces = 0;
  return s;
}

}  // namespace gift
