// Every division of tiles among workgroups that the weight-gradient product
// may take, walked on the host: each unit of each tile belongs to exactly one
// piece, no workgroup has more than its share, piece numbers are unique and
// inside what the workspace holds, and the join adds a tile's pieces in token
// order.  Prints "ok <divisions>" or the first fault.
#include <algorithm>
#include <array>
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "wgrad_levels.hpp"

using namespace gift;

static bool check(int tiles, int units, int G) {
  std::vector<int> cover((size_t)tiles * units, 0);
  std::vector<std::vector<std::array<int, 3>>> of(tiles);
  std::set<int> numbers;
  const WLevel v = wgrad_levels(tiles, units, G);
  const WSplit s = wgrad_split(v);
  bool good = true;
  for (int g = 0; g < G; ++g) {
    int load = 0;
    wgrad_walk(v, g, [](int x) { return x; }, [&](int tile, int from, int n, int number) {
      if (tile < 0 || tile >= tiles || from < 0 || n < 1 || from + n > units) {
        good = false;
        return;
      }
      load += n;
      for (int u = from; u < from + n; ++u) ++cover[(size_t)tile * units + u];
      if (from == 0 && n == units) return;
      good = good && numbers.insert(number).second && number >= 0 && number < s.pieces;
      good = good && tile >= s.first && tile < s.first + s.tiles;
      of[tile].push_back({from, n, number});
    });
    good = good && load <= v.C;
  }
  for (int c : cover) good = good && c == 1;
  for (int t = 0; t < tiles && good; ++t) {
    std::sort(of[t].begin(), of[t].end());
    std::vector<int> want, got;
    for (auto& p : of[t]) want.push_back(p[2]);
    if (t >= s.first && t < s.first + s.tiles) wgrad_pieces(v, t, [&](int number, int stride, int count) {
      for (int c = 0; c < count; ++c) got.push_back(number + c * stride);
    });
    good = got == want;
  }
  if (!good) std::printf("fault: %d tiles of %d units over %d workgroups\n", tiles, units, G);
  return good;
}

int main() {
  long n = 0;
  for (int tiles = 1; tiles <= 40; ++tiles)
    for (int units = 1; units <= 24; ++units)
      for (int G : {1, 2, 3, 7, 8, 16, 31}) {
        if (!check(tiles, units, G)) return 1;
        ++n;
      }
  std::srand(5);
  for (int i = 0; i < 3000; ++i) {
    if (!check(1 + std::rand() % 1200, 1 + std::rand() % 140, i % 2 ? 256 : 512)) return 1;
    ++n;
  }
  std::printf("ok %ld\n", n);
}
