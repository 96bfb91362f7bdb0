// The numbers that the pieces of split tiles get are exactly 0 .. pieces - 1
// for every division that the weight-gradient product may take: the
// workspace holds a place for each number, so one that no piece has would be
// memory that is asked for and counted, and never written.  Prints
// "ok <divisions>" or the first fault.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "wgrad_levels.hpp"

using namespace gift;

static bool check(int tiles, int units, int G) {
  const WLevel v = wgrad_levels(tiles, units, G);
  const WSplit s = wgrad_split(v);
  std::set<int> numbers;
  for (int g = 0; g < G; ++g)
    wgrad_walk(v, g, [](int x) { return x; }, [&](int, int from, int n, int number) {
      if (from != 0 || n != units) numbers.insert(number);
    });
  if ((int)numbers.size() == s.pieces && (numbers.empty() || (*numbers.begin() == 0 && *numbers.rbegin() == s.pieces - 1)))
    return true;
  std::printf("fault: %d tiles of %d units over %d workgroups: %d places, %d pieces\n", tiles, units, G, s.pieces,
              (int)numbers.size());
  return false;
}

int main() {
  long n = 0;
  for (int tiles = 1; tiles <= 40; ++tiles)
    for (int units = 1; units <= 24; ++units)
      for (int G : {1, 2, 3, 7, 8, 16, 31}) {
        if (!check(tiles, units, G)) return 1;
        ++n;
      }
  if (!check(304, 256, 256) || !check(1100, 17, 512)) return 1;
  std::srand(11);
  for (int i = 0; i < 3000; ++i) {
    if (!check(1 + std::rand() % 1200, 1 + std::rand() % 140, i % 2 ? 256 : 512)) return 1;
    ++n;
  }
  std::printf("ok %ld\n", n);
}
