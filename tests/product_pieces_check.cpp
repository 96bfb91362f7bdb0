// wgrad_piece, which a kernel asks for one piece at a time, against
// wgrad_walk, over the divisions that the products may take.  Prints "ok
// <divisions>" or the first fault.
#include <array>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "product_plan.hpp"

using namespace gift;

static bool check(int tiles, int units, int G) {
  const WLevel v = wgrad_levels(tiles, units, G);
  for (int g = 0; g < G; ++g) {
    std::vector<std::array<int, 4>> walk, got;
    wgrad_walk(v, g, [](int x) { return x; }, [&](int tile, int from, int n, int number) {
      // (whole tiles have no number)
      walk.push_back({tile, from, n, from == 0 && n == units ? -1 : number});
    });
    std::array<int, 4> p{};
    while (wgrad_piece(v, g, (int)got.size(), p[0], p[1], p[2], p[3])) {
      if (p[1] == 0 && p[2] == units) p[3] = -1;
      got.push_back(p);
      if (got.size() > walk.size()) break;
    }
    // and none after the last, whichever is asked for
    bool good = got == walk;
    for (int k = 0; k < 3; ++k) good = good && !wgrad_piece(v, g, (int)walk.size() + k, p[0], p[1], p[2], p[3]);
    if (!good) {
      std::printf("fault: %d tiles of %d units over %d workgroups, workgroup %d\n", tiles, units, G, g);
      return false;
    }
  }
  return true;
}

// The division that the plan of a product takes.
static bool planned(int epi, int64_t M, int64_t N, int64_t K, int nseg) {
  const ProdPlan p = product_plan(epi, epi != kEpiGlu, epi == kEpiGrad, M, N, K, nseg);
  return check(p.nbm * p.nbn, (int)ceil_div(p.nst * nseg, p.unit), p.grid);
}

int main() {
  long n = 0;
  for (int tiles = 1; tiles <= 40; ++tiles)
    for (int units = 1; units <= 24; ++units)
      for (int G : {1, 2, 3, 7, 8, 16, 31}) {
        if (!check(tiles, units, G)) return 1;
        ++n;
      }
  std::srand(23);
  for (int i = 0; i < 1500; ++i) {
    if (!check(1 + std::rand() % 1200, 1 + std::rand() % 140, i % 2 ? 256 : 512)) return 1;
    ++n;
  }
  for (int i = 0; i < 1500; ++i) {
    const int epi = i % 3;
    const int64_t M = 1 + std::rand() % 6000, N = 1 + std::rand() % 6000, K = 1 + std::rand() % 6000;
    if (!planned(epi, M, N, K, (epi == kEpiStore ? 2 : 1) * (i / 3 % 2 ? 6 : 1))) return 1;
    ++n;
  }
  std::printf("ok %ld\n", n);
}
