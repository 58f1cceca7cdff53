// The schedule of attention over shared prefixes, run on the host: units, runs, cut items, and what a row tile's tiles cover.
// Prints one line per seed: units, runs, cut items.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_shared.cuh"

using namespace qspec::att;

#define REQUIRE(x)                                  \
  do {                                              \
    if (!(x)) {                                     \
      std::printf("line %d: %s\n", __LINE__, #x);  \
      std::exit(1);                                 \
    }                                               \
  } while (0)

template <int kRows, int kKeys>
void check(int seed) {
  using W = SharedWalk<kRows, kKeys>;
  std::mt19937 r(seed);
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(r() % (hi - lo + 1)); };
  const int G = pick(1, 7), grid = pick(1, 152);
  std::vector<int2> grp(G + 1);
  std::vector<int> cu{0}, kv;
  W w{};
  w.heads = pick(1, 8);
  w.group = pick(1, 8);
  int shift = 0;
  while ((1 << shift) < w.group) ++shift;
  w.group_shift = 31 + shift;
  w.group_mul = static_cast<uint32_t>(((uint64_t(1) << w.group_shift) + w.group - 1) / w.group);
  w.window = pick(0, 2) ? 0 : pick(1, 900);
  for (int g = 0; g < G; ++g) {
    const int members = pick(0, 9), long_one = pick(0, 4) == 0;
    int p = pick(0, 3000);
    grp[g].x = static_cast<int>(kv.size());
    for (int m = 0; m < members; ++m) {
      const int n = pick(0, 3) ? pick(1, long_one ? 300 : 6) : 0;
      const int own = pick(0, 600);
      kv.push_back(n == 0 ? pick(0, 50) : pick(0, 9) ? p + n + own : pick(0, n + 5));  // (some shorter than their new tokens)
      cu.push_back(cu.back() + n);
      if (n > 0) p = std::min(p, std::max(kv.back() - n, 0));
    }
    grp[g].y = pick(0, 9) ? p : -1;
    // p may have shrunk after a longer sequence: fine, it holds for all
  }
  grp[G] = make_int2(static_cast<int>(kv.size()), -1);
  kv.push_back(0);
  w.grp = grp.data();
  w.cu = cu.data();
  w.kv = kv.data();
  w.groups = G;

  ScanShared sh{};
  for (int g = 0; g < G; ++g)
    for (int t = 0; t < 400; ++t) sh.total += w.units(g, t);
  if (sh.total == 0) return;
  sh.runs = static_cast<int>(sh.total < grid ? sh.total : grid);
  long long at = 0;
  int cut = 0, tile_after = 0;
  for (int c = 0; c < sh.runs; ++c) {
    W x = w;
    x.u = run_start(c, &sh);
    x.u1 = run_start(c + 1, &sh);
    const long long u0 = x.u, u1 = x.u1;
    x.start(0, 0, 0);
    while (x.next()) {
      const Item& it = x.it;
      const long long n = x.u - at;                       // units; tiles go on where the run before stopped
      REQUIRE(n > 0 && it.ub <= at && at + n <= it.ue && it.kt0 < it.kt1);
      REQUIRE(at == it.ub ? it.kt0 == 0 : it.kt0 == tile_after);
      tile_after = it.kt1;
      at += n;
      cut += it.ub < u0 || it.ue > u1;
      // the tiles of the item: the prefix's and each sequence's; every key that a row sees lies in one of them, once
      const int s0 = grp[it.b].x, s1 = grp[it.b + 1].x, p = grp[it.b].y;
      REQUIRE(p >= 0 && it.hi == p && it.tok0 == cu[s0] && it.rows > 0 && it.rows <= kRows);
      REQUIRE(it.kv >= s0 && it.kv < s1 && cu[it.kv + 1] > cu[it.kv] && cu[it.kv] == cu[s0]);
      const int t0 = it.tok0 + it.row0 / w.group, t1 = it.tok0 + (it.row0 + it.rows - 1) / w.group;
      int total = tiles_between<kKeys>(it.lo, p);
      for (int s = s0; s < s1; ++s) {
        const int f = std::max(cu[s], t0), l = std::min(cu[s + 1] - 1, t1);
        if (f > l) continue;
        int lo, hi;
        x.own_range(s, t0, t1, p, lo, hi);
        total += tiles_between<kKeys>(lo, hi);
        for (int t : {f, l}) {
          REQUIRE(x.seq_of(t, s0, s1) == s);
          const int pos = kv[s] - (cu[s + 1] - t);                          // sees max(0, pos - window + 1) .. pos
          const int first = w.window ? std::max(pos - w.window + 1, 0) : 0;
          if (pos >= p && pos >= 0) REQUIRE(lo <= std::max(first, p) && hi >= pos + 1 && hi <= kv[s]);
          if (first < p && pos >= 0) REQUIRE(it.lo <= first);
          REQUIRE(pos < 0 || pos >= p);                                     // the prefix ends before any new token
        }
      }
      REQUIRE(it.ue - it.ub == std::max(total, 1));
      if (at == it.ue) REQUIRE(it.kt1 == std::max(total, 1));
    }
    REQUIRE(at == u1);
  }
  REQUIRE(at == sh.total);
  std::printf("%lld %d %d\n", sh.total, sh.runs, cut);
}

int main() {
  for (int seed = 0; seed < 60; ++seed) {
    check<16, 64>(seed);
    check<32, 64>(seed + 100);
    check<256, 128>(seed + 200);
  }
  return 0;
}
