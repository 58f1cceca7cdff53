// The order in which the key tiles of a shared item are taken, on the host: every tile once, the prefix first, each part in its own
// order; and for an item whose rows see nothing, no segment.
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

void check(int prefix, int half0, int both, int half1) {
  Plan plan{};
  plan.prefix = prefix;
  plan.half0 = half0;
  plan.both = both;
  plan.half1 = half1;
  const int total = prefix + half0 + both + half1;
  std::vector<int> seen(total, -1);
  int last0 = -1, last1 = -1;
  for (int v = 0; v < total; ++v) {
    const int at = in_turn(&plan, v);
    REQUIRE(at >= 0 && at < total && seen[at] < 0);
    seen[at] = v;
    if (v < prefix) {
      REQUIRE(at == v);
    } else if (v < prefix + both) {
      REQUIRE(at == v + half0);
    } else if (at < prefix + half0) {
      REQUIRE(at > last0);
      last0 = at;
    } else {
      REQUIRE(at > last1);
      last1 = at;
    }
  }
}

int main() {
  std::mt19937 r(1);
  auto pick = [&](int hi) { return static_cast<int>(r() % (hi + 1)); };
  for (int i = 0; i < 2000; ++i) check(pick(3) ? pick(40) : 0, pick(2) ? pick(60) : 0, pick(2) ? 0 : pick(9), pick(2) ? pick(60) : 0);
  check(0, 1 << 20, 0, 3);
  // no row sees a key: one tile, of no segment (the prefix's is empty)
  Plan none{};
  none.count = 1;
  const int4 seg[1] = {make_int4(0, 0, -1, 0)};
  int key0 = 0;
  REQUIRE(seg_of<128>(seg, none.count, in_turn(&none, 0), key0) == -1);
  std::printf("ok\n");
  return 0;
}
