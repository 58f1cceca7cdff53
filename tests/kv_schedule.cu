// The attention kernels' schedule, run on the host: which CTA arrives at which ticket, when runs are given up half way.
// Prints one line per seed: units, runs, cut items, arrivals missed without the rest of a run that is given up.  Then
// "ctas", heads' size, row groups, sequences, CTAs an SM, shared memory of each, for the decode kernels' grids.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_decode.cuh"

using namespace qspec::att;
constexpr int kRows = 256, kKeys = 128;
using W = Walk<kRows, kKeys>;

#define REQUIRE(x)                                  \
  do {                                              \
    if (!(x)) {                                     \
      std::printf("line %d: %s\n", __LINE__, #x);  \
      std::exit(1);                                 \
    }                                               \
  } while (0)

struct Tickets {
  std::vector<int> at;
  void arrive(const Item& it, const ScanShared& sh) {
    const int c0 = owner_of(it.ub, &sh), c1 = owner_of(it.ue - 1, &sh);
    REQUIRE(c0 < c1);
    if (++at[c0] == c1 - c0 + 1) at[c0] = 0;
  }
  int left() const {
    int n = 0;
    for (int x : at) n += x != 0;
    return n;
  }
};

template <int D, int RG>
void grids() {
  using C = DecodeCfg<D, RG>;
  for (int b : {1, 64, 239, 240, 256, 300, 512, 1024}) std::printf("ctas %d %d %d %d %d\n", D, RG, b, C::ctas(b), C::smem(b));
}

int main() {
  for (int seed = 0; seed < 40; ++seed) {
    std::mt19937 r(seed);
    auto pick = [&](int lo, int hi) { return lo + static_cast<int>(r() % (hi - lo + 1)); };
    const int B = pick(1, 9), grid = pick(1, 152);
    std::vector<int2> seq(B + 1);
    W w{};
    w.heads = pick(1, 8);
    w.group = pick(1, 8);
    int shift = 0;
    while ((1 << shift) < w.group) ++shift;
    w.group_shift = 31 + shift;
    w.group_mul = static_cast<uint32_t>(((uint64_t(1) << w.group_shift) + w.group - 1) / w.group);
    w.window = pick(0, 2) ? 0 : pick(1, 900);
    w.tree = false;
    int tok = 0;
    for (int b = 0; b < B; ++b) {
      const int n = pick(0, 3) ? pick(0, 700) : 0;
      seq[b] = make_int2(tok, pick(0, 9) ? n + pick(0, 3000) : -1);
      tok += n;
    }
    seq[B] = make_int2(tok, -1);
    w.seq = seq.data();
    w.B = B;

    ScanShared sh{};
    for (int b = 0; b < B; ++b)
      for (int t = 0; t < 200; ++t) sh.total += w.units(b, t);
    if (sh.total == 0) continue;
    sh.runs = static_cast<int>(sh.total < grid ? sh.total : grid);
    auto run = [&](int c) {
      W x = w;
      x.u = run_start(c, &sh);
      x.u1 = run_start(c + 1, &sh);
      x.start(0, 0, 0);
      return x;
    };

    // every unit once, in order
    long long at = 0;
    int cut = 0;
    std::vector<int> items(sh.runs);
    for (int c = 0; c < sh.runs; ++c) {
      W x = run(c);
      const long long u0 = x.u, u1 = x.u1;
      while (x.next()) {
        const long long n = x.it.kt1 - x.it.kt0;
        REQUIRE(n > 0 && x.it.ub <= at && at + n <= x.it.ue && at >= u0 && at + n <= u1);
        at += n;
        cut += x.it.ub < u0 || x.it.ue > u1;
        ++items[c];
      }
      REQUIRE(at == u1);
    }
    REQUIRE(at == sh.total);

    // some runs give up after the item at which they stand; with and without the rest of their arrivals
    int missed = 0;
    for (int rest = 0; rest < 2; ++rest) {
      Tickets t{std::vector<int>(sh.runs)};
      std::mt19937 s(1000 + seed);
      for (int c = 0; c < sh.runs; ++c) {
        W x = run(c);
        const long long u0 = x.u, u1 = x.u1;
        int stop = s() % 3 ? 1 << 30 : static_cast<int>(s() % items[c]);
        while (x.next()) {
          if (x.it.ub < u0 || x.it.ue > u1) t.arrive(x.it, sh);
          if (stop-- == 0) break;
        }
        if (rest)
          while (x.next_cut(u0, u1)) t.arrive(x.it, sh);
      }
      if (rest)
        REQUIRE(t.left() == 0);
      else
        missed = t.left();
    }
    std::printf("%lld %d %d %d\n", sh.total, sh.runs, cut, missed);
  }
  grids<64, 1>();
  grids<64, 2>();
  grids<128, 1>();
  grids<128, 2>();
  return 0;
}
