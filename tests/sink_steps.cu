// The dQ kernels' steps over the key tiles of a window with sinks, on the host:
// every tile's sum is taken once before Delta is known, every tile's dS is formed
// once, those of tiles with sinks with the known Delta, and the first dS is where
// the kernels overwrite dQ.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fa_bwd2.cuh"

#define CHECK(x)                                                                                             \
  do {                                                                                                       \
    if (!(x)) {                                                                                              \
      std::printf("failed: %s (i0 %d Nq %d Nk %d window %d sinks %d BN %d)\n", #x, i0, Nq, Nk, window, sinks, BN); \
      std::exit(1);                                                                                          \
    }                                                                                                        \
  } while (0)

template <int BN>
static void steps(int Nq, int Nk, int window, int sinks) {
  const int off = Nk - Nq;
  for (int i0 = 0; i0 < Nq; i0 += 128) {
    fa::KeySpan s{};
    s.lo = i0 + off - window + 1 > 0 ? i0 + off - window + 1 : 0;
    s.hi = (i0 + 128 < Nq ? i0 + 128 : Nq) + off;
    const auto k = fa::sink_dq_steps<BN>(sinks, s);
    std::vector<int> sums((Nk + BN - 1) / BN, 0), formed(sums.size(), 0), tiles(sums.size(), 0);
    int j0, skip, first = -1;
    const int n = fa::sink_key_tiles<BN>(sinks, s, j0, skip);
    for (int v = 0; v < n; ++v) ++tiles[fa::sink_key_tile<BN>(sinks, v, skip)];
    bool known = false;
    for (int j = 0; j < k.n; ++j) {
      const int t = k.key(j);
      CHECK(t >= 0 && t < static_cast<int>(sums.size()));
      if (!known) ++sums[t];
      if (k.knows(j)) {
        CHECK(!known);
        known = true;
        CHECK(sums == tiles);
      }
      if (!k.counts(j)) {
        if (first < 0) first = j;
        ++formed[t];
        if (t * BN < sinks && t * BN < s.hi) CHECK(known);
      }
    }
    CHECK(known && formed == tiles && first == k.first());
    if (sinks <= BN) CHECK(k.n == n);
  }
}

int main() {
  const int lengths[][2] = {{1, 700}, {300, 300}, {5, 1021}, {1021, 1021}, {130, 900}, {1500, 1600}};
  const int windows[] = {1, 63, 64, 128, 300, 511};
  const int sinks[] = {1, 64, 65, 127, 128, 129, 200, 260, 500, 900};
  for (auto& l : lengths)
    for (int w : windows)
      for (int s : sinks) {
        if (w + s >= l[1]) continue;
        steps<64>(l[0], l[1], w, s);
        steps<128>(l[0], l[1], w, s);
      }
  std::printf("ok\n");
  return 0;
}
