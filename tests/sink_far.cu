// The far units of a window with sinks in closed form against sums over the key
// tiles, and units of thousands of sinks against each other, on the host.  Prints
// "ok".
#include <cstdio>
#include <cstdlib>

#include "fa_bwd2.cuh"

#define CHECK(x)                                                                                       \
  do {                                                                                                 \
    if (!(x)) {                                                                                        \
      std::printf("failed: %s (Nq %d Nk %d window %d sinks %d BM %d)\n", #x, Nq, Nk, window, sinks, BM); \
      std::exit(1);                                                                                    \
    }                                                                                                  \
  } while (0)

template <int BM>
static void sums(int Nq, int Nk, int window, int sinks, int far_tiles) {
  const int off = Nk - Nq, tiles = (sinks + 127) / 128;
  long long units = 0;
  for (int j = 0; j <= tiles; ++j) {
    CHECK((fa::sink_far_before<BM, long long>(j, window, Nq, off, far_tiles)) == units);
    CHECK((fa::sink_far_before<BM, int>(j, window, Nq, off, far_tiles)) == units);
    if (j < tiles) units += fa::sink_tile<BM>(j, sinks, window, Nq, off, far_tiles).far;
  }
}

// parts and units as a walk over the key tiles finds them
template <int BM, int D>
static void walk(int Nq, int Nk, int window, int sinks) {
  const int off = Nk - Nq, tiles = (sinks + 127) / 128;
  const fa::SinkParts p = fa::sink_parts<BM>(sinks, window, Nq, Nk, D);
  fa::BwdParams prm{};
  prm.Nq = Nq;
  prm.Nk = Nk;
  prm.causal_off = off;
  prm.rule.window = window;
  prm.rule.sinks = sinks;
  prm.far_tiles = p.far_tiles;
  prm.far_units = p.far_units;
  prm.part_floats = p.floats;
  long long far = 0, units = 0, rows = 0;
  for (int j = 0; j < tiles; ++j) far += fa::sink_tile<BM>(j, sinks, window, Nq, off, 1).far;
  CHECK(p.far_tiles >= (far + 63) / 64);
  int v = p.far_units;  // far units are numbered from the last tile's
  for (int j = 0; j < tiles; ++j) {
    const fa::SinkTile t = fa::sink_tile<BM>(j, sinks, window, Nq, off, p.far_tiles);
    units += t.far;
    v -= t.far;
    CHECK(v >= 0);
    for (int f = 1; f <= t.far; ++f) {
      const fa::DkdvUnit w = fa::sink_dkdv_unit<BM, D, true>(prm, v + f - 1);
      CHECK(w.j == j && w.far == f && w.rows == t.rows && w.partial && w.i0 == t.near_end + (f - 1) * p.far_tiles);
      CHECK(w.part == (rows + 128 + static_cast<long long>(f - 1) * t.rows) * 2 * D);
    }
    const fa::DkdvUnit near = fa::sink_dkdv_unit<BM, D, true>(prm, p.far_units + j);
    CHECK(near.j == j && near.far == 0 && near.partial == (t.far > 0) && near.i0 == t.first);
    if (t.far > 0) {
      CHECK(near.part == rows * 2 * D);
      rows += 128 + static_cast<long long>(t.far) * t.rows;
    }
  }
  CHECK(units == p.far_units && rows * 2 * D == p.floats);
}

int main() {
  unsigned long long x = 88172645463325252ull;
  auto below = [&](int n) {
    x ^= x << 13;
    x ^= x >> 7;
    x ^= x << 17;
    return static_cast<int>(x % static_cast<unsigned long long>(n));
  };
  for (int n = 0; n < 4000; ++n) {
    const int Nk = 2 + below(n % 4 == 0 ? 300 : n % 4 == 1 ? 3000 : 40000);
    const int Nq = n % 3 == 0 ? Nk : 1 + below(Nk);
    const int window = 1 + below(n % 2 == 0 ? (Nk < 400 ? Nk : 400) : Nk), sinks = 1 + below(Nk);
    if (static_cast<long long>(window) + sinks >= Nk) continue;  // hides nothing: not such a kernel's
    const int far_tiles = 1 + below(40);
    sums<128>(Nq, Nk, window, sinks, far_tiles);
    sums<64>(Nq, Nk, window, sinks, far_tiles);
    walk<128, 128>(Nq, Nk, window, sinks);
    walk<64, 256>(Nq, Nk, window, sinks);
  }
  walk<128, 64>(1 << 20, 1 << 20, 1000, 1 << 19);
  walk<64, 256>(1 << 20, (1 << 20) + 77, 1, 1 << 19);
  std::printf("ok\n");
  return 0;
}
