// Walks the work units of a window with sinks on the host, as the kernels do:
// every (query tile, key tile) that has a visible pair exactly once, nothing
// out of range, and partial results that do not overlap.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "fa_bwd2.cuh"

#define CHECK(x)                                                                                                \
  do {                                                                                                          \
    if (!(x)) {                                                                                                 \
      std::printf("failed: %s (Nq %d Nk %d window %d sinks %d BM %d)\n", #x, Nq, Nk, window, sinks, BM);        \
      std::exit(1);                                                                                             \
    }                                                                                                           \
  } while (0)

static bool sees(int pos, int key, int window, int sinks) { return key <= pos && (key > pos - window || key < sinks); }

// the dK/dV kernel's units: key tiles of 128, query tiles of BM rows
template <int BM, int D>
static void dkdv(int Nq, int Nk, int window, int sinks) {
  const int off = Nk - Nq, nqt = (Nq + BM - 1) / BM, nkv = (Nk + 127) / 128;
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
  CHECK(p.far_units <= 64 + (sinks + 127) / 128);
  std::vector<int> met(static_cast<size_t>(nqt) * nkv, 0);
  std::vector<char> used(p.floats / (2 * D), 0);  // rows of partial results
  std::vector<int> writers(nkv, 0);               // near units (or whole ones) of a key tile
  int last = 1 << 30;
  for (int v = 0; v < p.far_units + nkv; ++v) {
    const fa::DkdvUnit w = fa::sink_dkdv_unit<BM, D, true>(prm, v);
    const fa::DkdvUnit same = fa::sink_dkdv_unit<BM, D, false>(prm, v);
    CHECK(w.j == same.j && w.i0 == same.i0 && w.n == same.n && w.partial == same.partial && w.far == same.far);
    CHECK(w.j >= 0 && w.j < nkv && w.i0 >= 0 && w.n >= 1 && w.i0 + w.n <= nqt);
    CHECK((w.far > 0) == (v < p.far_units));
    CHECK(w.n <= p.far_tiles);
    if (w.far == 0) {
      CHECK(w.n <= last || w.n <= 2);  // near units grow shorter (the first ones of a ragged offset may not)
      ++writers[w.j];
    }
    for (int i = w.i0; i < w.i0 + w.n; ++i) ++met[static_cast<size_t>(i) * nkv + w.j];
    if (w.partial) {
      CHECK(w.part >= 0 && w.part % (2 * D) == 0 && w.part / (2 * D) + w.rows <= p.floats / (2 * D));
      for (int r = 0; r < w.rows; ++r) {
        CHECK(!used[w.part / (2 * D) + r]);
        used[w.part / (2 * D) + r] = 1;
      }
      // what a far unit does not write, none of its queries sees
      if (w.far > 0)
        for (int key = w.j * 128 + w.rows; key < w.j * 128 + 128 && key < Nk; ++key)
          CHECK(!sees(w.i0 * BM + off, key, window, sinks));
    }
  }
  for (size_t r = 0; r < used.size(); ++r) CHECK(used[r]);
  for (int j = 0; j < nkv; ++j) CHECK(writers[j] == 1);
  for (int i = 0; i < nqt; ++i)
    for (int j = 0; j < nkv; ++j) {
      bool any = false;
      for (int q = i * BM; !any && q < (i + 1) * BM && q < Nq; ++q)
        for (int key = j * 128; !any && key < j * 128 + 128 && key < Nk; ++key) any = sees(q + off, key, window, sinks);
      const int n = met[static_cast<size_t>(i) * nkv + j];
      CHECK(n == 1 || (n == 0 && !any));
    }
}

// the forward's and the dQ kernel's key tiles of a query tile
template <int BN>
static void tiles(int Nq, int Nk, int window, int sinks) {
  const int BM = 128, off = Nk - Nq;
  for (int i0 = 0; i0 < Nq; i0 += BM) {
    const int i1 = (i0 + BM < Nq ? i0 + BM : Nq) - 1;
    fa::KeySpan s{};
    s.lo = i0 + off - window + 1 > 0 ? i0 + off - window + 1 : 0;
    s.hi = i1 + off + 1 < Nk ? i1 + off + 1 : Nk;
    int j0 = -1, skip = -1;
    const int n = fa::sink_key_tiles<BN>(sinks, s, j0, skip);
    CHECK(j0 == 0 && skip >= 0 && n >= 1);
    std::vector<int> met((Nk + BN - 1) / BN, 0);
    int before = -1;
    for (int v = 0; v < n; ++v) {
      const int j = fa::sink_key_tile<BN>(sinks, v, skip);
      CHECK(j > before && j < static_cast<int>(met.size()));
      before = j;
      ++met[j];
    }
    for (int j = 0; j < static_cast<int>(met.size()); ++j) {
      bool any = false;
      for (int q = i0; !any && q <= i1; ++q)
        for (int key = j * BN; !any && key < (j + 1) * BN && key < Nk; ++key) any = sees(q + off, key, window, sinks);
      CHECK(!any || met[j] == 1);
      const bool cover = j * BN < sinks || ((j + 1) * BN > s.lo && j * BN < s.hi);
      CHECK(met[j] == 0 || cover);  // no tile without a reason
    }
  }
}

int main() {
  const int lengths[][2] = {{129, 129}, {1, 700}, {300, 300}, {640, 640}, {5, 1021}, {1021, 1021}, {130, 900}, {1500, 1600}};
  const int windows[] = {1, 2, 63, 64, 127, 128, 129, 300, 511};
  const int sinks[] = {1, 4, 64, 127, 128, 129, 260, 500, 900};
  for (auto& l : lengths)
    for (int w : windows)
      for (int s : sinks) {
        if (w + s >= l[1]) continue;  // hides nothing: not such a kernel's
        dkdv<128, 64>(l[0], l[1], w, s);
        dkdv<64, 256>(l[0], l[1], w, s);
        tiles<128>(l[0], l[1], w, s);
        tiles<64>(l[0], l[1], w, s);
      }
  dkdv<128, 128>(8192, 8192, 64, 4000);
  std::printf("ok\n");
  return 0;
}
