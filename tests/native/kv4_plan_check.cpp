// Host check of split_rows (kv4_rows.cuh): whatever the rows of a call, the
// number of its requests and their sizes, each request is taken by exactly one
// of the kernels that are launched.  Also the work's cut in tiles of 24 rows.
#include "kv4_rows.cuh"

#include <cstdio>
#include <random>
#include <vector>

using namespace svdq;

#define CHECK(c)                                                                             \
  do {                                                                                       \
    if (!(c)) {                                                                              \
      std::printf("FAILED line %d: %s (rows %lld, requests %d)\n", __LINE__, #c, rows, requests); \
      return 1;                                                                              \
    }                                                                                        \
  } while (0)

int main() {
  const long long large[] = {16383, 16384, 16385, 65536, 1000003, 1ll << 30};
  for (int requests = 1; requests <= 70; ++requests)
    for (long long i = 1; i <= 3000; ++i)
      for (int ragged = 0; ragged < 2; ++ragged) {
        const long long rows = i <= 2994 ? i : large[i - 2995];
        if (!ragged && rows % requests != 0) continue;
        const RowSplit s = split_rows(rows, requests, ragged != 0);
        CHECK(s.few || s.many);
        // Sizes that a request of this call can have (more than 0 rows: others have nothing to do).
        const long long lo = ragged ? 1 : rows / requests, hi = ragged ? rows : lo;
        for (long long size = lo; size <= hi; size = size < 1100 || size >= hi ? size + 1 : (2 * size < hi ? 2 * size : hi)) {
          const bool few = s.few && size <= s.few_max, many = s.many && size >= s.many_min;
          CHECK(few != many);
        }
      }

  // Tiles of 24 rows: every row of a request lies in one tile, whose last row sees what the tile's units cover.
  std::mt19937 rng(11);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int trial = 0; trial < 4000; ++trial) {
    Kv4Work w;
    const int requests = 1;
    w.requests = requests;
    w.group = pick(1, 30);
    w.heads = pick(1, 3);
    w.tile_rows = 24;
    w.causal = pick(0, 1);
    w.min_rows = 0;
    w.max_rows = 0x7FFFFFFF;
    w.capacity = 4096;
    w.tokens = pick(1, 40);
    const std::vector<int> start = {0, w.tokens}, len = {pick(0, 1500)};
    w.q_start = start.data();
    w.kv_len = len.data();
    const RequestSpan s = span_of(w, 0);
    const long long rows = (long long)s.n * w.group, all = head_units(w, s) * w.heads;
    std::vector<int> units(w.heads * rows, 0);
    for (long long u = 0; u < all;) {
      const Segment g = segment_in(w, s, 0, u);
      CHECK(g.unit0 == 0 && g.units == tile_units(g.tile.last_key) && g.tile.rows > 0 && g.tile.rows <= 24);
      for (int i = 0; i < g.tile.rows; ++i) units[g.head * rows + g.tile.row0 + i] += g.units;
      u += g.units;
    }
    for (int h = 0; h < w.heads; ++h)
      for (long long r = 0; r < rows; ++r) {
        const RowTile t = tile_of(s, 0, w.group, 24, r / 24, w.causal);
        CHECK(units[h * rows + r] == tile_units(t.last_key));
        CHECK(t.keys_of((int)(r / w.group), w.causal) <= t.last_key);
      }
  }
  std::printf("ok\n");
  return 0;
}
