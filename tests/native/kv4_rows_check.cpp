// Host check of kv4_rows.cuh: which query rows and keys the tiles of the
// attention over the 4-bit cache take.  Random requests; every row is in one
// tile, the key parts of a tile cover its keys once, the joining kernel finds
// the same tile, and arrays with arbitrary content never lead out of range.
#include "kv4_rows.cuh"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

using namespace svdq;

#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      std::printf("FAILED line %d: %s (case %d)\n", __LINE__, #c, trial); \
      return 1;                                                           \
    }                                                                     \
  } while (0)

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int trial = 0; trial < 20000; ++trial) {
    const int requests = pick(1, 70), group = pick(1, 9), rows = pick(0, 1) ? 16 : (pick(0, 1) ? 32 : 128), causal = pick(0, 1);
    const bool ragged = pick(0, 3) != 0;
    const int page = 16 << pick(0, 4), max_pages = pick(0, 6);
    const long long capacity = (long long)page * max_pages;
    std::vector<int> start(requests + 1), len(requests);
    int tokens = pick(0, 3), per = pick(0, 5);           // tokens before the first request
    start[0] = tokens;
    for (int b = 0; b < requests; ++b) {
      tokens += pick(0, 2) ? pick(0, 40) : 0;
      start[b + 1] = tokens;
      len[b] = pick(0, 9) == 0 ? pick(-5, 5) : pick(0, (int)capacity + 20);
    }
    tokens += pick(0, 3);                                // and behind the last
    if (!ragged) tokens = per * requests;
    const int* qs = ragged ? start.data() : nullptr;
    const long long tiles = max_row_tiles(tokens, requests, group, rows, ragged);
    const int splits = pick(1, 9), chunk = 64 * pick(1, 4);
    std::vector<int> seen((size_t)tokens * group, 0), keys_at((size_t)tokens * group, -1);
    for (long long tile = 0; tile < tiles; ++tile) {
      const RowTile r = find_row_tile_serial(qs, len.data(), requests, tokens, group, rows, tile, capacity, causal);
      if (r.rows <= 0) continue;
      CHECK(r.keys >= 0 && r.keys <= capacity && r.rows <= rows);
      CHECK(r.last_key >= 0 && r.last_key <= r.keys);
      const int active = active_parts(r.last_key, splits, chunk);
      CHECK(active >= 1 && active <= splits);
      int covered = 0;
      for (int s = 0; s < active; ++s) {
        const int k0 = s * chunk, k1 = s == active - 1 ? r.last_key : k0 + chunk;
        CHECK(k0 == covered && k1 >= k0);
        covered = k1;
      }
      CHECK(covered == r.last_key);
      for (int i = 0; i < r.rows; ++i) {
        const int row = r.row0 + i, tok = row / group;
        CHECK(tok < r.n && r.token0 + tok < tokens);
        CHECK(r.keys_of(tok, causal) <= r.last_key);
        const size_t at = (size_t)(r.token0 + tok) * group + row % group;
        ++seen[at];
        keys_at[at] = r.last_key;
      }
    }
    for (int t = 0; t < tokens; ++t)
      for (int h = 0; h < group; ++h) {
        const size_t at = (size_t)t * group + h;
        const bool owned = !ragged || (t >= start[0] && t < start[requests]);
        CHECK(seen[at] == (owned ? 1 : 0));
        CHECK(find_last_key(qs, len.data(), requests, tokens, t, group, h, rows, capacity, causal) ==
              (owned ? keys_at[at] : -1));
      }
    // Arbitrary content: nothing out of range, whatever the order of the starts.
    for (auto& v : start) v = (int)rng();
    for (auto& v : len) v = (int)rng();
    for (long long tile = 0; tile < tiles; ++tile) {
      const RowTile r = find_row_tile_serial(qs, len.data(), requests, tokens, group, rows, tile, capacity, causal);
      if (r.rows <= 0) continue;
      CHECK(r.request >= 0 && r.request < requests && r.keys >= 0 && r.keys <= capacity);
      CHECK(r.last_key >= 0 && r.last_key <= r.keys);
      CHECK(r.row0 >= 0 && r.token0 >= 0 && r.token0 + (r.row0 + r.rows - 1) / group < tokens);
    }
    for (int t = 0; t < tokens; ++t)
      CHECK(find_last_key(qs, len.data(), requests, tokens, t, group, 0, rows, capacity, causal) <= capacity);
  }
  std::printf("ok\n");
  return 0;
}
