// Host check of kv4_rows.cuh: how the attention over the 4-bit cache cuts its
// work.  Random requests and numbers of CTAs; every key of every row is taken
// once, every cut segment's parts are found again by the joining kernel's
// arithmetic in distinct slots, and arrays with arbitrary content never lead
// out of range.
#include "kv4_rows.cuh"

#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

using namespace svdq;

#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      std::printf("FAILED line %d: %s (case %d)\n", __LINE__, #c, trial); \
      return 1;                                                           \
    }                                                                     \
  } while (0)

// Serial forms of the warp-wide searches.
static long long units_of(const Kv4Work& w, int b) { return head_units(w, span_of(w, b)) * w.heads; }
static long long total_units(const Kv4Work& w) {
  long long u = 0;
  for (int b = 0; b < w.requests; ++b) u += units_of(w, b);
  return u;
}

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int trial = 0; trial < 6000; ++trial) {
    Kv4Work w;
    w.requests = pick(1, 40);
    w.group = pick(1, 9);
    w.heads = pick(1, 4);
    w.tile_rows = 8 << pick(0, 5);
    w.causal = pick(0, 1);
    w.min_rows = pick(0, 2) ? 0 : pick(1, 50);
    w.max_rows = pick(0, 2) ? 0x7FFFFFFF : w.min_rows + pick(0, 100);
    const bool ragged = pick(0, 3) != 0;
    const int page = 16 << pick(0, 4), max_pages = pick(0, 6);
    w.capacity = (long long)page * max_pages;
    std::vector<int> start(w.requests + 1), len(w.requests);
    int tokens = pick(0, 3), per_request = pick(0, 5);   // tokens before the first request
    start[0] = tokens;
    for (int b = 0; b < w.requests; ++b) {
      tokens += pick(0, 2) ? pick(0, 40) : 0;
      start[b + 1] = tokens;
      len[b] = pick(0, 9) == 0 ? pick(-5, 5) : pick(0, (int)w.capacity + 20);
    }
    tokens += pick(0, 3);                                // and behind the last
    if (!ragged) tokens = per_request * w.requests;
    w.tokens = tokens;
    w.q_start = ragged ? start.data() : nullptr;
    w.kv_len = len.data();

    const long long total = total_units(w);
    CHECK(total <= max_units(tokens, w.requests, w.group, w.heads, w.tile_rows, ragged, (int)w.capacity));
    const int ctas = pick(1, 50);
    const long long per = (total + ctas - 1) / ctas;
    // (token, query head) -> keys taken so far; parts by slot.
    std::map<std::pair<int, int>, int> taken;
    std::map<long long, std::vector<std::pair<int, int>>> slots;
    struct Cut {
      int token0, row0, rows, head, last_cta, slot;
    };
    std::vector<Cut> cuts(ctas, Cut{0, 0, 0, 0, 0, 0});
    for (int c = 0; c < ctas; ++c) {
      const long long u0 = per * c, u1 = u0 + per < total ? u0 + per : total;
      for (long long u = u0; u < u1;) {
        int b = 0;
        long long first = 0;
        while (u >= first + units_of(w, b)) first += units_of(w, b), ++b;
        const Segment g = segment_in(w, span_of(w, b), b, u - first);
        const int n = (int)(g.units - g.unit0 < u1 - u ? g.units - g.unit0 : u1 - u);
        CHECK(n > 0 && g.head < w.heads && g.tile.rows > 0 && g.tile.rows <= w.tile_rows && g.tile.request == b);
        CHECK(g.tile.keys >= 0 && g.tile.keys <= w.capacity && g.tile.last_key <= g.tile.keys);
        const int k0 = g.unit0 * kUnitKeys;
        const int k1 = g.tile.last_key < k0 + n * kUnitKeys ? g.tile.last_key : k0 + n * kUnitKeys;
        CHECK(k0 <= k1 || (k0 == 0 && k1 == 0));
        const bool whole = n == g.units;
        const long long part = 2ll * c + (u == u0 ? 0 : 1);
        if (!whole) CHECK(slots.find(part) == slots.end());
        if (!whole && g.unit0 == 0) {
          CHECK(cuts[c].rows == 0 && u + n == u1);
          cuts[c] = Cut{g.tile.token0, g.tile.row0, g.tile.rows, g.head, (int)((u + g.units - 1) / per), u == u0 ? 0 : 1};
        }
        for (int i = 0; i < g.tile.rows; ++i) {
          const int row = g.tile.row0 + i, tok = row / w.group, head = g.head * w.group + row % w.group;
          CHECK(tok < g.tile.n && g.tile.token0 + tok < tokens);
          CHECK(g.tile.keys_of(tok, w.causal) <= g.tile.last_key);
          const auto key = std::make_pair(g.tile.token0 + tok, head);
          CHECK(taken[key] == k0);                       // in order, without gaps
          taken[key] = k1;
          if (!whole) slots[part].push_back(key);
        }
        u += n;
      }
    }
    // Every row of the requests that take part has all its keys.
    for (int b = 0; b < w.requests; ++b) {
      const RequestSpan s = span_of(w, b);
      for (int i = 0; i < s.n; ++i)
        for (int head = 0; head < w.group * w.heads; ++head) {
          const long long row = (long long)i * w.group + head % w.group;
          const auto key = std::make_pair(s.token0 + i, head);
          CHECK(taken.count(key) && taken[key] == tile_of(s, b, w.group, w.tile_rows, row / w.tile_rows, w.causal).last_key);
          taken.erase(key);
        }
    }
    CHECK(taken.empty());
    // The joining kernel's view: each cut segment from the note of the CTA that began it, its parts where they were left.
    std::set<long long> joined;
    for (int c0 = 0; c0 < ctas; ++c0) {
      if (!cuts[c0].rows) continue;
      for (int c = c0; c <= cuts[c0].last_cta; ++c) {
        const long long part = 2ll * c + (c == c0 ? cuts[c0].slot : 0);
        CHECK(c < ctas && joined.insert(part).second && (int)slots[part].size() == cuts[c0].rows);
        for (int i = 0; i < cuts[c0].rows; ++i) {
          const int row = cuts[c0].row0 + i;
          CHECK(slots[part][i] == std::make_pair(cuts[c0].token0 + row / w.group, cuts[c0].head * w.group + row % w.group));
        }
      }
    }
    CHECK(cuts[ctas - 1].rows == 0);
    CHECK(joined.size() == slots.size());
    // Arbitrary content: nothing out of range, whatever the order of the starts.
    for (auto& v : start) v = (int)rng();
    for (auto& v : len) v = (int)rng();
    for (int b = 0; b < w.requests; ++b) {
      const RequestSpan s = span_of(w, b);
      CHECK(s.n >= 0 && s.token0 >= 0 && s.token0 + s.n <= tokens && s.keys >= 0 && s.keys <= w.capacity);
      const long long mine = units_of(w, b);
      for (long long u = 0; u < mine; u += 1 + mine / 7) {
        const Segment g = segment_in(w, s, b, u);
        CHECK(g.head < w.heads && g.tile.last_key <= w.capacity && g.unit0 < g.units);
        CHECK(g.tile.token0 + (g.tile.row0 + g.tile.rows - 1) / w.group < tokens);
      }
    }
  }
  std::printf("ok\n");
  return 0;
}
