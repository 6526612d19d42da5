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
    w.tile_rows = pick(0, 1) ? 16 : 32;
    w.causal = pick(0, 1);
    w.max_rows = pick(0, 2) ? 0x7FFFFFFF : pick(1, 100);
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
    const int behind = tokens;
    tokens += pick(0, 3);                                // and behind the last
    if (!ragged) tokens = per_request * w.requests;
    w.tokens = tokens;
    w.q_start = ragged ? start.data() : nullptr;
    w.kv_len = len.data();

    const long long total = total_units(w);
    if (w.max_rows == 0x7FFFFFFF)
      CHECK(total <= max_units(tokens, w.requests, w.group, w.heads, w.tile_rows, ragged, (int)w.capacity));
    const int ctas = pick(1, 50);
    const long long per = (total + ctas - 1) / ctas;
    // (token, query head) -> keys taken so far; parts by slot.
    std::map<std::pair<int, int>, int> taken;
    std::map<long long, std::vector<std::pair<int, int>>> slots;
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
    // The joining kernel's view of every row.
    for (int t = 0; t < tokens; ++t)
      for (int head = 0; head < w.group * w.heads; ++head) {
        const auto key = std::make_pair(t, head);
        const int b = request_of(w.q_start, w.requests, tokens, t);
        CHECK((b >= 0) == (!ragged || (t >= start[0] && t < behind)));
        if (b < 0 || t - span_of(w, b).token0 >= span_of(w, b).n) {
          CHECK(taken.find(key) == taken.end());
          continue;
        }
        const RequestSpan s = span_of(w, b);
        const long long row = (long long)(t - s.token0) * w.group + head % w.group;
        const RowTile rt = tile_of(s, b, w.group, w.tile_rows, row / w.tile_rows, w.causal);
        CHECK(taken.count(key) && taken[key] == rt.last_key);
        int units;
        long long first = segment_start(w, s, row, head / w.group, &units);
        for (int i = 0; i < b; ++i) first += units_of(w, i);
        CHECK(units == tile_units(rt.last_key) && first + units <= total);
        const int c0 = (int)(first / per), c1 = (int)((first + units - 1) / per);
        CHECK(c1 < ctas);
        for (int c = c0; c <= c1 && c0 != c1; ++c) {
          const long long part = 2ll * c + (c == c0 && first != c0 * per ? 1 : 0);
          const auto& rows = slots[part];
          CHECK((int)rows.size() > (int)(row % w.tile_rows) && rows[row % w.tile_rows] == key);
        }
      }
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
    for (int t = 0; t < tokens; ++t) {
      const int b = request_of(w.q_start, w.requests, tokens, t);
      CHECK(b >= -1 && b < w.requests);
    }
  }
  std::printf("ok\n");
  return 0;
}
