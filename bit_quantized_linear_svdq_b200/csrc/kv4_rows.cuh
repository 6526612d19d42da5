// kv4_rows.cuh -- which query rows and keys a tile of the attention over the
// 4-bit cache has.  Plain integer code, also compiled for the host by the
// tests (no CUDA header is needed for that).
//
// Request b has the query tokens q_start[b] .. q_start[b+1] (or, without
// q_start, tokens / requests each) and kv_len[b] keys.  For one key head its
// rows are (token, head of the group), `group` rows a token.  Every value read
// from a device array is clamped to what exists, so that no content of the
// arrays leads to an access out of range.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define KV4_HD __host__ __device__ __forceinline__
#else
#define KV4_HD inline
#endif

namespace svdq {

KV4_HD int kv4_min(long long a, long long b) { return (int)(a < b ? a : b); }
KV4_HD int kv4_max(long long a, long long b) { return (int)(a > b ? a : b); }
// a / b for a >= 0, b > 0, by 32-bit division where both fit (a 64-bit one
// costs about 500 cycles; five of them in a row were most of the set-up).
KV4_HD long long kv4_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct RequestSpan {
  int token0, n, keys;                          // first token, tokens, keys
};
KV4_HD RequestSpan request_span(const int* q_start, const int* kv_len, int requests, int tokens, int b,
                                long long capacity) {
  RequestSpan s;
  if (q_start) {
    s.token0 = kv4_min(kv4_max(q_start[b], 0), tokens);
    s.n = kv4_min(kv4_max(q_start[b + 1], s.token0), tokens) - s.token0;
  } else {
    s.n = tokens / requests;
    s.token0 = b * s.n;
  }
  s.keys = kv_len ? kv4_min(kv4_max(kv_len[b], 0), capacity) : 0;
  return s;
}

// Keys that token i of the n of a request sees.
KV4_HD int keys_seen(int keys, int n, int i, int causal) {
  return causal ? kv4_max((long long)keys - n + i + 1, 0) : keys;
}

// A tile: `tile_rows` consecutive rows of a request under one key head.
struct RowTile {
  int request, token0, n, keys;                 // of the request
  int row0, rows;                               // of the tile; rows == 0: nothing to do
  int last_key;                                 // keys that its last row sees
  KV4_HD int keys_of(int tok, int causal) const { return keys_seen(keys, n, tok, causal); }
};
KV4_HD RowTile tile_of(const RequestSpan& s, int b, int group, int tile_rows, long long tile, int causal) {
  RowTile r;
  r.request = b;
  r.token0 = s.token0;
  r.n = s.n;
  r.keys = s.keys;
  // (tokens x query heads fits 31 bits: checked at the call)
  const int row0 = (int)tile * tile_rows, all = s.n * group;
  r.row0 = row0;
  r.rows = row0 < all ? (all - row0 < tile_rows ? all - row0 : tile_rows) : 0;
  const int last = r.rows > 0 ? (int)((uint32_t)(row0 + r.rows - 1) / (uint32_t)group) : 0;
  r.last_key = r.rows > 0 ? keys_seen(s.keys, s.n, last, causal) : 0;
  return r;
}

// The work of one launch, cut into equal shares.  A segment is a tile under
// one key head, a unit 128 of its keys (at least one unit, so that rows without
// keys are written too).  Units are numbered by request, head, tile, key; CTA
// c takes units c * per .. (c + 1) * per.  A segment that lies in one share is
// finished there; otherwise each of its CTAs leaves a part, in slot 0 if the
// segment covers the share's first unit and in slot 1 if it starts later (at
// most one of each a CTA).  A CTA begins at most one segment that it does not
// finish, the last of its share.
constexpr int kUnitKeys = 128;
struct Kv4Work {
  const int *q_start, *kv_len;
  int requests, tokens, group, heads, tile_rows, causal;
  int min_rows, max_rows;                       // requests with fewer or more rows are left out
  long long capacity;                           // keys that a block table can hold
};
KV4_HD RequestSpan span_of(const Kv4Work& w, int b) {
  RequestSpan s = request_span(w.q_start, w.kv_len, w.requests, w.tokens, b, w.capacity);
  const int rows = s.n * w.group;
  if (rows < w.min_rows || rows > w.max_rows) s.n = 0;
  return s;
}
KV4_HD int tile_units(int last_key) { return last_key > 0 ? (int)((uint32_t)(last_key - 1) / kUnitKeys) + 1 : 1; }
KV4_HD int tiles_of(const Kv4Work& w, const RequestSpan& s) {
  const int rows = s.n * w.group;
  return rows <= w.tile_rows ? (rows > 0 ? 1 : 0) : (int)((uint32_t)(rows + w.tile_rows - 1) / (uint32_t)w.tile_rows);
}
// Steps through a request's tiles: the token of each tile's last row, without
// a division a tile.
struct TileWalk {
  int tok, rem, more_tok, more_rem, group, last;
  KV4_HD TileWalk(const Kv4Work& w, const RequestSpan& s)
      : tok((w.tile_rows - 1) / w.group),
        rem((w.tile_rows - 1) % w.group),
        more_tok(w.tile_rows / w.group),
        more_rem(w.tile_rows % w.group),
        group(w.group),
        last(s.n - 1) {}
  KV4_HD int last_token() const { return tok < last ? tok : last; }
  KV4_HD void next() {
    tok += more_tok;
    rem += more_rem;
    if (rem >= group) {
      rem -= group;
      ++tok;
    }
  }
};
// Units of a request under one head.
KV4_HD long long head_units(const Kv4Work& w, const RequestSpan& s) {
  const int nt = tiles_of(w, s);
  // One tile, or tiles that all see the same keys: its last row is the request's last token, which sees every key.
  if (!w.causal || nt <= 1) return (long long)nt * tile_units(s.keys);
  TileWalk walk(w, s);
  long long u = 0;
  for (int t = 0; t < nt; ++t, walk.next()) u += tile_units(keys_seen(s.keys, s.n, walk.last_token(), 1));
  return u;
}
struct Segment {
  RowTile tile;
  int head, units, unit0;                       // units of the segment; the wanted unit's place in it
};
// Unit `u` of request b (u < heads * head_units).
KV4_HD Segment segment_in(const Kv4Work& w, const RequestSpan& s, int b, long long u) {
  const long long per_head = head_units(w, s);
  Segment g;
  g.head = (int)kv4_div(u, per_head);
  u -= g.head * per_head;
  int t = 0;
  if (!w.causal || s.n * w.group <= w.tile_rows) {
    g.units = tile_units(s.keys);
    t = u < g.units ? 0 : (int)kv4_div(u, g.units);
    u -= (long long)t * g.units;
  } else {
    TileWalk walk(w, s);
    for (;; ++t, walk.next()) {
      g.units = tile_units(keys_seen(s.keys, s.n, walk.last_token(), 1));
      if (u < g.units) break;
      u -= g.units;
    }
  }
  g.tile = tile_of(s, b, w.group, w.tile_rows, t, w.causal);
  g.unit0 = (int)u;
  return g;
}
// Upper bound of the units of a launch whose requests have at most `max_kv` keys.
KV4_HD long long max_units(int tokens, int requests, int group, int heads, int tile_rows, bool ragged, int max_kv) {
  const long long tiles = ragged ? ((long long)tokens * group + (long long)requests * (tile_rows - 1)) / tile_rows
                                 : requests * (((long long)(tokens / requests) * group + tile_rows - 1) / tile_rows);
  return tiles * heads * tile_units(max_kv);
}

// Which requests of a call each kernel takes, by their rows (query heads of one
// key head x tokens).  Every size that the call can hold belongs to one of the
// two that are launched (tests/native/kv4_plan_check.cpp).
struct RowSplit {
  bool few, many;                               // launched
  int few_max, many_min;                        // rows of a request at most / at least
};
constexpr int kFewRows = 64, kFewRowsInAll = 512, kManyRowsEach = 256;
KV4_HD RowSplit split_rows(long long rows, int requests, bool ragged) {
  RowSplit s;
  if (!ragged) {                                // the requests are alike
    s.many = rows > (long long)kFewRows * requests;
    s.few = !s.many;
  } else {
    // The requests' sizes are on the device: each kernel takes its own.  Where
    // requests have 256 rows on average all of them go to the many-row kernel:
    // small requests among them take no more of its tiles than the large ones.
    // Fewer are left to the few-row kernel alone up to a few hundred rows in all
    // (one request of 4096 keys, 8 key heads, D = 64 / 128: 96 rows 22.1 / 28.6
    // us, 252 rows 25.5 / 37.1; on the many-row kernel 17.7 / 20.7 and 23.5 /
    // 28.9, but beside small requests that one is a second pair of launches).
    s.few = rows < (long long)kManyRowsEach * requests;
    s.many = !s.few || rows > kFewRowsInAll;
  }
  s.few_max = s.many ? kFewRows : 0x7FFFFFFF;
  s.many_min = s.few ? kFewRows + 1 : 0;
  return s;
}

#if defined(__CUDACC__)
// Warp-wide view of the launch's units: total, and the first unit of a request.
// Every lane calls with the same arguments.
struct WarpUnits {
  long long total;
  long long mine, upto;                         // requests <= 32: units of request `lane`, inclusive prefix
};
__device__ __forceinline__ long long warp_prefix(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
__device__ __forceinline__ long long units_of_request(const Kv4Work& w, int b) {
  return b < w.requests ? head_units(w, span_of(w, b)) * w.heads : 0;
}
__device__ __forceinline__ WarpUnits warp_units(const Kv4Work& w) {
  const int lane = threadIdx.x & 31;
  WarpUnits r;
  r.total = 0;
  for (int b0 = 0; b0 < w.requests; b0 += 32) {
    r.mine = units_of_request(w, b0 + lane);
    r.upto = warp_prefix(r.mine);
    r.total += __shfl_sync(0xFFFFFFFFu, r.upto, 31);
  }
  return r;
}
// Request that holds unit u (< total), and that request's first unit.
__device__ __forceinline__ int request_of_unit(const Kv4Work& w, const WarpUnits& r, long long u, long long* first) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < w.requests; b0 += 32) {
    const long long mine = w.requests <= 32 ? r.mine : units_of_request(w, b0 + lane);
    const long long upto = w.requests <= 32 ? r.upto : warp_prefix(mine);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, u < before + upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *first = before + __shfl_sync(0xFFFFFFFFu, upto - mine, l);
      return b0 + l;
    }
    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  *first = before;
  return w.requests - 1;
}
#endif

}  // namespace svdq
