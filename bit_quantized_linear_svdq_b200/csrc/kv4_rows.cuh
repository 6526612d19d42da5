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
  s.keys = kv4_min(kv4_max(kv_len[b], 0), capacity);
  return s;
}

// Keys that token i of the n of a request sees.
KV4_HD int keys_seen(int keys, int n, int i, int causal) {
  return causal ? kv4_max((long long)keys - n + i + 1, 0) : keys;
}

// Number of row tiles to launch: exact without q_start, an upper bound with it
// (sum of ceil(n_b group / rows) with sum of n_b = tokens).
KV4_HD long long max_row_tiles(int tokens, int requests, int group, int rows, bool ragged) {
  if (!ragged) return requests * (((long long)(tokens / requests) * group + rows - 1) / rows);
  return ((long long)tokens * group + (long long)requests * (rows - 1)) / rows;
}

// Parts of the key axis that a tile with `last_key` keys uses.
KV4_HD int active_parts(int last_key, int splits, int chunk) {
  const int need = last_key > 0 ? (last_key - 1) / chunk + 1 : 1;
  return need < splits ? need : splits;
}

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
  const long long row0 = tile * tile_rows, all = (long long)s.n * group;
  r.row0 = (int)row0;
  r.rows = row0 < all ? kv4_min(tile_rows, all - row0) : 0;
  r.last_key = r.rows > 0 ? keys_seen(s.keys, s.n, (int)((row0 + r.rows - 1) / group), causal) : 0;
  return r;
}

// Row tile number `tile` of the launch, one thread at a time (host form).
KV4_HD RowTile find_row_tile_serial(const int* q_start, const int* kv_len, int requests, int tokens, int group,
                                    int tile_rows, long long tile, long long capacity, int causal) {
  for (int b = 0; b < requests; ++b) {
    const RequestSpan s = request_span(q_start, kv_len, requests, tokens, b, capacity);
    const long long nt = ((long long)s.n * group + tile_rows - 1) / tile_rows;
    if (tile < nt) return tile_of(s, b, group, tile_rows, tile, causal);
    tile -= nt;
  }
  RowTile r = {};
  return r;
}

// Keys that the last row of the tile sees that holds head `in_group` of query
// token `token`; -1: no request has the token.
KV4_HD int find_last_key(const int* q_start, const int* kv_len, int requests, int tokens, int token, int group,
                         int in_group, int tile_rows, long long capacity, int causal) {
  int b;
  if (q_start) {
    // The last request that starts at or before the token (starts ascend).
    int lo = 0, hi = requests;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (q_start[mid] <= token) lo = mid + 1;
      else hi = mid;
    }
    b = lo - 1;
    if (b < 0) return -1;
  } else {
    const int n = tokens / requests;
    b = n > 0 ? token / n : requests;
    if (b >= requests) return -1;
  }
  const RequestSpan s = request_span(q_start, kv_len, requests, tokens, b, capacity);
  if (token < s.token0 || token >= s.token0 + s.n) return -1;
  const long long row = (long long)(token - s.token0) * group + in_group;
  return tile_of(s, b, group, tile_rows, row / tile_rows, causal).last_key;
}

#if defined(__CUDACC__)
// The same as find_row_tile_serial, by a warp: 32 requests at a time.  Every
// lane of the warp calls it with the same arguments and gets the same answer.
__device__ __forceinline__ RowTile find_row_tile(const int* q_start, const int* kv_len, int requests, int tokens,
                                                 int group, int tile_rows, long long tile, long long capacity,
                                                 int causal) {
  if (!q_start) {
    const long long per = ((long long)(tokens / requests) * group + tile_rows - 1) / tile_rows;
    const int b = per > 0 ? (int)(tile / per) : requests;
    RowTile r = {};
    if (b >= requests) return r;
    return tile_of(request_span(nullptr, kv_len, requests, tokens, b, capacity), b, group, tile_rows, tile % per,
                   causal);
  }
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < requests; b0 += 32) {
    const int b = b0 + lane;
    long long nt = 0;
    if (b < requests) {
      const RequestSpan s = request_span(q_start, kv_len, requests, tokens, b, capacity);
      nt = ((long long)s.n * group + tile_rows - 1) / tile_rows;
    }
    long long upto = nt;                        // inclusive prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, tile < before + upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const long long first = before + __shfl_sync(0xFFFFFFFFu, upto - nt, l);
      return tile_of(request_span(q_start, kv_len, requests, tokens, b0 + l, capacity), b0 + l, group, tile_rows,
                     tile - first, causal);
    }
    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  RowTile r = {};
  return r;
}
#endif

}  // namespace svdq
