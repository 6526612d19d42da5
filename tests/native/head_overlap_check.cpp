// Host check of head_overlap.h: the answer for two strided tensors of heads
// against one byte map of each.
#include "head_overlap.h"

#include <cstdio>
#include <random>
#include <vector>

using namespace svdq;

static void mark(const HeadRuns& r, std::vector<char>& map, char bit) {
  for (long long t = 0; t < r.tokens; ++t)
    for (long long h = 0; h < r.heads; ++h)
      for (long long i = 0; i < r.bytes; ++i) map[r.at + t * r.token_stride + h * r.head_stride + i] |= bit;
}

int main() {
  std::mt19937 rng(5);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  long long meet = 0;
  const int trials = 60000;
  for (int trial = 0; trial < trials; ++trial) {
    HeadRuns r[2];
    const int packed = pick(0, 3);                // slices of one packed buffer more often than not
    const long long bytes = pick(1, 6), wide = pick(1, 8), token = packed == 1 ? bytes : bytes * wide;
    const long long head = packed == 1 ? bytes * pick(1, 7) : bytes;
    for (HeadRuns& x : r) {
      x.tokens = pick(1, 6);
      x.heads = pick(1, 5);
      x.bytes = bytes;
      x.token_stride = token;
      x.head_stride = head * (pick(0, 3) ? 1 : pick(0, 3));
      x.at = pick(0, 5) * bytes + (pick(0, 2) ? 0 : pick(0, 9)) + pick(0, 4) * token;
      if (packed == 3) {                          // anything
        x.bytes = pick(1, 20);
        x.token_stride = pick(0, 30);
        x.head_stride = pick(0, 30);
        x.at = pick(0, 120);
      }
    }
    std::vector<char> map(2000, 0);
    mark(r[0], map, 1);
    mark(r[1], map, 2);
    bool want = false;
    for (char c : map) want |= c == 3;
    meet += want;
    if (runs_overlap(r[0], r[1]) != want || runs_overlap(r[1], r[0]) != want) {
      std::printf("FAILED case %d: want %d\n", trial, (int)want);
      return 1;
    }
  }
  // Both answers occur often.
  if (meet < trials / 10 || meet > trials - trials / 10) {
    std::printf("FAILED: %lld of %d overlap\n", meet, trials);
    return 1;
  }
  std::printf("ok\n");
  return 0;
}
