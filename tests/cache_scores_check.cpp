// score_first and scores_length of csrc/ltc_cache.h: whatever a call's sequences
// are, each one's steps lie within the room of a row's scores.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>

#include "ltc_cache.h"

int main() {
  std::mt19937_64 rng(11);
  auto pick = [&](uint64_t lo, uint64_t hi) { return lo + rng() % (hi - lo + 1); };
  long bad = 0;
  for (int i = 0; i < 2000000; ++i) {
    const uint64_t capacity = 16 * pick(1, pick(0, 1) ? 200 : (1u << 26));
    const uint32_t n = (uint32_t)pick(1, std::min<uint64_t>(capacity, pick(0, 1) ? 70 : 5000));
    const uint32_t rows = n + (uint32_t)pick(0, 3) * (uint32_t)pick(0, 500);
    const uint32_t len = (uint32_t)pick(n, capacity), start = len - n;
    const uint64_t most[] = {0, 1, 2, 200, 5000, 1u << 30, 0x7fffffffu};
    const uint64_t up = most[pick(0, 6)];
    const uint32_t window = (uint32_t)pick(up > 3 ? up - 3 : 0, up);
    const uint64_t stride = ltc::scores_length(capacity, rows, window);
    const uint32_t first = ltc::score_first(start, window);
    const uint64_t end = ((uint64_t)len + 63) / 64 * 64;  // of the last step
    const uint64_t seen = window && start + 1 > window ? start + 1 - window : 0;
    bad += first % 64 || first > seen || seen - first >= 64;
    bad += end - first > stride || stride % 64;
    bad += stride > (capacity + 63) / 64 * 64 || (window && stride > (uint64_t)window + rows + 192);
  }
  std::printf(bad ? "%ld wrong\n" : "ok\n", bad);
  return bad != 0;
}
