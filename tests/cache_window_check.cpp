// some_hidden of csrc/ltc_cache.h against its definition, position by position and
// row by row, and at the ends of what windows and positions can be.
#include <cstdint>
#include <cstdio>

#include "ltc_cache.h"

static bool hidden(int64_t t0, int64_t t1, int64_t first, int64_t last, int64_t window) {
  for (int64_t t = t0; t < t1; ++t)
    for (int64_t row = first; row <= last; ++row)
      if (t > row || (window && t <= row - window)) return true;
  return false;
}

int main() {
  long bad = 0;
  for (int first = 0; first < 14; ++first)
    for (int last = first; last < first + 4; ++last)
      for (int t0 = 0; t0 < 14; ++t0)
        for (unsigned window = 0; window < 16; ++window)
          bad += ltc::some_hidden(t0, t0 + 3, first, last, window) != hidden(t0, t0 + 3, first, last, window);
  // a window that no row's position reaches hides nothing, however far the step
  const int far[] = {0, 63, 64, 128, 1 << 20, (1 << 30) - 128};
  const unsigned most = 0x7fffffffu;
  for (int t0 : far) {
    bad += ltc::some_hidden(t0, t0 + 64, t0 + 63, t0 + 78, most);
    bad += ltc::some_hidden(t0, t0 + 64, t0 + 63, t0 + 78, most - 1);
    bad += !ltc::some_hidden(t0, t0 + 64, t0 + 62, t0 + 78, most);
  }
  bad += ltc::some_hidden(0, 64, (1 << 30) - 1, (1 << 30) - 1, 1u << 30);
  bad += !ltc::some_hidden(0, 64, (1 << 30) - 1, (1 << 30) - 1, (1u << 30) - 1);
  std::printf(bad ? "%ld wrong\n" : "ok\n", bad);
  return bad != 0;
}
