// The 4-bit cache's host arithmetic: exponents against their definition for every
// number of both types, and that a cache's last byte is its arrays' last.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "ltc_cache.h"

static float bf16(unsigned u) {
  u <<= 16;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}

static float fp16(unsigned u) {
  const int e = (int)(u >> 10), m = (int)(u & 1023);
  return e ? std::ldexp((float)(1024 + m), e - 25) : std::ldexp((float)m, -24);
}

int main() {
  long bad = 0;
  auto check = [&](float x) {
    if (x == 0.0f) {
      bad += ltc::e2m1_exponent(x) > -120;  // below all others, whatever the clamp
      return;
    }
    const int e = ltc::e2m1_exponent(x);
    if (x < 0x1p-126f) {  // a subnormal number: far below the lowest exponent
      bad += e > -120;
      return;
    }
    bad += !((double)x <= std::ldexp(6.0, e) && (double)x > std::ldexp(6.0, e - 1));
  };
  for (unsigned u = 0; u < 0x7f80; ++u) check(bf16(u));
  for (unsigned u = 0; u < 0x7c00; ++u) check(fp16(u));
  const unsigned dims[] = {64, 96, 128, 192, 256};
  for (unsigned dim : dims)
    for (unsigned page_log = 4; page_log <= 8; ++page_log) {
      ltc::CacheView c = {};
      c.pages = 70001;
      c.heads = 9;
      c.dim = dim;
      c.page_log = page_log;
      const unsigned long long page = 1ull << page_log, all = 1ull * c.pages * c.heads;
      // codes: the last block of 16 tokens, its last dims
      const unsigned long long last = ltc::head_offset(c, c.pages - 1, c.heads - 1) / 2 + (page / 16 - 1) * 8 * dim;
      bad += last + (dim / 32 - 1) * 256 + 15 * 16 + 16 != all * page * dim / 2;  // keys
      bad += last + (dim - 1) * 8 + 8 != all * page * dim / 2;                    // values
      const unsigned long long drops = ltc::drop_bytes(dim);
      bad += 8 * drops < 4 * (dim / 32);
      bad += ltc::token_scales(c, c.pages - 1, c.heads - 1) + 2 * page + (page - 1) * drops + drops != all * page * (2 + drops);
      bad += ltc::token_scales(c, 1, 1) % 16 != 0;  // 16 tokens' bytes are read at once
    }
  std::printf(bad ? "%ld wrong\n" : "ok\n", bad);
  return bad != 0;
}
