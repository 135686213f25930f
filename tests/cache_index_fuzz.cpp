// cache_index_fuzz.cpp -- the key/value cache's index arithmetic
// (csrc/ltc_cache.h) on the CPU: every unit of calls with good and with bad
// tables, lengths and row offsets is walked as the kernels walk it, reading
// and writing buffers of exactly the sizes a caller has to bring.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "ltc_cache.h"

using namespace ltc;

static std::mt19937_64 rng(7);
static uint32_t pick(uint32_t lo, uint32_t hi) { return lo + (uint32_t)(rng() % (hi - lo + 1)); }

#define CHECK(x)                                          \
  do {                                                    \
    if (!(x)) {                                           \
      printf("%s:%d: %s\n", __FILE__, __LINE__, #x);      \
      exit(1);                                            \
    }                                                     \
  } while (0)

// the wave's 64 questions in a loop
struct LoopCount {
  const SeqView& s;
  const UnitMap& m;
  uint64_t unit;
  uint32_t operator()(uint32_t lo, uint32_t step, uint32_t n) const {
    uint32_t c = 0;
    for (uint32_t l = 0; l < 64; ++l)
      if (l * step < n && unit_first(m, s, lo + l * step) <= unit) ++c;
    return c;
  }
};

static void walk(bool bad, bool single) {
  CacheView c = {};
  c.page_log = pick(4, 8);
  const uint32_t P = 1u << c.page_log;
  c.heads = pick(1, 2);
  c.dim = 64;
  const uint32_t seqs = pick(1, pick(1, 300));
  std::vector<int32_t> lengths(seqs), cu(seqs + 1);
  uint32_t need = 0, width = 1;
  for (uint32_t i = 0; i < seqs; ++i) {
    const uint32_t n = single ? 1 : (pick(0, 3) ? pick(0, 3 * P) : 0);
    lengths[i] = (int32_t)(n + pick(0, 3 * P));
    cu[i + 1] = cu[i] + (int32_t)n;
    const uint32_t pages = ((uint32_t)lengths[i] + P - 1) / P;
    need += pages;
    width = std::max(width, pages);
  }
  const uint32_t rows = (uint32_t)cu[seqs];
  c.pages = need + 1;
  std::vector<int32_t> order(c.pages), table((size_t)seqs * width);
  for (uint32_t i = 0; i < c.pages; ++i) order[i] = (int32_t)i;
  std::shuffle(order.begin(), order.end(), rng);
  for (uint32_t i = 0, at = 0; i < seqs; ++i)
    for (uint32_t j = 0; j < width; ++j)
      table[(size_t)i * width + j] = j < ((uint32_t)lengths[i] + P - 1) / P ? order[at++] : (int32_t)rng();
  if (bad) {
    for (int k = pick(0, 4); k > 0; --k) table[rng() % table.size()] = (int32_t)rng();
    for (int k = pick(0, 3); k > 0; --k) lengths[rng() % seqs] = pick(0, 1) ? (int32_t)rng() : (int32_t)pick(0, 4 * P * width);
    if (!single)
      for (int k = pick(0, 3); k > 0; --k) cu[rng() % (seqs + 1)] = pick(0, 1) ? (int32_t)rng() : (int32_t)pick(0, rows + 3);
  }
  // exact allocations: the sanitizer sees any step outside
  std::vector<uint8_t> codes((size_t)c.pages * c.heads * c.dim * P);
  std::vector<uint16_t> out((size_t)rows * c.heads * c.dim);
  c.k = c.v = codes.data();
  SeqView s = {table.data(), lengths.data(), single ? nullptr : cu.data(), width, seqs, rows, width};
  const UnitMap m = single ? UnitMap{0, 1, 1} : UnitMap{1, P, 2};
  std::vector<int> row_seen(rows), page_seen(c.pages);
  for (uint64_t u = 0; u < unit_count(m, rows, seqs); ++u) {
    uint32_t seq;
    Span sp;
    uint64_t j;
    if (!locate_unit(c, s, m, u, LoopCount{s, m, u}, &seq, &sp, &j)) continue;
    CHECK(seq < seqs && sp.row0 + sp.n <= rows && (!sp.ok || sp.len <= (uint64_t)width * P));
    j += sp.start >> c.page_log;
    const uint32_t last = sp.start + sp.n - 1;
    if (j > (last >> c.page_log)) continue;
    uint32_t page = 0;
    const bool have = sp.ok && page_at(s, seq, (uint32_t)j, c.pages, &page);
    if (!bad) CHECK(have);
    const uint32_t first = (uint32_t)j << c.page_log;
    const uint32_t t0 = sp.start > first ? sp.start - first : 0, t1 = std::min(last - first + 1, P);
    CHECK(t0 < t1 && t1 <= P);
    if (have) ++page_seen[page];
    for (uint32_t t = t0; t < t1; ++t) {
      const uint32_t row = sp.row0 + (first + t - sp.start);
      ++row_seen[row];
      for (uint32_t h = 0; h < c.heads; ++h) {
        out[((size_t)row * c.heads + h) * c.dim + c.dim - 1] = 1;
        if (!have) continue;
        for (uint32_t d = 0; d < c.dim; d += 21) {
          codes[head_offset(c, page, h) + k_code(t, d, c.dim)] = 1;
          codes[head_offset(c, page, h) + v_code(t, d, c.dim)] = 1;
        }
      }
    }
  }
  if (!bad) {
    for (int n : row_seen) CHECK(n == 1);
    for (int n : page_seen) CHECK(n <= 1);
  }
  // rows of packed heads in tiles
  const uint32_t G = pick(1, 16), R = 1u << pick(4, 7);
  const UnitMap mt = single ? UnitMap{0, 1, (G + R - 1) / R} : UnitMap{G, R, 1};
  std::vector<int> packed((size_t)rows * G);
  for (uint64_t u = 0; u < unit_count(mt, rows, seqs); ++u) {
    uint32_t seq;
    Span sp;
    uint64_t tile;
    if (!locate_unit(c, s, mt, u, LoopCount{s, mt, u}, &seq, &sp, &tile) || tile * R >= (uint64_t)sp.n * G) continue;
    for (uint64_t r = tile * R; r < std::min<uint64_t>((tile + 1) * R, (uint64_t)sp.n * G); ++r)
      ++packed[(size_t)sp.row0 * G + r];
  }
  if (!bad)
    for (int n : packed) CHECK(n == 1);
}

static void layouts() {
  const uint32_t dims[] = {64, 96, 128, 192, 256};
  for (uint32_t dim : dims)
    for (uint32_t P = 16; P <= 256; P *= 2) {
      std::vector<int> k(P * dim), v(P * dim);
      for (uint32_t t = 0; t < P; ++t)
        for (uint32_t d = 0; d < dim; ++d) ++k[k_code(t, d, dim)], ++v[v_code(t, d, dim)];
      for (size_t i = 0; i < k.size(); ++i) CHECK(k[i] == 1 && v[i] == 1);
    }
  CacheView c = {};
  c.pages = 1u << 30, c.heads = 16, c.dim = 256, c.page_log = 8;
  CHECK(head_offset(c, c.pages - 1, 15) == (((uint64_t)(c.pages - 1) * 16 + 15) << 16));
  for (int e = -126; e < 128; ++e) {
    double want = 1;
    for (int i = 0; i < (e < 0 ? -e : e); ++i) want *= e < 0 ? 0.5 : 2.0;
    CHECK((double)power_of_two(e) == want);
  }
  for (int i = 0; i < 200000; ++i) {
    union { uint32_t u; float f; } x;
    x.u = (uint32_t)rng() & 0x7fffffff;
    if (pick(0, 3) == 0) x.u = (x.u & 0x7f800000) | (pick(0, 1) ? 0x600000 : 0x7e0000) + pick(0, 2) - 1;
    if ((x.u >> 23) == 255) continue;
    for (int e4m3 = 0; e4m3 < 2; ++e4m3) {
      const int e = (int)scale_byte(x.f, e4m3) - 127;
      const double top = e4m3 ? 448 : 127;
      CHECK(e >= kLowestScale && e <= 127);
      auto fits = [&](int q) { return (double)x.f <= top * (q < 0 ? 1.0 / power_of_two(-q) : (double)power_of_two(q)); };
      CHECK(fits(e) && (e == kLowestScale || !fits(e - 1)));
    }
  }
}

int main() {
  layouts();
  for (int i = 0; i < 3000; ++i) walk(i % 2, (i / 2) % 3 == 0);
  printf("ok\n");
  return 0;
}
