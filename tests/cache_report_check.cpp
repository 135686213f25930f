// Calls of the key/value cache whose row offsets leave rows out, decrease or
// pass the call's rows: some unit finds each sequence that is refused, whatever
// its numbering, and rows that no sequence has are cleared once, no others.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "ltc_cache.h"

using namespace ltc;

static std::mt19937_64 rng(5);
static uint32_t pick(uint32_t lo, uint32_t hi) { return lo + (uint32_t)(rng() % (hi - lo + 1)); }

#define CHECK(x)                                          \
  do {                                                    \
    if (!(x)) {                                           \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x); \
      std::exit(1);                                       \
    }                                                     \
  } while (0)

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

static long refused, passed_by;

static void call(bool bad) {
  const uint32_t seqs = pick(1, pick(1, 200)), most = pick(0, 60);
  std::vector<int32_t> lengths(seqs), cu(seqs + 1);
  cu[0] = pick(0, 2) ? 0 : (int32_t)pick(0, 100);
  for (uint32_t i = 0; i < seqs; ++i) {
    cu[i + 1] = cu[i] + (int32_t)pick(0, most);
    lengths[i] = cu[i + 1] - cu[i] + (int32_t)pick(0, 300);
  }
  const uint32_t rows = (uint32_t)cu[seqs] + (pick(0, 2) ? 0 : pick(0, 100));
  if (bad) {
    for (int k = pick(1, 2); k > 0; --k) cu[rng() % (seqs + 1)] = pick(0, 3) ? (int32_t)pick(0, rows + 3) : (int32_t)rng();
    if (!pick(0, 3)) lengths[rng() % seqs] = (int32_t)rng();
  }
  CacheView c = {};
  c.page_log = pick(4, 8);
  SeqView s = {nullptr, lengths.data(), cu.data(), 30, seqs, rows, 30};
  const uint32_t G = pick(1, 16);
  const UnitMap maps[] = {{1, 1u << c.page_log, 2}, {G, 16, 1}, {G, 32, 1}, {G, 128, 1}};
  bool any = false;
  for (uint32_t i = 0; i < seqs; ++i) any = any || !load_span(c, s, i).ok;
  for (const UnitMap& m : maps) {
    bool reported = false, searched = false;
    for (uint64_t u = 0; u < unit_count(m, rows, seqs); ++u) {
      uint32_t seq;
      Span sp;
      uint64_t own;
      locate_unit(c, s, m, u, LoopCount{s, m, u}, &seq, &sp, &own);
      searched = searched || !sp.ok;
      reported = reported || !sp.ok || !check_sequence(c, s, load_early(s, u));
    }
    CHECK(reported == any);
    refused += any;
    passed_by += any && !searched;
  }
  const Unnamed none = unnamed_rows(s, load_early(s, 0));
  std::vector<int> taken(rows);
  for (uint32_t i = 0; i < none.n; ++i) {
    CHECK(unnamed_row(none, i) < rows);
    ++taken[unnamed_row(none, i)];
  }
  for (int n : taken) CHECK(n <= 1);
  if (bad) return;
  for (uint32_t i = 0; i < seqs; ++i)
    for (int32_t r = cu[i]; r < cu[i + 1]; ++r) ++taken[r];
  for (int n : taken) CHECK(n == 1);
}

int main() {
  for (int i = 0; i < 20000; ++i) call(i % 2);
  SeqView s = {nullptr, nullptr, nullptr, 0, 3, 3, 0};
  const int32_t lengths[] = {1, 2, 3};
  s.lengths = lengths;
  CHECK(unnamed_rows(s, load_early(s, 2)).n == 0);
  // the check is not idle: a search alone passes some of them by
  CHECK(refused > 10000 && passed_by > 0);
  std::printf("%ld of %ld refused calls passed by the search alone: ok\n", passed_by, refused);
  return 0;
}
