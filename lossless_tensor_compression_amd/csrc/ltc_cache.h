// ltc_cache.h -- the paged key/value cache: what a kernel is given, and
// the index arithmetic that turns a workgroup's number into a sequence, its
// rows and the pages under them.  Everything here runs on the host too, so
// that it can be checked there against bad tables, lengths and row offsets.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define LTC_HD __host__ __device__ __forceinline__
#else
#define LTC_HD inline
#endif

namespace ltc {

// bits of the cache's status word
constexpr uint32_t kCacheBadPage = 1;  // a table entry outside [0, pages)
constexpr uint32_t kCacheBadSeq = 2;   // lengths or row offsets that contradict each other

struct CacheView {
  uint8_t* k;        // [pages][heads][page/16][dim/16][16 tokens][16 dims]; of 4 bits [dim/32][16 tokens][32 dims]
  uint8_t* v;        // [pages][heads][page/16][dim][16 tokens]
  uint8_t* scales;   // [pages][heads][2], 2^(byte - 127); of 4 bits see token_scales
  uint32_t* status;  // one word, bits above
  uint32_t pages, heads, dim;
  uint32_t page_log;  // log2 of a page's tokens
};

struct SeqView {
  const int32_t* table;    // [seqs][width], page of tokens [j << page_log, (j + 1) << page_log)
  const int32_t* lengths;  // [seqs]
  const int32_t* cu;       // [seqs + 1] row offsets; null: one row per sequence
  uint64_t table_stride;
  uint32_t seqs, rows, width;
};

// A sequence's rows in the call and the positions they stand for.
struct Span {
  uint32_t row0, n;  // rows [row0, row0 + n)
  uint32_t len;      // positions the sequence has; the rows are its last n
  uint32_t start;    // len - n
  bool ok;           // false: the numbers contradict each other; then len = start = 0
};

LTC_HD uint32_t clip_rows(int32_t c, uint32_t rows) {
  return c < 0 ? 0 : ((uint32_t)c < rows ? (uint32_t)c : rows);
}

LTC_HD Span span_of(int32_t c0, int32_t c1, int32_t length, uint32_t rows, uint64_t capacity) {
  Span s;
  s.row0 = clip_rows(c0, rows);
  const uint32_t r1 = clip_rows(c1, rows);
  s.n = r1 > s.row0 ? r1 - s.row0 : 0;
  s.ok = c0 >= 0 && c1 >= c0 && (uint32_t)c1 <= rows && length >= 0 && (uint64_t)length <= capacity &&
         length >= c1 - c0;
  s.len = s.ok ? (uint32_t)length : 0;
  s.start = s.ok ? s.len - s.n : 0;
  return s;
}

// Workgroups are numbered so that a workgroup finds its sequence without
// knowing any count but the rows and sequences of the call: sequence i's
// units begin at first(i) = clip(cu[i]) * mul / div + extra * i, a
// nondecreasing map, and the caller picks mul, div and extra so that
// first(i + 1) - first(i) covers what sequence i can need (the rest of the
// numbers find no work).  Pages of P tokens under n rows: at most
// floor((n - 2) / P) + 2, so mul = 1, div = P, extra = 2.  Tiles of R of n * G
// rows: ceil(n * G / R), so mul = G, div = R, extra = 1.
struct UnitMap {
  uint32_t mul, div, extra;
};

LTC_HD uint64_t unit_first(const UnitMap& m, uint32_t cu_clipped, uint32_t i) {
  return (uint64_t)cu_clipped * m.mul / m.div + (uint64_t)m.extra * i;
}

LTC_HD uint64_t unit_count(const UnitMap& m, uint32_t rows, uint32_t seqs) {
  return (uint64_t)rows * m.mul / m.div + (uint64_t)m.extra * seqs;
}

// Which head, unit and split workgroup `id` of an attention takes.  Workgroups
// go to the eight chiplets in turn, and a chiplet's L2 holds what its workgroups
// read: so the heads are shared out over the chiplets, as far as a power of two
// divides them, and chiplets that have heads in common take every share-th of
// their units.  The last units come first: a long prompt's last rows see the
// most.  share divides per_head, the units times splits of a head and a few
// numbers without work (unit too large; head too large behind them all).
LTC_HD uint32_t chiplet_share(uint32_t heads) {
  return heads % 8 == 0 ? 1 : heads % 4 == 0 ? 2 : heads % 2 == 0 ? 4 : 8;
}
LTC_HD void place(uint32_t id, uint32_t heads, uint32_t splits, uint32_t per_head, uint32_t* head, uint32_t* unit,
                  uint32_t* split) {
  const uint32_t share = chiplet_share(heads), classes = 8 / share;
  const uint32_t chiplet = id % 8, i = id / 8 * share + chiplet / classes;
  *head = chiplet % classes + i / per_head * classes;
  const uint32_t x = per_head - 1 - i % per_head;
  *unit = x / splits;
  *split = x % splits;
}

// The last sequence whose units begin at or before `unit`, in steps of 64:
// count(lo, step, n) says at how many of lo, lo + step, ... (64 at most, below
// lo + n) first() is at most `unit`; on the GPU a wave asks all 64 at once.
template <class Count>
LTC_HD uint32_t find_sequence(uint32_t seqs, Count count) {
  uint32_t lo = 0, n = seqs;
  while (n > 1) {
    const uint32_t step = (n + 63) / 64;
    const uint32_t c = count(lo, step, n);
    const uint32_t skip = c > 1 ? (c - 1) * step : 0;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return lo;
}

// Positions stay below 2^30, so that sums of them and steps past the end fit
// 32 bits.
constexpr uint64_t kMaxPositions = 1u << 30;

LTC_HD uint64_t capacity_of(const CacheView& c, const SeqView& s) {
  const uint64_t capacity = (uint64_t)s.width << c.page_log;
  return capacity < kMaxPositions ? capacity : kMaxPositions;
}

LTC_HD Span load_span(const CacheView& c, const SeqView& s, uint32_t seq) {
  const int32_t c0 = s.cu ? s.cu[seq] : (int32_t)seq, c1 = s.cu ? s.cu[seq + 1] : (int32_t)seq + 1;
  return span_of(c0, c1, s.lengths[seq], s.rows, capacity_of(c, s));
}

// Whether one of the positions [t0, t1) is hidden from one of the rows at positions
// first .. last.  (t0 + window may pass 2^31.)
LTC_HD bool some_hidden(int t0, int t1, int first, int last, uint32_t window) {
  return t1 > first + 1 || (window && last - t0 >= (int)window);
}

// Scores that an attention writes down, for each row and query head: those of the
// positions from score_first on, which is in order for the sequence's first row and a
// step's first; scores_length holds them whatever the lengths are.
constexpr uint32_t kScoreStep = 64;
LTC_HD uint32_t score_first(uint32_t start, uint32_t window) {
  const uint32_t first = window && start + 1 > window ? start + 1 - window : 0;
  return first / kScoreStep * kScoreStep;
}
LTC_HD uint64_t scores_length(uint64_t capacity, uint32_t rows, uint32_t window) {
  const uint64_t seen = (uint64_t)window + rows + 2 * kScoreStep, most = window && seen < capacity ? seen : capacity;
  return (most + kScoreStep - 1) / kScoreStep * kScoreStep;
}

// What a unit loads besides its own sequence's numbers, early and without
// branches, so that it comes with other loads: the ends of the row offsets, and
// the numbers of the sequence that it checks (check_sequence).
struct Early {
  int32_t first, last;
  int32_t c0, c1, length;
};

LTC_HD Early load_early(const SeqView& s, uint64_t unit) {
  const uint32_t i = unit < s.seqs ? (uint32_t)unit : s.seqs - 1;
  const int32_t* p = s.cu ? s.cu : s.lengths;
  const uint32_t end = s.cu ? s.seqs : 0, c0 = s.cu ? i : 0, c1 = s.cu ? i + 1 : 0;
  return {p[0], p[end], p[c0], p[c1], s.lengths[i]};
}

// Whether the sequence of the unit's own number is in order.  A search over row
// offsets that decrease may pass by the sequence at fault, and a call has at
// least as many units as sequences: so all are checked.
LTC_HD bool check_sequence(const CacheView& c, const SeqView& s, const Early& e) {
  return !s.cu || span_of(e.c0, e.c1, e.length, s.rows, capacity_of(c, s)).ok;
}

// Rows of the call that belong to no sequence, [0, before) and [behind, rows):
// a call of a fixed number of rows may have fewer sequences' rows in it.
struct Unnamed {
  uint32_t before, behind, n;
};

LTC_HD Unnamed unnamed_rows(const SeqView& s, const Early& e) {
  const uint32_t before = s.cu ? clip_rows(e.first, s.rows) : 0, end = s.cu ? clip_rows(e.last, s.rows) : s.rows;
  const uint32_t behind = end > before ? end : before;
  return {before, behind, before + (s.rows - behind)};
}

LTC_HD uint32_t unnamed_row(const Unnamed& u, uint32_t i) { return i < u.before ? i : u.behind + (i - u.before); }

LTC_HD uint64_t unit_first(const UnitMap& m, const SeqView& s, uint32_t seq) {
  return unit_first(m, s.cu ? clip_rows(s.cu[seq], s.rows) : seq, seq);
}

// The unit's sequence, its span and the unit's number within the sequence's
// own; false if the number is no unit of it (its rows are none, or row
// offsets that decrease).  What the number can be at most is the caller's.
template <class Count>
LTC_HD bool locate_unit(const CacheView& c, const SeqView& s, const UnitMap& m, uint64_t unit, Count count,
                        uint32_t* seq, Span* sp, uint64_t* own) {
  *seq = find_sequence(s.seqs, count);
  *sp = load_span(c, s, *seq);
  const uint64_t first = unit_first(m, sp->row0, *seq);
  *own = unit - first;
  return sp->n != 0 && unit >= first;
}

// Bytes from the start of k (or v) to the codes of a page and head; 64 bits,
// since a cache passes 4 GiB.
LTC_HD uint64_t head_offset(const CacheView& c, uint32_t page, uint32_t head) {
  return (((uint64_t)page * c.heads + head) * c.dim) << c.page_log;
}

// A cache of 4-bit codes: half of head_offset's bytes, and for each page and head
// the exponents of the tokens' keys, those of their values (a byte each, 2^(byte -
// 127)), and drop_bytes for each token: nibble j, the lowest first, is how far
// below the token's the exponent of its key's dims 32 j .. 32 j + 31 lies.
constexpr int kMostDrop = 15;
LTC_HD constexpr uint32_t drop_bytes(uint32_t dim) { return dim <= 64 ? 1 : dim <= 128 ? 2 : 4; }
LTC_HD uint64_t token_scales(const CacheView& c, uint32_t page, uint32_t head) {
  return (((uint64_t)page * c.heads + head) * (2 + drop_bytes(c.dim))) << c.page_log;
}

// Within a page and head: the code of token t (0 <= t < page) and dim d.
LTC_HD uint32_t k_code(uint32_t t, uint32_t d, uint32_t dim) {
  return (t >> 4) * 16 * dim + (d >> 4) * 256 + (t & 15) * 16 + (d & 15);
}
LTC_HD uint32_t v_code(uint32_t t, uint32_t d, uint32_t dim) {
  return (t >> 4) * 16 * dim + d * 16 + (t & 15);
}

// The table's entry for a position below len; false if it names no page.
LTC_HD bool page_at(const SeqView& s, uint32_t seq, uint32_t page_index, uint32_t pages, uint32_t* page) {
  if (page_index >= s.width) return false;
  const int32_t p = s.table[seq * s.table_stride + page_index];
  if (p < 0 || (uint32_t)p >= pages) return false;
  *page = (uint32_t)p;
  return true;
}

// 2^e for the exponents of scales: exact in -126..127; 2^-127 (byte 0) is 0
// and 2^128 (byte 255) infinity.
LTC_HD float power_of_two(int e) {
  union {
    uint32_t u;
    float f;
  } x;
  x.u = (uint32_t)(e + 127) << 23;
  return x.f;
}

// The least e >= kLowestScale with largest <= top * 2^e, as a scale's byte.
// top is 448 = 0.875 * 2^9 for E4M3 codes and 127 = 127/128 * 2^7 for INT8.
constexpr int kLowestScale = -100;
LTC_HD uint32_t scale_byte(float largest, bool e4m3) {
  union {
    float f;
    uint32_t u;
  } x;
  x.f = largest;
  const uint32_t mantissa = x.u & 0x7fffff;
  const int e = (int)(x.u >> 23) - 126;  // largest = 0.5..1 times 2^e; subnormal: far below the lowest
  const int s = e4m3 ? (mantissa <= 0x600000 ? e - 9 : e - 8) : (mantissa <= 0x7e0000 ? e - 7 : e - 6);
  return (uint32_t)((s < kLowestScale ? kLowestScale : s) + 127);
}

// The least e with largest <= 6 * 2^e = 0.75 * 2^(e + 3), the top of E2M1's codes;
// of 0 one that is below all others.
LTC_HD int e2m1_exponent(float largest) {
  union {
    float f;
    uint32_t u;
  } x;
  x.f = largest;
  const int e = (int)(x.u >> 23) - 126;
  return (x.u & 0x7fffff) <= 0x400000 ? e - 3 : e - 2;
}

}  // namespace ltc
