// ltc_cache_attend.hip -- attention of new queries over the 8-bit cache.
//
// One pass over the positions with the softmax's running maximum and sum.
// Per head, with x_t = log2(e) scale (q . k_t) and 2^w the scale of token t's
// values (its page's):
//   out = sum_t 2^(x_t) 2^w c_t / sum_t 2^(x_t),   c_t the value's codes.
// The weights u_t = 2^(x_t + w - m) carry the values' scale, m is a running
// bound of x_t + w (not below its maximum by more than kSlack), and the sum
// below the fraction gathers u_t 2^-w: so the weights that multiply the codes
// have one range whatever the pages' scales are, and the codes go into the
// matrix cores as they are.  The matrix cores get 2^kHead u_t, rounded to fp16.
#include <type_traits>

#include "ltc_cache_device.h"

namespace ltc {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
// A step whose largest x + w is within kSlack of the running bound keeps the
// bound, so the accumulators are seldom scaled.
constexpr int kSlack = 6;
// Far from zero the bound and the sums with it are rounded to steps of 2^-23 of
// it: it is put four to eight steps higher, so that no weight passes fp16's top.
// Past 2^26 that takes all of a weight's bits.
constexpr float kFar = 0x1p-21f;
// Weights meet the codes times 2^kHead, which puts the largest at 2^15, below
// fp16's top.  A position that takes nearly all of the weight may have values
// near zero, and then the output is what thousands of far smaller weights make
// of theirs: these keep 11 bits down to 2^-(14 + kHead) of the bound and are lost
// at 2^-(25 + kHead).  kSlack 6 / 4 / 2 / 1: two prompts of 2,500-4,096 rows 648 /
// 652 / 657 / 661 us, others the same.
constexpr int kHead = 15 - kSlack;

// Eight codes (two dwords) as fp16, exactly: E4M3 has 3 bits of mantissa and
// exponents down to 2^-9, INT8 7 bits.
template <bool E4M3> __device__ __forceinline__ half8 codes_to_half(uint32_t a, uint32_t b) {
  union {
    half8 h8;
    half2v h2[4];
    uint32_t u[4];
  } r;
  if constexpr (E4M3) {
    r.h2[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)a, 1.0f, false);
    r.h2[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)a, 1.0f, true);
    r.h2[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b, 1.0f, false);
    r.h2[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b, 1.0f, true);
  } else {
    // 0x6400 | u is 1024 + u in fp16; u = code + 128
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    r.u[0] = __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u);
    r.u[1] = __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u);
    r.u[2] = __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u);
    r.u[3] = __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u);
    const half2v off = {(_Float16)1152, (_Float16)1152};
    for (int i = 0; i < 4; ++i) r.h2[i] -= off;
  }
  return r.h8;
}

// Whether any of four E4M3 codes is a NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// The positions that a tile of packed rows looks at, in steps of kStep, and
// how they are shared out: split i takes steps [i * per, (i + 1) * per).
constexpr int kStep = 64;
struct Range {
  int lo, hi;            // positions [lo, hi) that some row sees
  int first, steps;      // steps first .. first + steps cover them
  int per, used;         // steps of a split, splits with work
};

__device__ __forceinline__ Range range_of(const Span& sp, uint32_t tok0, uint32_t tok1, uint32_t window,
                                          uint32_t splits, int least) {
  Range r;
  r.hi = (int)(sp.start + tok1);
  r.lo = (int)(sp.start + tok0) + 1 - (int)window;
  if (!window || r.lo < 0) r.lo = 0;
  r.first = r.lo / kStep;
  r.steps = (r.hi + kStep - 1) / kStep - r.first;
  r.per = max(least, (int)((r.steps + splits - 1) / splits));
  r.used = (r.steps + r.per - 1) / r.per;
  return r;
}

// The workspace: kCounters counters, all zero between calls, then the splits'
// partial results: [unit][head][split][row of the tile] numerators (dim
// floats), and bound and sum (2 floats) in an array behind them.
constexpr uint32_t kCounters = 16384;
constexpr uint64_t kCounterBytes = kCounters * 4;

// Partial results travel between workgroups of any chiplet through atomic
// accesses of the device's scope, which go past the chiplet's own L2.  The
// writer's are waited for (wait_stores) before its counter is raised, so no
// fence has to write an L2 back: with __threadfence() in every workgroup the
// call of 64 rows at 1,000-6,000 positions took 462 us where it took 115.
__device__ __forceinline__ void put2(float* p, float a, float b) {
  const float2v x = {a, b};
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, x), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2v get2(const float* p) {
  return __builtin_bit_cast(float2v, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                                       __HIP_MEMORY_SCOPE_AGENT));
}
__device__ __forceinline__ void wait_stores() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

__device__ __forceinline__ uint32_t pack2_as(bool bf16, float a, float b) {
  return bf16 ? pack2<LTC_BF16>(a, b) : pack2<LTC_FP16>(a, b);
}

// A denominator's part from one bound to another.  Where pages' scales lie far
// apart it may be large while 2^(from - to) is below fp32's numbers: so that
// comes in two halves.
__device__ __forceinline__ float rebase(float l, float from, float to) {
  const float half = __builtin_amdgcn_exp2f(0.5f * (from - to));
  return from == to ? l : l * half * half;
}

// What a wave keeps of its 16 * NC rows; lane 16 g + n has row n of each 16.
template <int D, int NC> struct Rows {
  half8 q[NC][D / 32];     // the k-group g of the queries, times 2^up
  int up[NC];
  int lo[NC], hi[NC];      // the positions [lo, hi) that the row sees
  float4v acc[NC][D / 16]; // dims 16 i + 4 g + 0..3 of the numerator
  float m[NC], l[NC];      // bound, and the lane's part of the denominator
  uint64_t nan[NC];        // bit 4 i + j: acc[nc][i][j] met a NaN among the values
};

// Rows r0.. of a sequence and head; those from packed on are none, and see nothing.
template <int D, int NC>
__device__ __forceinline__ void load_rows(Rows<D, NC>& w, const AttendArgs& a, const Span& sp, uint32_t head, uint32_t G,
                                          uint32_t r0, uint32_t packed, bool bf16, int n, int g) {
  constexpr int KS = D / 32, KL = D / 64;
  for (int nc = 0; nc < NC; ++nc) {
    const uint32_t r = r0 + nc * 16 + n;
    const bool live = r < packed;
    const uint32_t token = live ? r / G : 0, qh = head * G + (live ? r % G : 0);
    const uint16_t* src = a.q.base + (uint64_t)(sp.row0 + token) * a.q.row_stride + (uint64_t)qh * a.q.head_stride;
    w.hi[nc] = live ? (int)(sp.start + token) + 1 : 0;
    w.lo[nc] = a.window ? max(w.hi[nc] - (int)a.window, 0) : 0;
    uint4v raw[KS];
    for (int x = 0; x < KS; ++x) {
      const int d = x < 2 * KL ? (4 * (x / 2) + g) * 16 + (x & 1) * 8 : 64 * KL + g * 8;
      raw[x] = live ? *reinterpret_cast<const uint4v*>(src + d) : uint4v{0, 0, 0, 0};
    }
    w.up[nc] = 0;
    if (bf16) {
      // to fp16 by a power of two that brings the row's largest number to
      // 2^14..2^15: what is lost is below 2^-39 of it, less than the sum's
      // own rounding in fp32
      uint32_t top = 0;
      for (int x = 0; x < KS; ++x)
        for (int i = 0; i < 4; ++i) top = max(top, max(raw[x][i] & 0x7fffu, (raw[x][i] >> 16) & 0x7fffu));
      top = max(top, (uint32_t)__shfl_xor((int)top, 16));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const int e = (int)(top >> 7);  // biased exponent; 255: infinities or NaN, which no factor helps
      w.up[nc] = e == 255 ? 0 : min(141 - e, 126);
      const float f = power_of_two(w.up[nc]);
      for (int x = 0; x < KS; ++x)
        for (int i = 0; i < 4; ++i) {
          w.q[nc][x][2 * i] = (_Float16)(widen<LTC_BF16>(raw[x][i] & 0xffffu) * f);
          w.q[nc][x][2 * i + 1] = (_Float16)(widen<LTC_BF16>(raw[x][i] >> 16) * f);
        }
    } else {
      for (int x = 0; x < KS; ++x) w.q[nc][x] = __builtin_bit_cast(half8, raw[x]);
    }
    w.m[nc] = -INFINITY;
    w.l[nc] = 0.0f;
    w.nan[nc] = 0;
    for (int i = 0; i < D / 16; ++i) w.acc[nc][i] = float4v{0, 0, 0, 0};
  }
}

// The products of a step to weights: st[nc][b][i] is the one of the token at
// tv + 4 b + i, sc the scales of the lane's 16 tokens.  edge: some row does not
// see some token, or it has no page.
template <int D, int NC>
__device__ __forceinline__ void step_weights(Rows<D, NC>& w, float4v (&st)[NC][4], half8 (&p)[NC][2], float base,
                                             uint32_t sc, int tv, bool edge, bool have) {
  const int ke = (int)(sc & 0xff) - 127, we = (int)(sc >> 8) - 127;
  const float wv = (float)we, wh = (float)(we + kHead);
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    // not 0: hidden scores are -infinity
    const float f = fmaxf(__builtin_amdgcn_ldexpf(base, ke - w.up[nc]), 0x1p-126f);
    if (edge) {
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 4; ++i) {
          const int t = tv + 4 * b + i;
          const bool seen = t >= w.lo[nc] && t < w.hi[nc] && have;
          st[nc][b][i] = seen ? st[nc][b][i] : -INFINITY;
        }
    }
    float top = st[nc][0][0];
    for (int b = 0; b < 4; ++b)
      for (int i = 0; i < 4; ++i) top = fmaxf(top, st[nc][b][i]);
    top = fmaf(top, f, wv);
    if (__any(top > fmaf(fabsf(w.m[nc]), -kFar, w.m[nc]) + kSlack)) {
      float now = fmaxf(top, __shfl_xor(top, 16));
      now = fmaxf(now, __shfl_xor(now, 32));
      now = fmaxf(fmaf(fabsf(now), kFar, now), w.m[nc]);  // -infinity: NaN, and the maximum is the other
      const float keep = now == w.m[nc] ? 1.0f : __builtin_amdgcn_exp2f(w.m[nc] - now);
      w.l[nc] = rebase(w.l[nc], w.m[nc], now);
      w.m[nc] = now;
      for (int i = 0; i < D / 16; ++i) w.acc[nc][i] *= keep;
    }
    // weights near or below fp32's smallest are nothing above the fraction, but
    // if their scale is as small they may be something below it
    const bool tiny = top < w.m[nc] - 100.0f && top > -INFINITY;
    float lift = 0.0f;
    if (__any(tiny)) {
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 4; ++i) lift += __builtin_amdgcn_exp2f(fmaf(st[nc][b][i], f, wv - top));
      lift = rebase(lift, top, w.m[nc] + wv);
    }
    // nothing seen yet: every weight is 0
    const float shift = w.m[nc] == -INFINITY ? 0.0f : wh - w.m[nc];
    float sum = 0.0f;
    for (int b = 0; b < 4; ++b)
      for (int i = 0; i < 4; ++i) {
        const float u = __builtin_amdgcn_exp2f(fmaf(st[nc][b][i], f, shift));
        sum += u;
        p[nc][b >> 1][(b & 1) * 4 + i] = (_Float16)u;
      }
    sum = __builtin_amdgcn_ldexpf(sum, -we - kHead);
    w.l[nc] += tiny ? lift : sum;
  }
}

// NaN among a step's value codes (the lane's 16 of dim 16 i + n are at
// v + 256 i): the rows that see one take note of it, by a product of
// indicators, so that the codes can lose it before they meet the weights of
// rows that do not (0 * NaN is NaN).
template <int D, int NC>
__device__ __forceinline__ void note_nan(Rows<D, NC>& w, int tv, bool have, const uint8_t* v) {
  asm volatile("" : "+v"(tv));  // nothing of this before the branch that leads here
  for (int nc = 0; nc < NC; ++nc) {
    half8 ind[2];
    for (int b = 0; b < 4; ++b)
      for (int i = 0; i < 4; ++i) {
        const int t = tv + 4 * b + i;
        ind[b >> 1][(b & 1) * 4 + i] = (_Float16)(t >= w.lo[nc] && t < w.hi[nc] && have ? 1.0f : 0.0f);
      }
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {  // a loop over memory: rare, and it must not cost registers
      const uint4v x = *reinterpret_cast<const uint4v*>(v + i * 256);
      float4v hit = {0, 0, 0, 0};
      for (int h = 0; h < 2; ++h) {
        half8 is;
        for (int j = 0; j < 8; ++j)
          is[j] = (_Float16)(nan_bytes(x[2 * h + j / 4]) >> (8 * (j & 3) + 7) & 1 ? 1.0f : 0.0f);
        hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(is, ind[h], hit, 0, 0, 0);
      }
      for (int j = 0; j < 4; ++j) w.nan[nc] |= (uint64_t)(hit[j] > 0.0f) << (4 * i + j);
    }
  }
}

template <int D, int NC> __device__ __forceinline__ void apply_nan(Rows<D, NC>& w) {
  for (int nc = 0; nc < NC; ++nc)
    if (__any(w.nan[nc] != 0))
      for (int i = 0; i < D / 16; ++i)
        for (int j = 0; j < 4; ++j)
          if (w.nan[nc] >> (4 * i + j) & 1) w.acc[nc][i][j] = __builtin_nanf("");
}

__device__ __forceinline__ uint32_t without_nan(uint32_t x) { return x & ~((nan_bytes(x) >> 7) * 0xffu); }

// dims d..d+3 of row r of the sequence and head; sum is 2^kHead times the numerator
template <int D>
__device__ __forceinline__ void store_row(const AttendArgs& a, const Span& sp, uint32_t head, uint32_t G, bool bf16,
                                          uint32_t r, int d, float4v sum, float below) {
  const uint32_t token = r / G, qh = head * G + r % G;
  const float4v o = below == 0.0f ? float4v{0, 0, 0, 0} : sum * (power_of_two(-kHead) / below);
  const uint2v out = {pack2_as(bf16, o[0], o[1]), pack2_as(bf16, o[2], o[3])};
  *reinterpret_cast<uint2v*>(a.out + ((uint64_t)(sp.row0 + token) * a.q_heads + qh) * D + d) = out;
}

// A denominator of 0 is a row that sees nothing, and keeps its zeros, or one
// whose scores are all -infinity, as an infinity in its query can make them:
// that becomes NaN.  zero: the lane's row r is one; after its zeros are stored.
template <int D>
__device__ __forceinline__ void spoil_rows(const CacheView& c, const AttendArgs& a, const Span& sp, const int32_t* table,
                                           uint32_t head, uint32_t G, uint32_t r, bool zero) {
  const int lane = threadIdx.x & 63;
  for (uint64_t left = __ballot(zero && sp.ok); left; left &= left - 1) {
    const uint32_t row = __shfl(r, __builtin_ctzll(left)), token = row / G;
    const uint32_t at = sp.start + token, last = at >> c.page_log;
    const uint32_t first = (a.window && at >= a.window ? at + 1 - a.window : 0) >> c.page_log;
    bool seen = false;
    for (uint32_t j = first + lane; j <= last; j += 64) seen |= (uint32_t)table[j] < c.pages;
    if (!__any(seen)) continue;
    uint16_t* out = a.out + ((uint64_t)(sp.row0 + token) * a.q_heads + head * G + row % G) * D;
    for (int d = lane * 2; d < D; d += 128) *reinterpret_cast<uint32_t*>(out + d) = 0x7fff7fffu;  // NaN in both types
  }
}

// Waves for each SIMD that the kernel's registers are to leave room for.  3
// instead of 2 for one column block of 64 dims, where the join of the splits then
// spills 32 registers (the loop none): 23 rows with a window of 1,024 18.7 -> 16.1
// us, 64 rows at 1,000-6,000 positions of 16 heads 109 -> 102 us, 200 at 10-900
// 32 -> 26 us.  3 instead of 2 for one of 128 dims: 64 rows at 1,000-6,000 93 -> 107
// us, one at 131,071 57 -> 61 us; 2 instead of 1 for 192 dims: 170 -> 207 us.  The
// most that go without spills else, but for 3 registers of E4M3's two blocks of
// 128 dims.
constexpr int rows_occupancy(int D, int NC) { return D * NC <= 64 ? 3 : D * NC <= 256 && D < 192 ? 2 : 1; }

// W waves on a tile of 16 * NC packed rows (row r of a sequence and key head
// is token r / G, query head r % G of the head's G) and one split of its
// positions; each wave takes every W-th step of 64 tokens, from memory into
// registers with nothing in between.  Lane l = 16 g + n of a wave:
//  - S^T = K Q^T (16x16x32, fp16 in, fp32 out) in four blocks b: row m of the
//    product is token 16 (m / 4) + 4 b + m % 4 of the step, so the lane, which
//    gets rows 4 g + i, holds the scores of tokens 16 g + 4 b + i against row n:
//    16 tokens in a row, all of one page, so the page's scales are the lane's;
//  - O^T = V^T P^T: the lane's 16 bytes of value codes of a dim are those same
//    tokens, so the weights go from the first product's registers into the
//    second's, rounded to fp16, with no move between lanes.
// Keys are read 16 dims of a token a lane (k may come in any order, as long as
// Q's does too), values 16 tokens of a dim a lane; a load instruction covers
// whole 64- and 256-byte runs.  The next step's keys are loaded once this
// step's are used up, and so for values, so one step (2 * 64 * D bytes) is in
// flight for each wave.  Bound by memory where there is enough to read: 64 rows
// at 1,001-6,001 positions (8 heads of 128, 32 query heads) 93 us, 4.6 TB/s, one
// at 131,071 58 us; by the chain lengths, table, codes, partial results, join
// where there is not: one at 777 positions 9 us.
template <bool E4M3, int D, int NC, int W>
__global__ __launch_bounds__(64 * W, rows_occupancy(D, NC)) void k_attend_rows(
    CacheView c, SeqView s, UnitMap map, AttendArgs a, bool bf16, uint32_t units, uint32_t splits, uint32_t per_head) {
  constexpr int R = 16 * NC, KS = D / 32, KL = D / 64, TAIL = D % 64 / 32, DB = D / 16;
  __shared__ float lds_acc[W][16][D + 4];
  __shared__ float lds_m[W][R], lds_l[W][R];
  __shared__ bool lds_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  uint32_t head, unit, split;
  place(blockIdx.x + gridDim.x * blockIdx.y, c.heads, splits, per_head, &head, &unit, &split);
  if (head >= c.heads || unit >= units) return;
  const uint32_t G = a.q_heads / c.heads;
  uint32_t seq;
  Span sp;
  uint64_t own;
  const Early early = load_early(s, unit);
  const bool mine = locate_unit(c, s, map, unit, WaveCount{s, map, unit}, &seq, &sp, &own);
  const Unnamed none = unnamed_rows(s, early);
  if (none.n)
    clear_unnamed(none, a.out + (uint64_t)head * G * D, (uint64_t)a.q_heads * D, G * D, (uint64_t)unit * splits + split,
                  (uint64_t)units * splits);
  if (!(sp.ok && check_sequence(c, s, early)) && threadIdx.x == 0) report(c, kCacheBadSeq);
  const uint32_t packed = sp.n * G;
  if (!mine || own * R >= packed) return;
  const uint32_t r0 = (uint32_t)own * R, r1 = min(r0 + R, packed);
  Range rg = range_of(sp, r0 / G, (r1 - 1) / G + 1, a.window, splits, W);
  if (!sp.ok || c.pages == 0) {
    if (sp.ok && threadIdx.x == 0) report(c, kCacheBadPage);
    rg.hi = rg.lo = rg.steps = rg.used = 0;
  }
  if ((int)split >= max(rg.used, 1)) return;

  const float base = a.scale * kLog2e;
  Rows<D, NC> w;
  load_rows<D, NC>(w, a, sp, head, G, r0, packed, bf16, n, g);
  // positions that every row sees need no masks
  const int all_lo = a.window ? max((int)(sp.start + (r1 - 1) / G) + 1 - (int)a.window, 0) : 0;
  const int all_hi = (int)(sp.start + r0 / G) + 1;

  const int step_end = rg.first + min((int)(split + 1) * rg.per, rg.steps);
  int step = rg.first + (int)split * rg.per + wave;

  const uint32_t page_mask = (1u << c.page_log) - 1;
  const int kb = n >> 2;  // the block whose tokens' keys this lane reads
  const int32_t* table = s.table + seq * s.table_stride;
  // the table's entry for the 16 tokens at t, -1 behind the end; and their
  // byte offset within k or v, and whether they have a page
  auto page_of = [&](int t) -> int32_t { return t < rg.hi ? table[(uint32_t)t >> c.page_log] : -1; };
  auto block_at = [&](int t, int32_t p, bool* have) -> uint64_t {
    *have = (uint32_t)p < c.pages;
    return head_offset(c, *have ? (uint32_t)p : 0, head) + (((uint32_t)t & page_mask) >> 4) * (16 * D);
  };
  uint4v kr[4][KL], vr[DB];
  uint2v kt[4];
  uint32_t scales;
  bool have_v, next_have_v = false;
  auto load_k = [&](uint64_t off) {
    const uint8_t* p = c.k + off + g * 256 + (n & 3) * 16;
    for (int b = 0; b < 4; ++b)
      for (int j = 0; j < KL; ++j) kr[b][j] = *reinterpret_cast<const uint4v*>(p + j * 1024 + b * 64);
    if constexpr (TAIL) {
      const uint8_t* pt = c.k + off + KL * 1024 + (g >> 1) * 256 + (n & 3) * 16 + (g & 1) * 8;
      for (int b = 0; b < 4; ++b) kt[b] = *reinterpret_cast<const uint2v*>(pt + b * 64);
    }
  };
  auto load_v = [&](uint64_t off) {
    const uint8_t* p = c.v + off + n * 16;
    for (int i = 0; i < DB; ++i) vr[i] = *reinterpret_cast<const uint4v*>(p + i * 256);
  };
  auto load_scales = [&](int32_t p, bool have) -> uint32_t {
    return *reinterpret_cast<const uint16_t*>(c.scales + ((uint64_t)(have ? (uint32_t)p : 0) * c.heads + head) * 2);
  };

  // table entries are read a step before the addresses that need them
  bool have_k;
  uint64_t v_off = 0;
  int32_t k_page = -1, v_page = -1;
  if (step < step_end) {
    k_page = page_of(step * kStep + kb * 16);
    v_page = page_of(step * kStep + g * 16);
    const uint64_t k_off = block_at(step * kStep + kb * 16, k_page, &have_k);
    v_off = block_at(step * kStep + g * 16, v_page, &next_have_v);
    load_k(k_off);
    load_v(v_off);
    scales = load_scales(v_page, next_have_v);
    k_page = page_of((step + W) * kStep + kb * 16);
    v_page = page_of((step + W) * kStep + g * 16);
  }
  for (; step < step_end; step += W) {
    const int t0 = step * kStep, tv = t0 + g * 16;
    have_v = next_have_v;
    const uint32_t sc = scales;
    // ---- S^T
    float4v st[NC][4];
    for (int nc = 0; nc < NC; ++nc)
      for (int b = 0; b < 4; ++b) st[nc][b] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const half8 k8 = x < 2 * KL ? codes_to_half<E4M3>(kr[b][x / 2][(x & 1) * 2], kr[b][x / 2][(x & 1) * 2 + 1])
                                    : codes_to_half<E4M3>(kt[b][0], kt[b][1]);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
          st[nc][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, w.q[nc][x], st[nc][b], 0, 0, 0);
      }
    const int next = step + W;
    uint64_t next_v = v_off;
    if (next < step_end) {
      const uint64_t k_off = block_at(next * kStep + kb * 16, k_page, &have_k);
      next_v = block_at(next * kStep + g * 16, v_page, &next_have_v);
      load_k(k_off);
      scales = load_scales(v_page, next_have_v);
      k_page = page_of((next + W) * kStep + kb * 16);
      v_page = page_of((next + W) * kStep + g * 16);
    }
    // ---- weights
    const bool lost = tv < rg.hi && tv + 16 > rg.lo && !have_v;
    if (lost && n == 0) report(c, kCacheBadPage);
    const bool edge = t0 < all_lo || t0 + kStep > all_hi || __any(lost);
    half8 p[NC][2];
    step_weights<D, NC>(w, st, p, base, sc, tv, edge, have_v);
    // ---- O^T
    if (edge) {
      // codes that no row sees may be anything, and 0 * NaN is NaN
      for (int dw = 0; dw < 4; ++dw) {
        const uint32_t keep = have_v ? byte_mask(tv + 4 * dw, rg.lo, rg.hi) : 0;
        for (int i = 0; i < DB; ++i) vr[i][dw] &= keep;
      }
      if constexpr (E4M3) {
        uint32_t any = 0;
        for (int i = 0; i < DB; ++i)
          for (int dw = 0; dw < 4; ++dw) any |= nan_bytes(vr[i][dw]);
        if (__any(any != 0)) {
          note_nan<D, NC>(w, tv, have_v, c.v + v_off + n * 16);
          for (int dw = 0; dw < 4; ++dw) {
            const uint32_t keep = have_v ? byte_mask(tv + 4 * dw, rg.lo, rg.hi) : 0;
            for (int i = 0; i < DB; ++i)
              vr[i][dw] = without_nan(*reinterpret_cast<const uint32_t*>(c.v + v_off + n * 16 + i * 256 + dw * 4) & keep);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const half8 v8 = codes_to_half<E4M3>(vr[i][2 * h], vr[i][2 * h + 1]);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
          w.acc[nc][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, p[nc][h], w.acc[nc][i], 0, 0, 0);
      }
    v_off = next_v;
    if (next < step_end) load_v(v_off);
  }

  if constexpr (E4M3) apply_nan<D, NC>(w);
  // ---- the waves' parts together
  for (int nc = 0; nc < NC; ++nc) {
    w.l[nc] += __shfl_xor(w.l[nc], 16);
    w.l[nc] += __shfl_xor(w.l[nc], 32);
    if (g == 0) {
      lds_m[wave][nc * 16 + n] = w.m[nc];
      lds_l[wave][nc * 16 + n] = w.l[nc];
    }
  }
  __syncthreads();
  const uint64_t tiles = (uint64_t)units * c.heads, tile = (uint64_t)unit * c.heads + head;
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kCounterBytes);
  float* part_ml = part + tiles * splits * R * D;
  const uint64_t at = (tile * splits + split) * R;
  for (int nc = 0; nc < NC; ++nc) {
    {
      const int r = nc * 16 + n;
      float top = -INFINITY;
      for (int v = 0; v < W; ++v) top = fmaxf(top, lds_m[v][r]);
      const float keep = w.m[nc] == top ? 1.0f : __builtin_amdgcn_exp2f(w.m[nc] - top);
      for (int i = 0; i < DB; ++i) {
        const float4v x = w.acc[nc][i] * keep;
        *reinterpret_cast<float4v*>(&lds_acc[wave][n][i * 16 + 4 * g]) = x;
      }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 16 * D / 4; x += 64 * W) {
      const int row = x / (D / 4), d = x % (D / 4) * 4, r = nc * 16 + row;
      float4v sum = {0, 0, 0, 0};
      for (int v = 0; v < W; ++v) sum += *reinterpret_cast<const float4v*>(&lds_acc[v][row][d]);
      float top = -INFINITY, below = 0.0f;
      for (int v = 0; v < W; ++v) top = fmaxf(top, lds_m[v][r]);
      for (int v = 0; v < W; ++v)
        below += rebase(lds_l[v][r], lds_m[v][r], top);
      if (r0 + r >= packed) continue;
      if (rg.used > 1) {
        put2(part + (at + r) * D + d, sum[0], sum[1]);
        put2(part + (at + r) * D + d + 2, sum[2], sum[3]);
        if (d == 0) put2(part_ml + (at + r) * 2, top, below);
      } else {
        store_row<D>(a, sp, head, G, bf16, r0 + r, d, sum, below);
      }
    }
    __syncthreads();
  }
  if (rg.used <= 1) {
    if (wave == 0) {
      bool zero = lane < R && r0 + lane < packed;
      for (int v = 0; v < W; ++v) zero = zero && lds_m[v][lane % R] == -INFINITY && lds_l[v][lane % R] == 0.0f;
      spoil_rows<D>(c, a, sp, table, head, G, r0 + lane, zero);
    }
    return;
  }

  // ---- the splits' parts together, by the workgroup that comes last (and in
  // the splits' order, so that the order of coming does not matter).  One
  // launch, where a second kernel would cost its launch: for one row at 777
  // positions 12.8 us a call with it, 11 without.
  wait_stores();
  __syncthreads();
  if (threadIdx.x == 0) lds_last = atomicInc(static_cast<uint32_t*>(a.ws) + tile, (uint32_t)rg.used - 1) + 1 == (uint32_t)rg.used;
  __syncthreads();
  if (!lds_last) return;
  constexpr int LANES = D / 4, GROUPS = 64 * W / LANES;
  const int grp = threadIdx.x / LANES, x = threadIdx.x % LANES;
  const uint64_t at0 = tile * splits * R;
  const int live = (int)min(packed - r0, (uint32_t)R);
  // the rows' bounds, then their weighted sums: a group of lanes takes rows
  // whole, or, where there are fewer rows than groups, a row's every
  // parts-th split
  const int width = rg.used <= 4 ? 4 : rg.used <= 16 ? 16 : 64;  // lanes of a row
  for (int r = threadIdx.x / width; r < live; r += 64 * W / width) {
    float top = -INFINITY;
    for (int i = lane % width; i < rg.used; i += width) top = fmaxf(top, get2(part_ml + (at0 + (uint64_t)i * R + r) * 2)[0]);
    for (int v = width / 2; v; v >>= 1) top = fmaxf(top, __shfl_xor(top, v));
    if (lane % width == 0) lds_m[0][r] = top;
  }
  __syncthreads();
  // RA rows' SA splits at once: they come from beyond the L2
  auto gather = [&](auto ra, auto sa, int first, int dr, int i0, int di, float4v* sum, float* below) {
    constexpr int RA = decltype(ra)::value, SA = decltype(sa)::value;
    float top[RA];
    for (int k = 0; k < RA; ++k) {
      sum[k] = float4v{0, 0, 0, 0};
      below[k] = 0.0f;
      top[k] = lds_m[0][min(first + k * dr, live - 1)];
    }
    for (int i = i0; i < rg.used; i += SA * di) {
      float2v ml[RA][SA], lo[RA][SA], hi[RA][SA];
#pragma unroll
      for (int k = 0; k < RA; ++k)
#pragma unroll
        for (int j = 0; j < SA; ++j) {
          const uint64_t p = at0 + (uint64_t)min(i + j * di, rg.used - 1) * R + min(first + k * dr, live - 1);
          ml[k][j] = get2(part_ml + p * 2);
          lo[k][j] = get2(part + p * D + x * 4);
          hi[k][j] = get2(part + p * D + x * 4 + 2);
        }
#pragma unroll
      for (int k = 0; k < RA; ++k)
#pragma unroll
        for (int j = 0; j < SA; ++j)
          if (i + j * di < rg.used) {
            const float keep = ml[k][j][0] == top[k] ? 1.0f : __builtin_amdgcn_exp2f(ml[k][j][0] - top[k]);
            sum[k] += float4v{lo[k][j][0], lo[k][j][1], hi[k][j][0], hi[k][j][1]} * keep;
            below[k] += rebase(ml[k][j][1], ml[k][j][0], top[k]);
          }
    }
  };
  const int parts = max(GROUPS / live, 1), mine_of = grp % parts;
  float* lds_flat = &lds_acc[0][0][0];
  // all waves ask the same, since the answer holds a barrier
  auto spoil = [&] {
    const bool none = lane < live && lds_m[0][lane % R] == -INFINITY;
    if (!__any(none)) return;
    bool zero = none;
    for (int i = 0; i < rg.used; ++i) zero = zero && get2(part_ml + (at0 + (uint64_t)i * R + lane % R) * 2)[1] == 0.0f;
    __syncthreads();
    if (wave == 0) spoil_rows<D>(c, a, sp, table, head, G, r0 + lane, zero);
  };
  if (parts == 1) {
    constexpr int RA = 4;
    for (int r = grp; r < live && grp < GROUPS; r += RA * GROUPS) {
      float4v sum[RA];
      float below[RA];
      gather(std::integral_constant<int, RA>(), std::integral_constant<int, 4>(), r, GROUPS, 0, 1, sum, below);
      for (int k = 0; k < RA; ++k)
        if (r + k * GROUPS < live) store_row<D>(a, sp, head, G, bf16, r0 + r + k * GROUPS, x * 4, sum[k], below[k]);
    }
    spoil();
    return;
  }
  const int row = grp / parts;
  if (row < live && grp < GROUPS) {
    float4v sum[1];
    float below[1];
    gather(std::integral_constant<int, 1>(), std::integral_constant<int, 8>(), row, 0, mine_of, parts, sum, below);
    *reinterpret_cast<float4v*>(lds_flat + (grp * LANES + x) * 4) = sum[0];
    if (x == 0) lds_l[0][grp] = below[0];
  }
  __syncthreads();
  if (mine_of == 0 && row < live && grp < GROUPS) {
    float4v sum = {0, 0, 0, 0};
    float below = 0.0f;
    for (int i = 0; i < parts; ++i) {
      sum += *reinterpret_cast<const float4v*>(lds_flat + ((grp + i) * LANES + x) * 4);
      below += lds_l[0][grp + i];
    }
    store_row<D>(a, sp, head, G, bf16, r0 + row, x * 4, sum, below);
  }
  spoil();
}

constexpr uint32_t kTileRows = 128;
// Workgroups on a CU: as many as registers and shared memory hold.  3 instead
// of 2 for one prompt of 4,096 rows of 64 dims: 142 -> 115 us; for 2,048 rows of
// 96 dims registers spill: 64 -> 94 us (for E4M3's 64 dims one does).
constexpr int tiles_occupancy(int D) { return D <= 64 ? 3 : D <= 128 ? 2 : 1; }

// The order of a run of 4 * N reads of shared memory and their 4 * N * NC
// products: always four reads ahead.
template <int N, int NC> __device__ __forceinline__ void reads_ahead() {
  constexpr int kRead = 0x100, kProduct = 0x8;
  __builtin_amdgcn_sched_group_barrier(kRead, N > 1 ? 8 : 4, 0);
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, NC, 0);
    if (i + 8 < 4 * N) __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
}

// Prompts: four waves, 32 rows each, on the same positions.  The same two
// products as above, but each wave turns a quarter of a step's codes into fp16,
// once for the four, and shared memory holds them in the order in which the
// lanes take them, so that every access is one run of 1 KB: while a step is
// computed the next one's are turned, and those of the one behind it are on
// their way from memory.  Eight prompts of 4,096 rows behind 4,096 positions (8
// heads of 128, 32 query heads) 3.64 ms, 906 TFLOP/s, where k_attend_rows takes
// 4.2 ms: a library product of 8,192 reaches 1,250.  Matrix cores are busy for
// 35% of the time, vector units for 60%; without exp2 it is as fast, without
// turning 12% faster, without loads 14%, with an eighth of the second product
// 10%: the chain of a step (read, product, maximum, exp2, product) is longer
// than two waves a SIMD hide.
template <bool E4M3, int D>
__global__ __launch_bounds__(256, tiles_occupancy(D)) void k_attend_tiles(CacheView c, SeqView s, UnitMap map,
                                                                          AttendArgs a, bool bf16, uint32_t units,
                                                                          uint32_t per_head) {
  constexpr int NC = 2, WR = 16 * NC, R = kTileRows, KS = D / 32, KL = D / 64, TAIL = D % 64 / 32, DB = D / 16, VL = (DB + 3) / 4;
  __shared__ half8 lds[2][(KS * 4 + DB * 2) * 64];  // keys [x][b][lane], values [i][h][lane]
  __shared__ int lds_nan[2];                        // 1 + the step whose values have a NaN
  constexpr int kValues = KS * 4;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t head, unit, split;
  place(blockIdx.x + gridDim.x * blockIdx.y, c.heads, 1, per_head, &head, &unit, &split);
  if (head >= c.heads || unit >= units) return;
  const uint32_t G = a.q_heads / c.heads;
  uint32_t seq;
  Span sp;
  uint64_t own;
  const Early early = load_early(s, unit);
  const bool mine = locate_unit(c, s, map, unit, WaveCount{s, map, unit}, &seq, &sp, &own);
  const Unnamed none = unnamed_rows(s, early);
  if (none.n) clear_unnamed(none, a.out + (uint64_t)head * G * D, (uint64_t)a.q_heads * D, G * D, unit, units);
  if (!(sp.ok && check_sequence(c, s, early)) && threadIdx.x == 0) report(c, kCacheBadSeq);
  const uint32_t packed = sp.n * G;
  if (!mine || own * R >= packed) return;
  const uint32_t r0 = (uint32_t)own * R, r1 = min(r0 + R, packed);
  Range rg = range_of(sp, r0 / G, (r1 - 1) / G + 1, a.window, 1, 1);
  if (!sp.ok || c.pages == 0) {
    if (sp.ok && threadIdx.x == 0) report(c, kCacheBadPage);
    rg.hi = rg.lo = rg.steps = 0;
  }
  const float base = a.scale * kLog2e;
  // the wave's rows, the positions that some of them see and those that all see
  const uint32_t w0 = r0 + wave * WR, w1 = min(w0 + WR, packed);
  const bool live = w0 < w1 && rg.steps > 0;
  const int hi = live ? (int)(sp.start + (w1 - 1) / G) + 1 : 0, all_hi = live ? (int)(sp.start + w0 / G) + 1 : 0;
  const int lo = a.window ? max(all_hi - (int)a.window, 0) : 0, all_lo = a.window ? max(hi - (int)a.window, 0) : 0;
  Rows<D, NC> w;
  load_rows<D, NC>(w, a, sp, head, G, w0, packed, bf16, n, g);

  const uint32_t page_mask = (1u << c.page_log) - 1;
  const int kb = n >> 2;
  const int32_t* table = s.table + seq * s.table_stride;
  auto page_of = [&](int t) -> int32_t { return t < rg.hi ? table[(uint32_t)t >> c.page_log] : -1; };
  auto block_at = [&](int t, int32_t p) -> uint64_t {
    return head_offset(c, (uint32_t)p < c.pages ? (uint32_t)p : 0, head) + (((uint32_t)t & page_mask) >> 4) * (16 * D);
  };
  // a quarter of a step's codes: block b = wave of the keys, dims 16 i + n of the values, i = wave, wave + 4 ..
  uint4v kr[KL], vr[VL];
  uint2v kt = {0, 0};
  int32_t k_page = -1, v_page = -1;           // of the step to load next
  int32_t page = -1, next_page = -1;          // of the step computed, and of the next one, at g's tokens
  uint32_t scales = 0, next_scales = 0;
  auto pages = [&](int step) {
    k_page = page_of(step * kStep + kb * 16);
    v_page = page_of(step * kStep + g * 16);
  };
  auto load = [&](int step) {
    const uint8_t* k = c.k + block_at(step * kStep + kb * 16, k_page) + (n & 3) * 16 + wave * 64;
    const uint8_t* v = c.v + block_at(step * kStep + g * 16, v_page) + n * 16;
    for (int j = 0; j < KL; ++j) kr[j] = *reinterpret_cast<const uint4v*>(k + g * 256 + j * 1024);
    if constexpr (TAIL) kt = *reinterpret_cast<const uint2v*>(k + KL * 1024 + (g >> 1) * 256 + (g & 1) * 8);
    for (int i = 0; i < VL; ++i)
      if (DB % 4 == 0 || wave + 4 * i < DB) vr[i] = *reinterpret_cast<const uint4v*>(v + (wave + 4 * i) * 256);
    next_page = v_page;
    next_scales = *reinterpret_cast<const uint16_t*>(
        c.scales + ((uint64_t)((uint32_t)v_page < c.pages ? (uint32_t)v_page : 0) * c.heads + head) * 2);
    pages(step + 1);
  };
  auto turn = [&](int step) {
    half8* to = lds[step & 1] + lane;
    for (int j = 0; j < KL; ++j)
      for (int x = 0; x < 2; ++x)
        to[((2 * j + x) * 4 + wave) * 64] = codes_to_half<E4M3>(kr[j][2 * x], kr[j][2 * x + 1]);
    if constexpr (TAIL) to[((KS - 1) * 4 + wave) * 64] = codes_to_half<E4M3>(kt[0], kt[1]);
    // values that no row sees may be anything, and 0 * NaN is NaN
    const int t0 = step * kStep, tv = t0 + g * 16;
    const bool lost = (uint32_t)next_page >= c.pages;
    if (t0 < rg.lo || t0 + kStep > rg.hi || __any(lost))
      for (int dw = 0; dw < 4; ++dw) {
        const uint32_t keep = lost ? 0 : byte_mask(tv + 4 * dw, rg.lo, rg.hi);
        for (int i = 0; i < VL; ++i) vr[i][dw] &= keep;
      }
    if constexpr (E4M3) {
      uint32_t any = 0;
      for (int i = 0; i < VL; ++i)
        for (int dw = 0; dw < 4; ++dw) any |= nan_bytes(vr[i][dw]);
      if (__any(any != 0)) {
        for (int i = 0; i < VL; ++i)
          for (int dw = 0; dw < 4; ++dw) vr[i][dw] = without_nan(vr[i][dw]);
        if (lane == 0) lds_nan[step & 1] = step + 1;
      }
    }
    for (int i = 0; i < VL; ++i)
      if (DB % 4 == 0 || wave + 4 * i < DB)
        for (int h = 0; h < 2; ++h)
          to[(kValues + 2 * (wave + 4 * i) + h) * 64] = codes_to_half<E4M3>(vr[i][2 * h], vr[i][2 * h + 1]);
  };

  int step = rg.first;
  const int step_end = rg.first + rg.steps;
  for (int i = 0; i < VL; ++i) vr[i] = uint4v{0, 0, 0, 0};
  if (threadIdx.x < 2) lds_nan[threadIdx.x] = 0;
  __syncthreads();
  if (step < step_end) {
    pages(step);
    load(step);
    turn(step);
    page = next_page;
    scales = next_scales;
    if (step + 1 < step_end) load(step + 1);
  }
  for (; step < step_end; ++step) {
    __syncthreads();  // the step's values are there, and the other buffer is not read any more
    const int32_t p_now = page;
    const bool have = (uint32_t)p_now < c.pages;
    const uint32_t sc = scales;
    if (step + 1 < step_end) {
      turn(step + 1);
      page = next_page;
      scales = next_scales;
      if (step + 2 < step_end) load(step + 2);
    }
    const int t0 = step * kStep, tv = t0 + g * 16;
    if (t0 >= hi || t0 + kStep <= lo) continue;
    const half8* from = lds[step & 1] + lane;
    // ---- S^T; no two products in a row on the same sums, four reads ahead
    float4v st[NC][4];
    for (int nc = 0; nc < NC; ++nc)
      for (int b = 0; b < 4; ++b) st[nc][b] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const half8 k8 = from[(x * 4 + b) * 64];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
          st[nc][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, w.q[nc][x], st[nc][b], 0, 0, 0);
      }
    reads_ahead<KS, NC>();
    // ---- weights
    const bool lost = tv < hi && tv + 16 > lo && !have;
    if (lost && n == 0) report(c, kCacheBadPage);
    const bool edge = t0 < all_lo || t0 + kStep > all_hi || __any(lost);
    half8 p[NC][2];
    step_weights<D, NC>(w, st, p, base, sc, tv, edge, have);
    // ---- O^T
    from += kValues * 64;
#pragma unroll
    for (int i = 0; i < DB; i += 2)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = i; j < i + 2; ++j) {
          const half8 v8 = from[(2 * j + h) * 64];
#pragma unroll
          for (int nc = 0; nc < NC; ++nc)
            w.acc[nc][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, p[nc][h], w.acc[nc][j], 0, 0, 0);
        }
    reads_ahead<DB / 2, NC>();
    if (E4M3 && lds_nan[step & 1] == step + 1) note_nan<D, NC>(w, tv, have, c.v + block_at(tv, p_now) + n * 16);
  }
  if constexpr (E4M3) apply_nan<D, NC>(w);
  for (int nc = 0; nc < NC; ++nc) {
    float below = w.l[nc];
    below += __shfl_xor(below, 16);
    below += __shfl_xor(below, 32);
    const uint32_t r = w0 + nc * 16 + n;
    if (r < packed)
      for (int i = 0; i < DB; ++i) store_row<D>(a, sp, head, G, bf16, r, i * 16 + 4 * g, w.acc[nc][i], below);
    spoil_rows<D>(c, a, sp, table, head, G, r, g == 0 && r < packed && below == 0.0f);
  }
}

constexpr int kWaves = 4;
// Workgroups that the splits are to make: two for each CU, one where a CU holds
// one.  One row at 131,071 positions (D = 128) with 256 / 512 / 768 / 1024 of
// them: 64 / 61 / 67 / 75 us; 16 sequences of 5 rows: 39 / 29 / 39 / 41 us; four
// rows at 20,001 positions of 2 heads of 256 dims with 256 / 512: 46 / 78 us.
constexpr uint32_t fill(int D, int NC) { return 256 * (rows_occupancy(D, NC) < 2 ? 1 : 2); }
constexpr uint32_t kGridWidth = 1u << 20;  // times a workgroup's lanes below 2^32

struct Plan {
  UnitMap map;
  uint32_t units, nc, splits;
  uint32_t per_head;  // workgroups of a head
  bool tiles;
  dim3 grid;
};

Plan plan_rows(const CacheView& c, const SeqView& s, uint32_t q_heads, uint32_t window) {
  Plan p;
  const uint32_t G = q_heads / c.heads;
  const uint64_t mean = ((uint64_t)s.rows * G + s.seqs - 1) / s.seqs;  // packed rows of a sequence and head
  // k_attend_tiles where there are workgroups for all CUs and rows to fill its
  // tiles, else k_attend_rows, which splits the positions.  tiles / rows: one
  // prompt of 512, 1,024, 2,048 and 16 of 2,048 rows (8 heads of 128, 4 query
  // heads each) 24 / 15, 38 / 31, 72 / 76 and 778 / 1,216 us; two of 1,024 rows of
  // 256 dims 96 / 145 us.  100 times 64 and 96 packed rows of 64 dims behind 1,000
  // positions 76 / 62 and 78 / 99 us, 100 times 128 and 192 of 128 dims 182 / 136
  // and 189 / 213 us.
  const uint64_t tiles = unit_count(UnitMap{G, kTileRows, 1}, s.rows, s.seqs) * c.heads;
  p.tiles = s.cu && mean > (c.dim <= 96 ? 64 : 128) && tiles >= (c.dim <= 128 ? 512 : 256);
  // Two column blocks a wave where there are rows for them; four leave a SIMD one
  // wave: 80 times 10 rows (40 packed) of 96 dims 106 / 161 us with two / four, 20
  // times 16 of 64 dims 29 / 47 us, and two instead of one of 256 dims 76 / 65 us.
  p.nc = mean <= 16 || c.dim > 192 ? 1 : 2;
  const uint32_t R = p.tiles ? kTileRows : 16 * p.nc;
  p.map = s.cu ? UnitMap{G, R, 1} : UnitMap{0, 1, (G + R - 1) / R};
  p.units = (uint32_t)unit_count(p.map, s.rows, s.seqs);
  uint64_t longest = (uint64_t)s.width << c.page_log;
  if (window && window + 64 < longest) longest = window + 64;
  const uint64_t most = (longest + kStep * kWaves - 1) / (kStep * kWaves);
  const uint64_t base = (uint64_t)p.units * c.heads;
  const uint64_t want = (fill((int)c.dim, (int)p.nc) + base - 1) / base;
  p.splits = (uint32_t)(want < most ? want : most);
  if (p.splits < 1 || base > kCounters || p.tiles) p.splits = 1;
  const uint32_t share = chiplet_share(c.heads);
  p.per_head = (p.units * p.splits + share - 1) / share * share;
  const uint64_t groups = (uint64_t)p.per_head * c.heads;  // a multiple of 8
  p.grid = dim3((uint32_t)(groups < kGridWidth ? groups : kGridWidth), (uint32_t)((groups + kGridWidth - 1) / kGridWidth));
  return p;
}

template <bool E4M3, int D, int W>
hipError_t launch_waves(const CacheView& c, const SeqView& s, bool bf16, const AttendArgs& a, const Plan& p,
                        hipStream_t st) {
  auto launch = [&](auto kernel) {
    kernel<<<p.grid, 64 * W, 0, st>>>(c, s, p.map, a, bf16, p.units, p.splits, p.per_head);
  };
  if (p.nc == 1) launch(k_attend_rows<E4M3, D, 1, W>);
  else if constexpr (D <= 192) launch(k_attend_rows<E4M3, D, 2, W>);
  return hipGetLastError();
}

template <bool E4M3, int D>
hipError_t launch_rows(const CacheView& c, const SeqView& s, bool bf16, const AttendArgs& a, const Plan& p,
                       hipStream_t st) {
  if (p.tiles) {
    k_attend_tiles<E4M3, D><<<p.grid, 256, 0, st>>>(c, s, p.map, a, bf16, p.units, p.per_head);
    return hipGetLastError();
  }
  // Heads of 192 and 256 dims leave a SIMD one wave: where nothing is split, two
  // workgroups of two waves hide each other's beginnings and ends.  2 / 4 waves:
  // 9 prompts of 33-517 rows of 256 dims 47 / 65 us, 300 rows at 10-900 positions
  // 143 / 176 us, 64 at 1,000-6,000 194 / 192 us.  With 128 dims: 62 / 72 us and
  // 113 / 92 us, so four there.
  if constexpr (D >= 192) {
    if (p.splits == 1) return launch_waves<E4M3, D, 2>(c, s, bf16, a, p, st);
  }
  return launch_waves<E4M3, D, kWaves>(c, s, bf16, a, p, st);
}

template <bool E4M3>
hipError_t launch_dim(const CacheView& c, const SeqView& s, bool bf16, const AttendArgs& a, hipStream_t st) {
  const Plan p = plan_rows(c, s, a.q_heads, a.window);
  switch (c.dim) {
    case 64: return launch_rows<E4M3, 64>(c, s, bf16, a, p, st);
    case 96: return launch_rows<E4M3, 96>(c, s, bf16, a, p, st);
    case 128: return launch_rows<E4M3, 128>(c, s, bf16, a, p, st);
    case 192: return launch_rows<E4M3, 192>(c, s, bf16, a, p, st);
    case 256: return launch_rows<E4M3, 256>(c, s, bf16, a, p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

uint64_t cache_attend_workspace(const CacheView& c, const SeqView& s, uint32_t q_heads, uint32_t window) {
  if (!s.rows) return 0;
  const Plan p = plan_rows(c, s, q_heads, window);
  return p.splits == 1 ? 0 : kCounterBytes + (uint64_t)p.units * c.heads * p.splits * 16 * p.nc * (c.dim + 2) * sizeof(float);
}

hipError_t launch_cache_attend(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const AttendArgs& a,
                               hipStream_t st) {
  const bool bf16 = dtype == LTC_BF16;
  return e4m3 ? launch_dim<true>(c, s, bf16, a, st) : launch_dim<false>(c, s, bf16, a, st);
}

}  // namespace ltc
