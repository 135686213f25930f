// ltc_cache_evict.hip -- a cache cut to the positions of most weight: which they
// are (k_pick), and their move to other pages (k_move).
#include "ltc_cache_device.h"

namespace ltc {
namespace {

constexpr int kPickLanes = 1024, kPickWaves = kPickLanes / 64, kBins = 2048;

// A number's place in the order of weights, as an unsigned one; a NaN is below
// all others, and the zeros are equal.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x != x ? 0 : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

constexpr int kRound = 4 * kPickLanes;  // positions that a workgroup goes over at a time, four a lane
constexpr int kAhead = 4;               // rounds whose loads are in flight

// A workgroup takes a sequence and head.  The least weight that is kept is found
// in three digits, of 11, 11 and 10 bits, from histograms in shared memory; then
// the kept positions are counted wave by wave, and written behind one another.
// The first HELD rounds of the weights stay in shared memory, those behind are read
// again for each pass.  64 sequences of 700-6,000 positions in 8 heads to 1,024: 17.6
// us, of which the weights' 7 MB are 2: a chain of a dozen steps of the whole
// workgroup.  Digits of 8 bits with a histogram for each wave, and a second look at
// memory in each pass: 38 us.
template <int HELD>
__global__ __launch_bounds__(kPickLanes, HELD > 4 ? 4 : 8) void k_pick(CacheView c, SeqView s, const float* weights, uint32_t keep,
                                                     uint32_t recent, int32_t* lengths, int32_t* positions) {
  constexpr int SCANNED = 16;  // rounds that are counted before they are written
  __shared__ uint4v held[HELD][kPickLanes];
  __shared__ uint32_t counts[kBins];
  __shared__ uint32_t sums[2][SCANNED][kPickWaves];
  __shared__ uint32_t found[3], totals[2][kPickWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t head = blockIdx.x, seq = blockIdx.y;
  const int32_t length = s.lengths[seq];
  const bool ok = length >= 0 && (uint64_t)length <= capacity_of(c, s);
  if (!ok && threadIdx.x == 0) report(c, kCacheBadSeq);
  const uint32_t n = ok ? (uint32_t)length : 0;
  if (head == 0 && threadIdx.x == 0) lengths[seq] = (int32_t)min(n, keep);
  int32_t* out = positions + ((uint64_t)seq * c.heads + head) * keep;
  if (n <= keep) {
    for (uint32_t i = threadIdx.x; i < keep; i += kPickLanes) out[i] = i < n ? (int32_t)i : -1;
    return;
  }
  const uint32_t others = n - recent;
  for (uint32_t i = threadIdx.x; i < recent; i += kPickLanes) out[keep - recent + i] = (int32_t)(others + i);
  if (keep == recent) return;
  const int32_t* table = s.table + seq * s.table_stride;
  const uint32_t mask = (1u << c.page_log) - 1, rounds = (others + kRound - 1) / kRound;
  auto first_of = [&](uint32_t round) -> uint32_t { return round * kRound + 4 * threadIdx.x; };
  auto load = [&](uint32_t t) -> uint4v {  // a page has its four positions, or none of them
    const uint32_t page = t < others ? (uint32_t)table[t >> c.page_log] : c.pages;
    if (page >= c.pages) return uint4v{0, 0, 0, 0};
    const float4v w = *reinterpret_cast<const float4v*>(weights + (((uint64_t)page * c.heads + head) << c.page_log) + (t & mask));
    return uint4v{order_of(w[0]), order_of(w[1]), order_of(w[2]), order_of(w[3])};
  };
  // visit(round, first position, its keys) for rounds [from, to)
  auto each_round = [&](uint32_t from, uint32_t to, auto visit) {
    for (uint32_t r0 = from; r0 < to; r0 += kAhead) {
      uint4v keys[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t r = r0 + i;
        if (r < to) keys[i] = r < HELD ? held[r][threadIdx.x] : load(first_of(r));
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r0 + i < to) visit(r0 + i, first_of(r0 + i), keys[i]);
    }
  };
  for (uint32_t r0 = 0; r0 < min(rounds, (uint32_t)HELD); r0 += kAhead) {
    uint4v keys[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) keys[i] = load(first_of(r0 + i));
#pragma unroll
    for (int i = 0; i < kAhead; ++i) held[r0 + i][threadIdx.x] = keys[i];
  }
  uint32_t need = keep - recent, border = 0;  // `need` of those that begin with border's digits so far are kept
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, above_bits = digit == 0 ? 32 : digit == 1 ? 21 : 10;
    const uint32_t bins = digit == 2 ? 1024 : kBins;
    for (uint32_t i = threadIdx.x; i < bins; i += kPickLanes) counts[i] = 0;
    __syncthreads();
    each_round(0, rounds, [&](uint32_t, uint32_t t, uint4v key) {
      for (int j = 0; j < 4; ++j)
        if (t + j < others && (uint64_t)(key[j] ^ border) >> above_bits == 0)
          atomicAdd(&counts[key[j] >> shift & (bins - 1)], 1u);
    });
    __syncthreads();
    // the digit at which those of it and of the higher ones are `need`, from the top
    // down: lanes have two neighbouring digits each
    const uint32_t top = bins - 1 - 2 * threadIdx.x;
    const bool mine = 2 * threadIdx.x < bins;
    const uint32_t hi = mine ? counts[top] : 0, lo = mine ? counts[top - 1] : 0;
    uint32_t sum = hi + lo;
    for (int w = 1; w < 64; w <<= 1) {
      const uint32_t x = __shfl_up(sum, w);
      if (lane >= w) sum += x;
    }
    if (lane == 63) totals[0][wave] = sum;
    __syncthreads();
    uint32_t above = sum - hi - lo;
    for (int w = 0; w < wave; ++w) above += totals[0][w];
    if (mine && above < need && need <= above + hi + lo) {
      const bool first = need <= above + hi;
      found[0] = first ? top : top - 1;
      found[1] = need - above - (first ? 0 : hi);
      found[2] = shift && border | found[0] && found[1] == (first ? hi : lo);
    }
    __syncthreads();
    border |= found[0] << shift;
    need = found[1];
    if (found[2]) {  // all that begin like the border are kept: the rest of it does not matter
      --border;      // they are above this
      need = 0;
      break;
    }
  }
  // `need` of the weights equal to the border are kept, the first ones
  const uint64_t below = (1ull << lane) - 1;
  uint32_t kept = 0, equal = 0;  // of the rounds before
  for (uint32_t r0 = 0; r0 < rounds; r0 += SCANNED) {
    const uint32_t r1 = min(rounds, r0 + SCANNED);
    // how many lie above the border and on it in each wave's 256
    each_round(r0, r1, [&](uint32_t r, uint32_t t, uint4v key) {
      uint32_t more = 0, same = 0;
      for (int j = 0; j < 4; ++j) {
        more += __popcll(__ballot(t + j < others && key[j] > border));
        same += __popcll(__ballot(t + j < others && key[j] == border));
      }
      if (lane == 0) {
        sums[0][r - r0][wave] = more;
        sums[1][r - r0][wave] = same;
      }
    });
    __syncthreads();
    // the sums become those of the waves before; lanes have one each of a kind
    static_assert(SCANNED * kPickWaves <= kPickLanes / 2);
    constexpr int EACH = kPickLanes / 2;
    const int kind = threadIdx.x / EACH, at = threadIdx.x % EACH;
    const bool mine = at < (int)(r1 - r0) * kPickWaves;
    const uint32_t own = mine ? sums[kind][at / kPickWaves][at % kPickWaves] : 0;
    uint32_t run = own;
    for (int w = 1; w < 64; w <<= 1) {
      const uint32_t x = __shfl_up(run, w);
      if (lane >= w) run += x;
    }
    if (lane == 63) totals[0][wave] = run;
    __syncthreads();
    for (int w = kind * (kPickWaves / 2); w < wave; ++w) run += totals[0][w];
    if (mine) sums[kind][at / kPickWaves][at % kPickWaves] = run - own;
    uint32_t all[2] = {0, 0};
    for (int w = 0; w < kPickWaves; ++w) all[w / (kPickWaves / 2)] += totals[0][w];
    __syncthreads();
    each_round(r0, r1, [&](uint32_t r, uint32_t t, uint4v key) {
      uint32_t more = kept + sums[0][r - r0][wave], same = equal + sums[1][r - r0][wave];  // before this lane's
      for (int j = 0; j < 4; ++j) {
        more += __popcll(__ballot(t + j < others && key[j] > border) & below);
        same += __popcll(__ballot(t + j < others && key[j] == border) & below);
      }
      for (int j = 0; j < 4; ++j) {
        if (t + j >= others) break;
        const bool is = key[j] == border;
        // kept counts those equal to the border as well, as many as are kept
        if (key[j] > border || (is && same < need)) out[more + min(same, need) - min(equal, need)] = (int32_t)(t + j);
        more += key[j] > border;
        same += is;
      }
    });
    kept += all[0] + min(equal + all[1], need) - min(equal, need);
    equal += all[1];
    __syncthreads();
  }
}

// Few sequences and heads of many positions: `splits` workgroups share each, and
// every digit, the counts and the positions are a launch of their own.  A sequence
// and head has in the workspace
//   {border, need, done, 0} as found so far, twice, counts[2][splits], and
//   histograms [2][splits][kBins].
// A launch reads one of a pair and writes the other, since its workgroups do not
// wait for each other.
constexpr int kSplitLanes = 512, kSplitWaves = kSplitLanes / 64, kSplitRound = 4 * kSplitLanes;
constexpr uint32_t kMostSplits = 16;

LTC_HD uint64_t split_words(uint32_t splits) { return 8 + 2 * kMostSplits + (uint64_t)2 * splits * kBins; }

struct PickArgs {
  const float* weights;
  uint32_t keep, recent;
  int32_t *lengths, *positions;
  uint32_t* ws;
  uint32_t splits;
};

// PHASE 0, 1, 2: the histogram of that digit; 3: how many lie above the border and
// on it; 4: the positions.
template <int PHASE>
__global__ __launch_bounds__(kSplitLanes) void k_pick_split(CacheView c, SeqView s, PickArgs a) {
  __shared__ uint32_t counts[kBins];
  __shared__ uint32_t sums[2][kSplitWaves];
  __shared__ uint32_t found[3];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t head = blockIdx.x, split = blockIdx.y, seq = blockIdx.z;
  const int32_t length = s.lengths[seq];
  const bool ok = length >= 0 && (uint64_t)length <= capacity_of(c, s);
  const uint32_t n = ok ? (uint32_t)length : 0, others = n > a.keep ? n - a.recent : 0;
  const uint64_t pair = (uint64_t)seq * c.heads + head;
  int32_t* out = a.positions + pair * a.keep;
  if (PHASE == 0) {
    if (!ok && threadIdx.x == 0) report(c, kCacheBadSeq);
    if (head == 0 && split == 0 && threadIdx.x == 0) a.lengths[seq] = (int32_t)min(n, a.keep);
    // all are kept, or the last ones
    const uint32_t at = split * kSplitLanes + threadIdx.x, step = a.splits * kSplitLanes;
    if (!others)
      for (uint32_t i = at; i < a.keep; i += step) out[i] = i < n ? (int32_t)i : -1;
    else
      for (uint32_t i = at; i < a.recent; i += step) out[a.keep - a.recent + i] = (int32_t)(others + i);
  }
  if (!others || a.keep == a.recent) return;
  uint32_t* state = a.ws + pair * split_words(a.splits);
  uint32_t* side[2] = {state + 8, state + 8 + kMostSplits};
  uint32_t* histograms = state + 8 + 2 * kMostSplits;
  const int32_t* table = s.table + seq * s.table_stride;
  const uint32_t mask = (1u << c.page_log) - 1;
  const uint32_t rounds = (others + kSplitRound - 1) / kSplitRound, per = (rounds + a.splits - 1) / a.splits;
  const uint32_t r0 = min(split * per, rounds), r1 = min(r0 + per, rounds);
  auto load = [&](uint32_t t) -> uint4v {
    const uint32_t page = t < others ? (uint32_t)table[t >> c.page_log] : c.pages;
    if (page >= c.pages) return uint4v{0, 0, 0, 0};
    const float4v w = *reinterpret_cast<const float4v*>(a.weights + (((uint64_t)page * c.heads + head) << c.page_log) + (t & mask));
    return uint4v{order_of(w[0]), order_of(w[1]), order_of(w[2]), order_of(w[3])};
  };
  uint4v first[kAhead];  // the first rounds' weights come while the digit before is found
#pragma unroll
  for (int i = 0; i < kAhead; ++i) first[i] = load(r0 + i < r1 ? (r0 + i) * kSplitRound + 4 * threadIdx.x : others);
  uint32_t border = 0, need = a.keep - a.recent;
  bool done = false;
  if (PHASE >= 2) {
    const uint32_t* from = state + 4 * (PHASE & 1);
    border = from[0];
    need = from[1];
    done = from[2] != 0;
  }
  if (PHASE >= 1 && PHASE <= 3 && !done) {  // the digit before: all splits' histograms together
    constexpr int DIGIT = PHASE - 1, SHIFT = DIGIT == 0 ? 21 : DIGIT == 1 ? 10 : 0, BINS = DIGIT == 2 ? 1024 : kBins;
    const uint32_t* from = histograms + (uint64_t)(DIGIT & 1) * a.splits * kBins;
    const bool mine = 4 * threadIdx.x < BINS;
    const uint32_t low = BINS - 4 - 4 * threadIdx.x;  // the lane's four digits, from the top down
    uint4v sum = {0, 0, 0, 0};
    if (mine) {  // all at once
      uint4v x[kMostSplits];
#pragma unroll
      for (uint32_t i = 0; i < kMostSplits; ++i)
        x[i] = *reinterpret_cast<const uint4v*>(from + (uint64_t)min(i, a.splits - 1) * kBins + low);
#pragma unroll
      for (uint32_t i = 0; i < kMostSplits; ++i)
        if (i < a.splits) sum += x[i];
    }
    uint32_t run = sum[0] + sum[1] + sum[2] + sum[3];
    const uint32_t own = run;
    for (int w = 1; w < 64; w <<= 1) {
      const uint32_t x = __shfl_up(run, w);
      if (lane >= w) run += x;
    }
    if (lane == 63) sums[0][wave] = run;
    __syncthreads();
    uint32_t above = run - own;
    for (int w = 0; w < wave; ++w) above += sums[0][w];
    if (mine)
      for (int i = 3; i >= 0; --i) {
        if (above < need && need <= above + sum[i]) {
          found[0] = low + i;
          found[1] = need - above;
          found[2] = SHIFT && (border | (low + i)) && need - above == sum[i];
        }
        above += sum[i];
      }
    __syncthreads();
    border |= found[0] << SHIFT;
    need = found[1];
    if (found[2]) {  // all that begin like the border are kept: they are above this
      --border;
      need = 0;
      done = true;
    }
  }
  auto each_round = [&](auto visit) {
    for (uint32_t r = r0; r < r1; r += kAhead) {
      uint4v keys[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        keys[i] = r == r0 ? first[i] : load(r + i < r1 ? (r + i) * kSplitRound + 4 * threadIdx.x : others);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r + i < r1) visit((r + i) * kSplitRound + 4 * threadIdx.x, keys[i]);
    }
  };
  if constexpr (PHASE <= 2) {
    constexpr int SHIFT = PHASE == 0 ? 21 : PHASE == 1 ? 10 : 0, BINS = PHASE == 2 ? 1024 : kBins;
    constexpr int ABOVE = PHASE == 0 ? 32 : PHASE == 1 ? 21 : 10;
    if (!done) {
      for (int i = threadIdx.x; i < BINS; i += kSplitLanes) counts[i] = 0;
      __syncthreads();
      each_round([&](uint32_t t, uint4v key) {
        for (int j = 0; j < 4; ++j)
          if (t + j < others && (uint64_t)(key[j] ^ border) >> ABOVE == 0) atomicAdd(&counts[key[j] >> SHIFT & (BINS - 1)], 1u);
      });
      __syncthreads();
      uint32_t* to = histograms + ((uint64_t)(PHASE & 1) * a.splits + split) * kBins;
      for (int i = threadIdx.x; i < BINS / 4; i += kSplitLanes)
        *reinterpret_cast<uint4v*>(to + 4 * i) = *reinterpret_cast<const uint4v*>(counts + 4 * i);
    }
  } else if constexpr (PHASE == 3) {
    uint32_t more = 0, same = 0;
    each_round([&](uint32_t t, uint4v key) {
      for (int j = 0; j < 4; ++j) {
        more += __popcll(__ballot(t + j < others && key[j] > border));
        same += __popcll(__ballot(t + j < others && key[j] == border));
      }
    });
    if (lane == 0) {
      sums[0][wave] = more;
      sums[1][wave] = same;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      uint32_t all = 0;
      for (int w = 0; w < kSplitWaves; ++w) all += sums[threadIdx.x][w];
      side[threadIdx.x][split] = all;
    }
  } else {
    uint32_t kept = 0, equal = 0;  // of the splits before
    uint32_t x[2][kMostSplits];
#pragma unroll
    for (uint32_t i = 0; i < kMostSplits; ++i)
      for (int j = 0; j < 2; ++j) x[j][i] = side[j][min(i, a.splits - 1)];
#pragma unroll
    for (uint32_t i = 0; i < kMostSplits; ++i)
      if (i < split) {
        kept += x[0][i];
        equal += x[1][i];
      }
    const uint64_t below = (1ull << lane) - 1;
    each_round([&](uint32_t t, uint4v key) {
      uint64_t b_more[4], b_same[4];
      uint32_t more = 0, same = 0;
      for (int j = 0; j < 4; ++j) {
        b_more[j] = __ballot(t + j < others && key[j] > border);
        b_same[j] = __ballot(t + j < others && key[j] == border);
        more += __popcll(b_more[j]);
        same += __popcll(b_same[j]);
      }
      __syncthreads();
      if (lane == 0) {
        sums[0][wave] = more;
        sums[1][wave] = same;
      }
      __syncthreads();
      more = kept;
      same = equal;
      for (int w = 0; w < kSplitWaves; ++w) {
        if (w < wave) {
          more += sums[0][w];
          same += sums[1][w];
        }
        kept += sums[0][w];
        equal += sums[1][w];
      }
      for (int j = 0; j < 4; ++j) {
        more += __popcll(b_more[j] & below);
        same += __popcll(b_same[j] & below);
      }
      for (int j = 0; j < 4; ++j) {
        if (t + j >= others) break;
        const bool is = key[j] == border;
        if (key[j] > border || (is && same < need)) out[more + min(same, need)] = (int32_t)(t + j);
        more += key[j] > border;
        same += is;
      }
    });
  }
  if (PHASE >= 1 && PHASE <= 3 && split == 0 && threadIdx.x == 0) {
    uint32_t* to = state + 4 * ((PHASE + 1) & 1);
    to[0] = border;
    to[1] = need;
    to[2] = done;
  }
}

struct To {
  const int32_t* table;  // [seqs][width]
  uint64_t stride;
};

// A workgroup takes a page of the kept positions and a head, a wave 16 of its
// tokens.  4-bit codes are moved with their scales; 8-bit ones get the largest
// scale that one of the page's tokens had, and those of smaller scales are
// divided by the growth and rounded again.
// Bound by memory as the layouts make it: 16 tokens' values lie in one line, so all of
// them are read where one of 16 positions is kept, and keys, 16 bytes of a token
// beside the next one's, by lines of 64.  64 sequences of 700-6,000 positions (8 heads
// of 128, 4 bits) to 1,024: 56 us for about 260 MB, 4.7 TB/s; with the values' codes
// loaded one by one 107 us.
template <int CODES, int D>
__global__ __launch_bounds__(1024) void k_move(CacheView c, SeqView s, To to, float* weights, const int32_t* positions,
                                               uint32_t keep) {
  constexpr bool kFour = CODES == LTC_E2M1;
  constexpr int PARTS = kFour ? D / 32 : D / 16, DROPS = (int)drop_bytes(D);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const uint32_t head = blockIdx.x, seq = blockIdx.z, P = 1u << c.page_log, first = blockIdx.y << c.page_log;
  const int32_t* from = positions + ((uint64_t)seq * c.heads + head) * keep;
  const int32_t* table = s.table + seq * s.table_stride;
  const uint32_t slots = min(keep - first, P);  // of the page, if as many are kept
  if (from[first] < 0) return;
  const uint32_t page = (uint32_t)to.table[seq * to.stride + blockIdx.y];
  if (page >= c.pages) {
    if (threadIdx.x == 0) report(c, kCacheBadPage);
    return;
  }
  // the lane's token: where it is
  const uint32_t slot = wave * 16 + n;
  const int32_t p = slot < slots ? from[first + slot] : -1;
  const uint32_t old = p >= 0 ? (uint32_t)table[(uint32_t)p >> c.page_log] : 0, off = (uint32_t)p & (P - 1);
  const bool live = p >= 0, have = live && old < c.pages;
  if (live && !have && g == 0) report(c, kCacheBadPage);
  int top[2] = {0, 0}, scale[2] = {0, 0};  // of the page, and of the lane's token
  if constexpr (!kFour) {
    for (uint32_t t = lane; t < slots; t += 64) {
      const int32_t x = from[first + t];
      const uint32_t o = x >= 0 ? (uint32_t)table[(uint32_t)x >> c.page_log] : c.pages;
      if (o >= c.pages) continue;
      const uint8_t* z = c.scales + ((uint64_t)o * c.heads + head) * 2;
      for (int i = 0; i < 2; ++i) top[i] = max(top[i], (int)z[i]);
    }
    for (int w = 32; w; w >>= 1)
      for (int i = 0; i < 2; ++i) top[i] = max(top[i], __shfl_xor(top[i], w));
    if (have)
      for (int i = 0; i < 2; ++i) scale[i] = c.scales[((uint64_t)old * c.heads + head) * 2 + i];
    if (threadIdx.x < 2) c.scales[((uint64_t)page * c.heads + head) * 2 + threadIdx.x] = (uint8_t)(threadIdx.x ? top[1] : top[0]);
  }
  if (__ballot(live) == 0) return;
  const uint32_t block = kFour ? 8 * D : 16 * D;
  const uint64_t src = head_offset(c, have ? old : 0, head) / (kFour ? 2 : 1) + (off >> 4) * block;
  const uint64_t dst = head_offset(c, page, head) / (kFour ? 2 : 1) + (uint32_t)wave * block;
  // ---- scales and weights
  if (g == 0 && live) {
    weights[(((uint64_t)page * c.heads + head) << c.page_log) + slot] =
        have ? weights[(((uint64_t)old * c.heads + head) << c.page_log) + off] : 0.0f;
    if constexpr (kFour) {
      const uint8_t* x = c.scales + token_scales(c, have ? old : 0, head);
      uint8_t* y = c.scales + token_scales(c, page, head);
      y[slot] = have ? x[off] : 27;
      y[P + slot] = have ? x[P + off] : 27;
      store_drops<DROPS>(y + 2 * P + slot * DROPS, have ? load_drops<DROPS>(x + 2 * P + off * DROPS) : 0);
    }
  }
  // ---- keys: 16 bytes of a token at a time; loaded here, stored behind the values
  constexpr int MINE = (PARTS + 3) / 4;
  uint4v key[MINE];
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    key[j] = uint4v{0, 0, 0, 0};
    if (have && 4 * j + g < PARTS) key[j] = *reinterpret_cast<const uint4v*>(c.k + src + (4 * j + g) * 256 + (off & 15) * 16);
  }
  // ---- values: the tokens come in order, so those of one block of 16 follow one
  // another.  A lane loads 16 bytes of a block (a dim, or two of 4 bits) for each of
  // its dims, of several blocks at a time, takes its tokens' codes out of them one by
  // one, and shifts each into the new 16 bytes from above.
  constexpr int LANES = kFour ? D / 2 : D, DIMS = (LANES + 63) / 64, AHEAD = DIMS > 2 ? 4 : 8;
  const uint32_t live_mask = (uint32_t)__ballot(live && g == 0) & 0xffffu;  // the first ones: positions end with -1
  const int tokens = __popc(live_mask);
  const uint32_t here = have ? (old << c.page_log | off) >> 4 : ~0u;  // the block that the token is in
  const uint32_t before = (uint32_t)__shfl_up((int)here, 1);  // asked by all lanes: one that is not asked has nothing to give
  const uint32_t begins = (uint32_t)__ballot(n == 0 || here != before) & live_mask;
  const uint64_t block_at = head_offset(c, have ? old : 0, head) / (kFour ? 2 : 1) + (off >> 4) * block;
  auto shift_in = [](uint4v& x, uint4v from, uint32_t o) {  // code o of 16 bytes into another 16
    if constexpr (kFour) {
#pragma unroll
      for (int dim = 0; dim < 2; ++dim) {
        const uint32_t code = (uint32_t)(((uint64_t)from[2 * dim + 1] << 32 | from[2 * dim]) >> (4 * o));
        x[2 * dim] = __builtin_amdgcn_alignbit(x[2 * dim + 1], x[2 * dim], 4);
        x[2 * dim + 1] = __builtin_amdgcn_alignbit(code, x[2 * dim + 1], 4);
      }
    } else {
      const uint32_t code = o < 8 ? __builtin_amdgcn_perm(from[1], from[0], o | 0x0c0c0c00u)
                                  : __builtin_amdgcn_perm(from[3], from[2], (o - 8) | 0x0c0c0c00u);
      for (int w = 0; w < 3; ++w) x[w] = __builtin_amdgcn_alignbyte(x[w + 1], x[w], 1);
      x[3] = __builtin_amdgcn_alignbyte(code, x[3], 1);
    }
  };
  uint4v x[DIMS], kept[DIMS];
#pragma unroll
  for (int k = 0; k < DIMS; ++k) {
    x[k] = kept[k] = uint4v{0, 0, 0, 0};
    if (tokens < 16 && lane + 64 * k < LANES) kept[k] = *reinterpret_cast<const uint4v*>(c.v + dst + (lane + 64 * k) * 16);
  }
  for (uint32_t left = begins; left;) {
    uint4v in[AHEAD][DIMS];
    uint32_t ahead = left;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = ahead ? __builtin_ctz(ahead) : 0;
      const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)block_at, t) |
                            (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(block_at >> 32), t) << 32;
      const bool want = ahead && __builtin_amdgcn_readlane((int)have, t);
#pragma unroll
      for (int k = 0; k < DIMS; ++k) {
        in[i][k] = uint4v{0, 0, 0, 0};
        if (want && lane + 64 * k < LANES) in[i][k] = *reinterpret_cast<const uint4v*>(c.v + base + (lane + 64 * k) * 16);
      }
      ahead &= ahead - 1;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (!left) break;
      const int t0 = __builtin_ctz(left);
      left &= left - 1;
      const int t1 = left ? __builtin_ctz(left) : tokens;
      for (int t = t0; t < t1; ++t) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)off, t) & 15;
#pragma unroll
        for (int k = 0; k < DIMS; ++k) {
          shift_in(x[k], in[i][k], o);
          if constexpr (!kFour) {
            const int z = __builtin_amdgcn_readlane(scale[1], t);
            if (z < top[1]) {  // the byte that has just come in, rounded again
              const float shrink = power_of_two(max(z - top[1], -126));
              const uint32_t code = to_codes<CODES == LTC_E4M3>(code_values<CODES == LTC_E4M3>(x[k][3] >> 24) * shrink);
              x[k][3] = (x[k][3] & 0xffffffu) | code << 24;
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    if constexpr (!kFour) {
      if (scale[0] < top[0]) {
        const float shrink = power_of_two(max(scale[0] - top[0], -126));
        for (int i = 0; i < 4; ++i) key[j][i] = to_codes<CODES == LTC_E4M3>(code_values<CODES == LTC_E4M3>(key[j][i]) * shrink);
      }
    }
    if (live && 4 * j + g < PARTS) *reinterpret_cast<uint4v*>(c.k + dst + (4 * j + g) * 256 + n * 16) = key[j];
  }
  for (int t = tokens; t < 16; ++t)  // what lies behind stays as it was
    for (int k = 0; k < DIMS; ++k) shift_in(x[k], kept[k], (uint32_t)t);
  for (int k = 0; k < DIMS; ++k)
    if (lane + 64 * k < LANES) *reinterpret_cast<uint4v*>(c.v + dst + (lane + 64 * k) * 16) = x[k];
}

template <int CODES> hipError_t launch_move(const CacheView& c, const SeqView& s, const To& to, const EvictArgs& a, hipStream_t st) {
  return for_numbers(LTC_BF16, c.dim, [&](auto, auto dim) {  // codes alone: the numbers' type does not matter
    const dim3 grid(c.heads, (a.keep + (1u << c.page_log) - 1) >> c.page_log, s.seqs);
    k_move<CODES, decltype(dim)::value><<<grid, 4u << c.page_log, 0, st>>>(c, s, to, a.weights, a.positions, a.keep);
  });
}

// One workgroup a sequence and head, or several where that leaves most of the chip
// idle and there are positions to share, as the table has room for them.  One / several
// for cuts to 256 of 60,000 positions (of 64 dims): 4 sequences and heads 48 / 28 us, 32
// of them 48 / 35, 64 54 / 54, 128 63 / 97, 512 140 / 341 us.  Of 9,000 positions 4 and
// 64 of them 17 / 25 and 17 / 30 us, of 1,000 in tables of 131,072 13 / 23 and 13 / 39
// us: there several are too many, and the host does not see the lengths.
uint32_t pick_splits(const CacheView& c, const SeqView& s) {
  const uint64_t pairs = (uint64_t)s.seqs * c.heads, capacity = capacity_of(c, s);
  if (pairs > 64 || capacity <= 2 * kRound) return 0;
  const uint64_t rounds = (capacity + kSplitRound - 1) / kSplitRound;
  return (uint32_t)(rounds < kMostSplits ? rounds : kMostSplits);
}

hipError_t launch_pick(const CacheView& c, const SeqView& s, const EvictArgs& a, hipStream_t st) {
  const uint32_t splits = pick_splits(c, s);
  if (splits) {
    const PickArgs p = {a.weights, a.keep, a.recent, a.lengths, a.positions, a.ws, splits};
    const dim3 grid(c.heads, splits, s.seqs);
    k_pick_split<0><<<grid, kSplitLanes, 0, st>>>(c, s, p);
    k_pick_split<1><<<grid, kSplitLanes, 0, st>>>(c, s, p);
    k_pick_split<2><<<grid, kSplitLanes, 0, st>>>(c, s, p);
    k_pick_split<3><<<grid, kSplitLanes, 0, st>>>(c, s, p);
    k_pick_split<4><<<grid, kSplitLanes, 0, st>>>(c, s, p);
    return hipGetLastError();
  }
  auto pick = [&](auto kernel) {
    kernel<<<dim3(c.heads, s.seqs), kPickLanes, 0, st>>>(c, s, a.weights, a.keep, a.recent, a.lengths, a.positions);
  };
  // what a sequence can have at most says how much shared memory its weights want:
  // two workgroups on a CU, or one
  if (capacity_of(c, s) <= 4 * kRound) pick(k_pick<4>);
  else pick(k_pick<8>);
  return hipGetLastError();
}

}  // namespace

uint64_t cache_evict_workspace(const CacheView& c, const SeqView& s) {
  const uint32_t splits = pick_splits(c, s);
  return splits ? (uint64_t)s.seqs * c.heads * split_words(splits) * sizeof(uint32_t) : 0;
}

hipError_t launch_cache_evict(const CacheView& c, const SeqView& s, int codes, const EvictArgs& a, hipStream_t st) {
  const hipError_t e = launch_pick(c, s, a, st);
  if (e != hipSuccess) return e;
  const To to = {a.to, a.to_stride};
  switch (codes) {
    case LTC_E4M3: return launch_move<LTC_E4M3>(c, s, to, a, st);
    case LTC_INT8: return launch_move<LTC_INT8>(c, s, to, a, st);
    case LTC_E2M1: return launch_move<LTC_E2M1>(c, s, to, a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace ltc
