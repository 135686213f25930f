// ltc_cache_evict.hip -- a cache cut to the positions of most weight: which they
// are (k_pick), and their move to other pages (k_move).
#include "ltc_cache_device.h"

namespace ltc {
namespace {

constexpr int kPickLanes = 1024, kPickWaves = kPickLanes / 64;

// A number's place in the order of weights, as an unsigned one; a NaN is below
// all others, and the zeros are equal.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x != x ? 0 : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// A workgroup takes a sequence and head.  The least weight that is kept is found
// digit by digit (8 bits) from histograms in shared memory; then the positions
// are gone through in order and the kept ones written one behind the other.
__global__ __launch_bounds__(kPickLanes) void k_pick(CacheView c, SeqView s, const float* weights, uint32_t keep,
                                                     uint32_t recent, int32_t* lengths, int32_t* positions) {
  __shared__ uint32_t counts[kPickWaves][256];
  __shared__ uint32_t sums[2][kPickWaves];
  __shared__ uint32_t found[2];
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
  const int32_t* table = s.table + seq * s.table_stride;
  const uint32_t mask = (1u << c.page_log) - 1, others = n - recent;
  auto key_of = [&](uint32_t t) -> uint32_t {
    const uint32_t page = (uint32_t)table[t >> c.page_log];
    return page < c.pages ? order_of(weights[(((uint64_t)page * c.heads + head) << c.page_log) + (t & mask)]) : 0;
  };
  uint32_t need = keep - recent, border = 0;  // `need` of those that begin with border's digits so far are kept
  for (int shift = 24; shift >= 0 && need; shift -= 8) {
    for (int i = lane; i < 256; i += 64) counts[wave][i] = 0;
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < others; t += kPickLanes) {
      const uint32_t key = key_of(t);
      if (shift == 24 || (key ^ border) >> (shift + 8) == 0) atomicAdd(&counts[wave][key >> shift & 255], 1u);
    }
    __syncthreads();
    if (wave == 0) {
      uint32_t mine[4], sum = 0;  // digits 255 - 4 lane and the three below it
      for (int i = 0; i < 4; ++i) {
        mine[i] = 0;
        for (int w = 0; w < kPickWaves; ++w) mine[i] += counts[w][255 - 4 * lane - i];
        sum += mine[i];
      }
      uint32_t above = sum;  // those of this lane's digits and higher ones
      for (int w = 1; w < 64; w <<= 1) {
        const uint32_t x = __shfl_up(above, w);
        if (lane >= w) above += x;
      }
      above -= sum;
      for (int i = 0; i < 4; ++i) {
        if (above < need && need <= above + mine[i]) {
          found[0] = 255 - 4 * lane - i;
          found[1] = need - above;
        }
        above += mine[i];
      }
    }
    __syncthreads();
    border |= found[0] << shift;
    need = found[1];
  }
  // `need` of the weights equal to the border are kept, the first ones
  const bool none = keep == recent;
  uint32_t kept = 0, equal = 0;
  for (uint32_t t0 = 0; t0 < others && !none; t0 += kPickLanes) {
    const uint32_t t = t0 + threadIdx.x;
    const uint32_t key = t < others ? key_of(t) : 0;
    const bool more = t < others && key > border, same = t < others && key == border;
    const uint64_t below = (1ull << lane) - 1, b_more = __ballot(more), b_same = __ballot(same);
    if (lane == 0) {
      sums[0][wave] = __popcll(b_more);
      sums[1][wave] = __popcll(b_same);
    }
    __syncthreads();
    uint32_t more0 = 0, same0 = 0, more1 = 0, same1 = 0;  // of the waves before this one, and of all
    for (int w = 0; w < kPickWaves; ++w) {
      if (w == wave) {
        more0 = more1;
        same0 = same1;
      }
      more1 += sums[0][w];
      same1 += sums[1][w];
    }
    const uint32_t e = equal + same0 + __popcll(b_same & below);  // equal ones before this
    const uint32_t at = kept + more0 + __popcll(b_more & below) + min(e, need) - min(equal, need);
    if (more || (same && e < need)) out[at] = (int32_t)t;
    kept += more1 + min(equal + same1, need) - min(equal, need);
    equal += same1;
    __syncthreads();
  }
  for (uint32_t i = threadIdx.x; i < recent; i += kPickLanes) out[keep - recent + i] = (int32_t)(others + i);
}

struct To {
  const int32_t* table;  // [seqs][width]
  uint64_t stride;
};

// A workgroup takes a page of the kept positions and a head, a wave 16 of its
// tokens.  4-bit codes are moved with their scales; 8-bit ones get the largest
// scale that one of the page's tokens had, and those of smaller scales are
// divided by the growth and rounded again.
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
      for (int i = 0; i < DROPS; ++i) y[2 * P + slot * DROPS + i] = have ? x[2 * P + off * DROPS + i] : 0;
    }
  }
  // ---- keys: 16 bytes of a token at a time
  for (int j = g; j < PARTS; j += 4) {
    uint4v x = {0, 0, 0, 0};
    if (have) x = *reinterpret_cast<const uint4v*>(c.k + src + j * 256 + (off & 15) * 16);
    if constexpr (!kFour) {
      if (scale[0] < top[0]) {
        const float shrink = power_of_two(max(scale[0] - top[0], -126));
        for (int i = 0; i < 4; ++i) x[i] = to_codes<CODES == LTC_E4M3>(code_values<CODES == LTC_E4M3>(x[i]) * shrink);
      }
    }
    if (live) *reinterpret_cast<uint4v*>(c.k + dst + j * 256 + n * 16) = x;
  }
  // ---- values: a lane has a dim, and its 16 tokens' codes one by one
  const int tokens = __popcll(__ballot(live && g == 0));
  for (int d = lane; d < D; d += 64) {
    if constexpr (kFour) {
      uint2v* at = reinterpret_cast<uint2v*>(c.v + dst + d * 8);
      uint2v x = tokens < 16 ? *at : uint2v{0, 0};
      for (int t = 0; t < tokens; ++t) {
        const uint64_t base = __shfl((unsigned long long)src, t);
        const uint32_t o = __shfl(off, t) & 15;
        uint32_t code = c.v[base + d * 8 + o / 2] >> (4 * (o & 1)) & 15;
        if (!__shfl((int)have, t)) code = 0;
        const int at_bit = 4 * (t & 7);
        x[t >> 3] = (x[t >> 3] & ~(15u << at_bit)) | code << at_bit;
      }
      *at = x;
    } else {
      uint4v* at = reinterpret_cast<uint4v*>(c.v + dst + d * 16);
      uint4v x = tokens < 16 ? *at : uint4v{0, 0, 0, 0};
      for (int t = 0; t < tokens; ++t) {
        const uint64_t base = __shfl((unsigned long long)src, t);
        uint32_t code = c.v[base + d * 16 + (__shfl(off, t) & 15)];
        if (!__shfl((int)have, t)) code = 0;
        const int z = __shfl(scale[1], t);
        if (z < top[1])
          code = to_codes<CODES == LTC_E4M3>(code_values<CODES == LTC_E4M3>(code) * power_of_two(max(z - top[1], -126))) & 0xff;
        const int at_bit = 8 * (t & 3);
        x[t >> 2] = (x[t >> 2] & ~(255u << at_bit)) | code << at_bit;
      }
      *at = x;
    }
  }
}

template <int CODES> hipError_t launch_move(const CacheView& c, const SeqView& s, const To& to, const EvictArgs& a, hipStream_t st) {
  return for_numbers(LTC_BF16, c.dim, [&](auto, auto dim) {  // codes alone: the numbers' type does not matter
    const dim3 grid(c.heads, (a.keep + (1u << c.page_log) - 1) >> c.page_log, s.seqs);
    k_move<CODES, decltype(dim)::value><<<grid, 4u << c.page_log, 0, st>>>(c, s, to, a.weights, a.positions, a.keep);
  });
}

}  // namespace

hipError_t launch_cache_evict(const CacheView& c, const SeqView& s, int codes, const EvictArgs& a, hipStream_t st) {
  k_pick<<<dim3(c.heads, s.seqs), kPickLanes, 0, st>>>(c, s, a.weights, a.keep, a.recent, a.lengths, a.positions);
  hipError_t e = hipGetLastError();
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
