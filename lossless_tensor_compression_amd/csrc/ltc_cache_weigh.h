// ltc_cache_weigh.h -- what each cached position was worth to a call's rows: the
// kernel, for the file of each code type to build.
#pragma once

#include "ltc_cache_attend.h"

namespace ltc {
namespace {

// The sums of v[t] over the 16 lanes n of a lane row; lane n gets that of t = n.
__device__ __forceinline__ float sum_scattered(float (&v)[16], int n) {
#pragma unroll
  for (int w = 8; w; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) {
      float x = v[j], y = v[j + w];
      asm("" : "+v"(x), "+v"(y));  // two registers, not one array with a place to be found by comparisons
      const float send = n & w ? x : y, keep = n & w ? y : x;
      v[j] = keep + __shfl_xor(send, w);
    }
  return v[0];
}

// Waves for each SIMD that the kernel's registers are to leave room for: as many as go
// without spills (but for 256 dims' one wave where rows are shared).  40 single rows at
// 500-5,000 positions of 8 heads of 128 dims with 2 / 3: 39 / 34 us.
constexpr int weigh_occupancy(int D, bool share) { return D <= 128 ? share && D > 64 ? 2 : 3 : D <= 192 || !share ? 2 : 1; }

// A step's keys as they lie in memory.
template <int CODES, int D> struct RawKeys {
  static constexpr bool kFour = CODES == LTC_E2M1;
  static constexpr int KL = D / 64;
  Keys4<kFour ? D : 32> four[4];
  uint4v wide[4][kFour ? 1 : KL];
  uint2v tail[4];
  // the same, to the compiler other ones: what is made of them is not kept over a loop
  __device__ __forceinline__ void forget() {
    for (int b = 0; b < 4; ++b) {
      if constexpr (kFour) {
        for (int x = 0; x < D / 32; ++x) asm("" : "+v"(four[b].c[x]));
      } else {
        for (int j = 0; j < KL; ++j) asm("" : "+v"(wide[b][j]));
        if constexpr (D % 64) asm("" : "+v"(tail[b]));
      }
    }
  }
  // product x's part of block b
  template <int DT> __device__ __forceinline__ auto as(int b, int x, int g) const {
    if constexpr (kFour) return codes_as<CODES, DT>(four[b].c[x], 0, four[b].scale(x, g));
    else return x < 2 * KL ? codes_as<CODES, DT>(wide[b][x / 2][(x & 1) * 2], wide[b][x / 2][(x & 1) * 2 + 1], 1.0f)
                           : codes_as<CODES, DT>(tail[b][0], tail[b][1], 1.0f);
  }
};

// A wave takes 64 positions of a sequence and head and goes over rows that see
// them, 16 packed rows at a time: the products are k_attend_rows's first ones, in
// the cache's own type.  A lane holds the weights of 16 positions from one row,
// 2^(x - lse), adds them up over the rows, and at the end 16 lanes' sums are
// joined.  The order of all sums is fixed.
//
// Bound by the vector units and by what they wait for: two prompts of 1,500-2,100 rows
// (6 heads of 64, 12 query heads, a window of 1,600) 35 us, in half of which a vector
// instruction issues, 103 for 16 rows and 64 positions, 16 of them exponentials; matrix
// cores are busy for 16%.
//
// SHARE: a workgroup's waves have the same positions and share the rows out, for
// prompts; else each wave has every W-th step, for few rows.
template <int CODES, int DT, int D, bool SHARE, int W>
__global__ __launch_bounds__(64 * W, weigh_occupancy(D, SHARE)) void k_weigh(CacheView c, SeqView s, AttendArgs a, float* weights, uint32_t splits,
                                                  uint32_t per_head) {
  constexpr bool kFour = CODES == LTC_E2M1;
  constexpr int KS = D / 32, KL = D / 64;
  constexpr uint32_t kBlockBytes = kFour ? 8 * D : 16 * D;
  typedef decltype(codes_as<CODES, DT>(0, 0, 0.0f)) Eight;
  __shared__ float parts[SHARE ? W : 1][kStep];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t head, seq, split;
  place(blockIdx.x + gridDim.x * blockIdx.y, c.heads, splits, per_head, &head, &seq, &split);
  if (head >= c.heads || seq >= s.seqs) return;
  const Span sp = load_span(c, s, seq);
  if (!sp.ok || !sp.n || c.pages == 0) return;
  const uint32_t G = a.q_heads / c.heads;
  const int start = (int)sp.start, len = (int)sp.len, window = (int)a.window;
  const int lo = window && start + 1 > window ? start + 1 - window : 0;
  const uint32_t page_mask = (1u << c.page_log) - 1;
  const int32_t* table = s.table + seq * s.table_stride;
  const float f = fmaxf(a.scale * kLog2e * (kFour ? power_of_two(-kLift) : 1.0f), 0x1p-126f);
  const int kb = n >> 2;
  const int by = SHARE ? (int)splits : (int)splits * W;  // steps from one of the wave's to the next
  int step = lo / kStep + (SHARE ? (int)split : (int)split * W + wave);
  auto page_of = [&](int t) -> uint32_t { return t < len ? (uint32_t)table[(uint32_t)t >> c.page_log] : ~0u; };
  // a step's keys are loaded a step ahead, its pages two
  RawKeys<CODES, D> raw;
  uint4v exps = {0, 0, 0, 0};
  uint32_t k_page = page_of(step * kStep + kb * 16), v_page = page_of(step * kStep + g * 16), now_page = ~0u;
  auto load = [&](int at) {
    const int tk = at * kStep + kb * 16, tv = at * kStep + g * 16;
    const uint32_t kp = k_page < c.pages ? k_page : 0, vp = v_page < c.pages ? v_page : 0;
    const uint8_t* k = c.k + head_offset(c, kp, head) / (kFour ? 2 : 1) + (((uint32_t)tk & page_mask) >> 4) * kBlockBytes +
                       (n & 3) * 16;
    if constexpr (kFour) {
      const uint8_t* drops = c.scales + token_scales(c, kp, head) + 2 * (page_mask + 1) +
                             (((uint32_t)tk & page_mask) + (n & 3)) * drop_bytes(D);
      for (int b = 0; b < 4; ++b) raw.four[b].load(k + b * 64, drops + 4 * b * drop_bytes(D), g);
      exps = *reinterpret_cast<const uint4v*>(c.scales + token_scales(c, vp, head) + ((uint32_t)tv & page_mask));
    } else {
      for (int b = 0; b < 4; ++b) {
        for (int j = 0; j < KL; ++j) raw.wide[b][j] = *reinterpret_cast<const uint4v*>(k + g * 256 + j * 1024 + b * 64);
        if constexpr (D % 64) raw.tail[b] = *reinterpret_cast<const uint2v*>(k + KL * 1024 + (g >> 1) * 256 + (g & 1) * 8 + b * 64);
      }
      exps[0] = c.scales[((uint64_t)vp * c.heads + head) * 2];
    }
    now_page = v_page;
    k_page = page_of((at + by) * kStep + kb * 16);
    v_page = page_of((at + by) * kStep + g * 16);
  };
  if (!SHARE && step * kStep < len) load(step);
  for (; step * kStep < len; step += by) {
    const int t0 = step * kStep, tv = t0 + g * 16;
    if constexpr (SHARE) load(step);  // many rows make up for the wait, and registers are for more waves
    const uint32_t page = now_page;
    const bool have = page < c.pages;
    const int t = tv + n;  // whose weight the lane has in the end
    float* at = weights + (((uint64_t)(have ? page : 0) * c.heads + head) << c.page_log) + ((uint32_t)t & page_mask);
    const bool mine = t >= lo && t < len && have && (!SHARE || wave == 0);  // what no row sees is not touched
    const float before = mine && t < start ? *at : 0.0f;
    // many rows: the keys are turned into numbers once; few: for each 16 rows again,
    // which leaves registers for more waves
    RawKeys<CODES, D> now = raw;
    Eight key[SHARE ? 4 : 1][SHARE ? KS : 1];
    if constexpr (SHARE)
      for (int b = 0; b < 4; ++b)
        for (int x = 0; x < KS; ++x) key[b][x] = now.template as<DT>(b, x, g);
    // what a token's products are multiplied with: log2(e) scale times the keys' scale
    float by_token[kFour ? 16 : 1];
    if constexpr (kFour) {
      for (int t = 0; t < 16; ++t) by_token[t] = fmaxf(__builtin_amdgcn_ldexpf(f, (int)(exps[t / 4] >> (8 * (t % 4)) & 0xff) - 127), 0x1p-126f);
    } else {
      by_token[0] = fmaxf(__builtin_amdgcn_ldexpf(f, (int)exps[0] - 127), 0x1p-126f);
    }
    if (!SHARE && (step + by) * kStep < len) load(step + by);
    float sum[16];
    for (int t = 0; t < 16; ++t) sum[t] = 0.0f;
    // the rows at positions from t0 on, and with a window before t0 + 63 + window
    const uint32_t ra = (t0 > start ? (uint32_t)(t0 - start) : 0) * G;
    const uint32_t rb = (window ? min(sp.n, (uint32_t)max((int64_t)t0 + 63 + window - start, (int64_t)0)) : sp.n) * G;
    uint32_t r0 = ra + (SHARE ? 16 * wave : 0);
    constexpr uint32_t R = SHARE ? 16 * W : 16;
    // row r0 + n as token and query head, counted on
    uint32_t token = (r0 + n) / G, qh = (r0 + n) % G;
    const uint32_t token_by = R / G, qh_by = R % G;
    Eight q[KS];
    float lse = 0.0f;
    auto load_row = [&] {
      const uint64_t row = sp.row0 + min(token, sp.n - 1);
      const uint16_t* src = a.q.base + row * a.q.row_stride + (uint64_t)(head * G + qh) * a.q.head_stride;
      for (int x = 0; x < KS; ++x) q[x] = *reinterpret_cast<const Eight*>(src + dim_of<CODES, D>(x, g));
      lse = a.lse[row * a.q_heads + head * G + qh];
    };
    if (r0 < rb) load_row();
    for (; r0 < rb; r0 += R) {
      if constexpr (!SHARE) now.forget();
      float4v st[4];
      for (int b = 0; b < 4; ++b) st[b] = float4v{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if constexpr (SHARE) st[b] = product(key[b][x], q[x], st[b]);
          else st[b] = product(now.template as<DT>(b, x, g), q[x], st[b]);
        }
      const float less = lse;
      // all rows see all of the step's positions, or masks are needed
      const int first = start + __builtin_amdgcn_readlane((int)token, 0), last = start + __builtin_amdgcn_readlane((int)token, 15);
      const bool edge = r0 + 16 > rb || some_hidden(t0, t0 + kStep, first, last, a.window);
      const int hi = r0 + n < rb ? start + (int)token + 1 : 0, low = window ? hi - window : 0;
      token += token_by;
      qh += qh_by;
      if (qh >= G) {
        qh -= G;
        ++token;
      }
      if (r0 + R < rb) load_row();
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 4; ++i) st[b][i] = fmaf(st[b][i], by_token[kFour ? 4 * b + i : 0], -less);
      if (edge) {
        asm volatile("");  // a branch: as selections by `edge` these were most of the loop
        for (int b = 0; b < 4; ++b)
          for (int i = 0; i < 4; ++i) {
            const int t = tv + 4 * b + i;
            st[b][i] = t < hi && t >= low ? st[b][i] : -INFINITY;
          }
      }
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 4; ++i) sum[4 * b + i] += __builtin_amdgcn_exp2f(st[b][i]);
    }
    float w = sum_scattered(sum, n);
    if constexpr (SHARE) {
      parts[wave][lane] = w;
      __syncthreads();
      if (wave == 0) {
        w = 0.0f;
        for (int v = 0; v < W; ++v) w += parts[v][lane];
      }
      __syncthreads();
    }
    if (mine) *at = before + w;
  }
}

}  // namespace

template <int CODES>
hipError_t launch_weigh(const CacheView& c, const SeqView& s, int dtype, const AttendArgs& a, float* weights, hipStream_t st) {
  uint64_t longest = (uint64_t)s.width << c.page_log;
  if (longest > kMaxPositions) longest = kMaxPositions;
  const uint64_t steps = (longest + kStep - 1) / kStep, base = (uint64_t)s.seqs * c.heads;
  const uint64_t mean = ((uint64_t)s.rows * (a.q_heads / c.heads) + s.seqs - 1) / s.seqs;  // packed rows of a sequence and head
  // A workgroup's waves share the rows where there are many for each step, or fewer
  // steps than waves to fill the chip; else a step's keys are loaded and turned once.
  // sharing / not: 16 times 32, 64, 128 and 400 packed rows behind 500-5,000 positions
  // (8 heads of 128) 38 / 19, 43 / 27, 53 / 46 and 40 / 46 us, 6 and 16 prompts of
  // 8,192 245 / 469 and 621 / 861 us; one of 64 behind 5,000 in 2 heads 4.3 / 6.4 us.
  const bool share = mean > 256 || (mean > 16 && base * steps < 4096);
  const uint64_t most = share ? steps : (steps + kWaves - 1) / kWaves, want = ((share ? 4096 : 1536) + base - 1) / base;
  const uint32_t splits = (uint32_t)(want < most ? want : most < 1 ? 1 : most);
  const uint32_t apart = chiplet_share(c.heads);
  const uint32_t per_head = (s.seqs * splits + apart - 1) / apart * apart;
  const uint64_t groups = (uint64_t)per_head * c.heads;
  const dim3 grid((uint32_t)(groups < kGridWidth ? groups : kGridWidth), (uint32_t)((groups + kGridWidth - 1) / kGridWidth));
  return for_numbers(dtype, c.dim, [&](auto type, auto dim) {
    constexpr int DT = decltype(type)::value, D = decltype(dim)::value;
    constexpr int kShareWaves = 4;
    if (share)
      k_weigh<CODES, DT, D, true, kShareWaves><<<grid, 64 * kShareWaves, 0, st>>>(c, s, a, weights, splits, per_head);
    else
      k_weigh<CODES, DT, D, false, kWaves><<<grid, 64 * kWaves, 0, st>>>(c, s, a, weights, splits, per_head);
  });
}

}  // namespace ltc
