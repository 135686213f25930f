// ltc_cache_weigh.h -- what each cached position was worth to a call's rows: the
// kernel, for the file of each code type to build.
#pragma once

#include "ltc_cache_attend.h"

namespace ltc {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

// Eight codes as numbers of the cache's own type, exactly (E2M1: times scale).
template <int CODES, int DT> __device__ __forceinline__ auto codes_as(uint32_t a, uint32_t b, float scale) {
  if constexpr (DT == LTC_FP16) {
    if constexpr (CODES == LTC_E2M1) return codes4_to_half(a, scale);
    else return codes_to_half<CODES>(a, b);
  } else {
    union {
      bf8 b8;
      bf2v b2[4];
      uint32_t u[4];
    } r;
    if constexpr (CODES == LTC_E2M1) {
      r.b2[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 0);
      r.b2[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 1);
      r.b2[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 2);
      r.b2[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 3);
    } else if constexpr (CODES == LTC_E4M3) {
      r.b2[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, 1.0f, false);
      r.b2[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, 1.0f, true);
      r.b2[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, 1.0f, false);
      r.b2[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, 1.0f, true);
    } else {
      const float4v x = code_values<false>(a), y = code_values<false>(b);
      r.u[0] = pack2<LTC_BF16>(x[0], x[1]);
      r.u[1] = pack2<LTC_BF16>(x[2], x[3]);
      r.u[2] = pack2<LTC_BF16>(y[0], y[1]);
      r.u[3] = pack2<LTC_BF16>(y[2], y[3]);
    }
    return r.b8;
  }
}

__device__ __forceinline__ float4v product(half8 a, half8 b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float4v product(bf8 a, bf8 b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The sums of v[t] over the 16 lanes n of a lane row; lane n gets that of t = n.
__device__ __forceinline__ float sum_scattered(float (&v)[16], int n) {
#pragma unroll
  for (int w = 8; w; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = n & w ? v[j] : v[j + w], keep = n & w ? v[j + w] : v[j];
      v[j] = keep + __shfl_xor(send, w);
    }
  return v[0];
}

// A wave takes 64 positions of a sequence and head and goes over all rows that see
// them, 16 packed rows at a time: the products are k_attend_rows's first ones, in
// the cache's own type.  A lane holds the weights of 16 positions from one row,
// 2^(x - lse), adds them up over the rows, and at the end 16 lanes' sums are
// joined.  No two waves have a position in common, so the sums' order is fixed.
template <int CODES, int DT, int D>
__global__ __launch_bounds__(64 * kWaves) void k_weigh(CacheView c, SeqView s, AttendArgs a, float* weights, uint32_t splits,
                                                       uint32_t per_head) {
  constexpr bool kFour = CODES == LTC_E2M1;
  constexpr int KS = D / 32, KL = D / 64;
  constexpr uint32_t kBlockBytes = kFour ? 8 * D : 16 * D;
  typedef decltype(codes_as<CODES, DT>(0, 0, 0.0f)) Eight;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
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
  for (int step = lo / kStep + (int)split * kWaves + wave; step * kStep < len; step += (int)splits * kWaves) {
    const int t0 = step * kStep;
    auto page_of = [&](int t) -> uint32_t { return t < len ? (uint32_t)table[(uint32_t)t >> c.page_log] : ~0u; };
    const int tk = t0 + kb * 16, tv = t0 + g * 16;
    const uint32_t k_page = page_of(tk), v_page = page_of(tv);
    const bool have = v_page < c.pages;
    const uint32_t kp = k_page < c.pages ? k_page : 0, vp = have ? v_page : 0;
    const uint8_t* k = c.k + head_offset(c, kp, head) / (kFour ? 2 : 1) + (((uint32_t)tk & page_mask) >> 4) * kBlockBytes +
                       (n & 3) * 16;
    Eight key[4][KS];
    uint4v ke = {0, 0, 0, 0};
    if constexpr (kFour) {
      const uint8_t* drops = c.scales + token_scales(c, kp, head) + 2 * (page_mask + 1) +
                             (((uint32_t)tk & page_mask) + (n & 3)) * drop_bytes(D);
      Keys4<D> kq[4];
      for (int b = 0; b < 4; ++b) kq[b].load(k + b * 64, drops + 4 * b * drop_bytes(D), g);
      ke = *reinterpret_cast<const uint4v*>(c.scales + token_scales(c, vp, head) + ((uint32_t)tv & page_mask));
      for (int b = 0; b < 4; ++b)
        for (int x = 0; x < KS; ++x) key[b][x] = codes_as<CODES, DT>(kq[b].c[x], 0, kq[b].scale(x, g));
    } else {
      uint4v kr[4][KL];
      uint2v kt[4];
      for (int b = 0; b < 4; ++b) {
        for (int j = 0; j < KL; ++j) kr[b][j] = *reinterpret_cast<const uint4v*>(k + g * 256 + j * 1024 + b * 64);
        if constexpr (D % 64) kt[b] = *reinterpret_cast<const uint2v*>(k + KL * 1024 + (g >> 1) * 256 + (g & 1) * 8 + b * 64);
      }
      ke[0] = c.scales[((uint64_t)vp * c.heads + head) * 2];
      for (int b = 0; b < 4; ++b)
        for (int x = 0; x < KS; ++x)
          key[b][x] = x < 2 * KL ? codes_as<CODES, DT>(kr[b][x / 2][(x & 1) * 2], kr[b][x / 2][(x & 1) * 2 + 1], 1.0f)
                                 : codes_as<CODES, DT>(kt[b][0], kt[b][1], 1.0f);
    }
    float sum[16];
    for (int t = 0; t < 16; ++t) sum[t] = 0.0f;
    // the rows at positions from t0 on, and with a window before t0 + 63 + window
    const uint32_t ra = (t0 > start ? (uint32_t)(t0 - start) : 0) * G;
    const uint32_t rb = (window ? min(sp.n, (uint32_t)max((int64_t)t0 + 63 + window - start, (int64_t)0)) : sp.n) * G;
    for (uint32_t r0 = ra; r0 < rb; r0 += 16) {
      const uint32_t r = r0 + n;
      const bool live = r < rb;
      const uint32_t token = live ? r / G : 0, qh = head * G + (live ? r % G : 0);
      const uint64_t row = sp.row0 + token;
      const uint16_t* src = a.q.base + row * a.q.row_stride + (uint64_t)qh * a.q.head_stride;
      Eight q[KS];
      for (int x = 0; x < KS; ++x) q[x] = *reinterpret_cast<const Eight*>(src + dim_of<CODES, D>(x, g));
      const float lse = a.lse[row * a.q_heads + qh];
      float4v st[4];
      for (int b = 0; b < 4; ++b) st[b] = float4v{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int b = 0; b < 4; ++b) st[b] = product(key[b][x], q[x], st[b]);
      const int hi = live ? start + (int)token + 1 : 0, low = window ? hi - window : 0;
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 4; ++i) {
          const int t = tv + 4 * b + i, e = (int)(kFour ? ke[b] >> (8 * i) & 0xff : ke[0]) - 127;
          const float p = __builtin_amdgcn_exp2f(fmaf(__builtin_amdgcn_ldexpf(st[b][i], e), f, -lse));
          sum[4 * b + i] += t < hi && t >= low ? p : 0.0f;
        }
    }
    const float w = sum_scattered(sum, n);
    const int t = tv + n;
    if (t < len && have) {
      float* at = weights + (((uint64_t)v_page * c.heads + head) << c.page_log) + ((uint32_t)t & page_mask);
      *at = (t < start ? *at : 0.0f) + w;
    }
  }
}

}  // namespace

template <int CODES>
hipError_t launch_weigh(const CacheView& c, const SeqView& s, int dtype, const AttendArgs& a, float* weights, hipStream_t st) {
  uint64_t longest = (uint64_t)s.width << c.page_log;
  if (longest > kMaxPositions) longest = kMaxPositions;
  const uint64_t most = (longest + kStep * kWaves - 1) / (kStep * kWaves);
  const uint64_t base = (uint64_t)s.seqs * c.heads, want = (1024 + base - 1) / base;
  const uint32_t splits = (uint32_t)(want < most ? want : most < 1 ? 1 : most);
  const uint32_t share = chiplet_share(c.heads);
  const uint32_t per_head = (s.seqs * splits + share - 1) / share * share;
  const uint64_t groups = (uint64_t)per_head * c.heads;
  const dim3 grid((uint32_t)(groups < kGridWidth ? groups : kGridWidth), (uint32_t)((groups + kGridWidth - 1) / kGridWidth));
  return for_numbers(dtype, c.dim, [&](auto type, auto dim) {
    k_weigh<CODES, decltype(type)::value, decltype(dim)::value><<<grid, 64 * kWaves, 0, st>>>(c, s, a, weights, splits, per_head);
  });
}

}  // namespace ltc
