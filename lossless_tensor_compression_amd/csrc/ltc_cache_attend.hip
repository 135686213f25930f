// ltc_cache_attend.hip -- attention of new queries over the 8-bit cache.
#include "ltc_cache_device.h"

namespace ltc {
namespace {

constexpr int kMaxDim = 256;

// One wave for a row and query head: one pass over the positions it sees with
// the running maximum and sum of the softmax; lanes over the head's dims.
template <bool E4M3, int DT>
__global__ __launch_bounds__(64) void k_cache_attend(CacheView c, SeqView s, AttendArgs a) {
  const uint32_t row = blockIdx.x, qh = blockIdx.y, lane = threadIdx.x;
  const uint32_t head = qh / (a.q_heads / c.heads);
  const UnitMap map{1, 1, 0};
  uint32_t seq;
  Span sp;
  uint64_t own;
  const bool mine = locate_unit(c, s, map, row, WaveCount{s, map, row}, &seq, &sp, &own) && own < sp.n;
  if (!sp.ok && lane == 0) report(c, kCacheBadSeq);
  constexpr int N = kMaxDim / 64;
  float q[N], acc[N];
  for (int i = 0; i < N; ++i) {
    const uint32_t d = i * 64 + lane;
    q[i] = d < c.dim ? widen<DT>(a.q.base[row * a.q.row_stride + qh * a.q.head_stride + d]) * a.scale : 0.0f;
    acc[i] = 0.0f;
  }
  float m = -INFINITY, sum = 0.0f;
  if (sp.ok && mine) {
    const uint32_t end = sp.start + (uint32_t)own + 1;
    uint32_t t = a.window && end > a.window ? end - a.window : 0;
    for (; t < end; ++t) {
      uint32_t page;
      if (!page_at(s, seq, t >> c.page_log, c.pages, &page)) {
        if (lane == 0) report(c, kCacheBadPage);
        continue;
      }
      const uint8_t* kc = c.k + head_offset(c, page, head);
      const uint8_t* vc = c.v + head_offset(c, page, head);
      const uint8_t* scales = c.scales + ((uint64_t)page * c.heads + head) * 2;
      const float ks = power_of_two(scales[0] - 127), vs = power_of_two(scales[1] - 127);
      const uint32_t o = t & ((1u << c.page_log) - 1);
      float x = 0.0f;
      for (int i = 0; i < N; ++i) {
        const uint32_t d = i * 64 + lane;
        if (d < c.dim) x += q[i] * code_value<E4M3>(kc[k_code(o, d, c.dim)]);
      }
      for (int w = 32; w; w >>= 1) x += __shfl_xor(x, w);
      x *= ks;
      const float top = fmaxf(m, x), keep = expf(m - top), p = expf(x - top);
      m = top;
      sum = sum * keep + p;
      for (int i = 0; i < N; ++i) {
        const uint32_t d = i * 64 + lane;
        acc[i] = acc[i] * keep + (d < c.dim ? p * (code_value<E4M3>(vc[v_code(o, d, c.dim)]) * vs) : 0.0f);
      }
    }
  }
  for (int i = 0; i < N; ++i) {
    const uint32_t d = i * 64 + lane;
    if (d < c.dim) a.out[((uint64_t)row * a.q_heads + qh) * c.dim + d] = narrow<DT>(sum == 0.0f ? 0.0f : acc[i] / sum);
  }
}

}  // namespace

uint64_t cache_attend_workspace(const CacheView&, const SeqView&, uint32_t, uint32_t) { return 0; }

hipError_t launch_cache_attend(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const AttendArgs& a,
                               hipStream_t st) {
  const dim3 grid(s.rows, a.q_heads);
  if (e4m3) {
    if (dtype == LTC_BF16) k_cache_attend<true, LTC_BF16><<<grid, 64, 0, st>>>(c, s, a);
    else k_cache_attend<true, LTC_FP16><<<grid, 64, 0, st>>>(c, s, a);
  } else {
    if (dtype == LTC_BF16) k_cache_attend<false, LTC_BF16><<<grid, 64, 0, st>>>(c, s, a);
    else k_cache_attend<false, LTC_FP16><<<grid, 64, 0, st>>>(c, s, a);
  }
  return hipGetLastError();
}

}  // namespace ltc
