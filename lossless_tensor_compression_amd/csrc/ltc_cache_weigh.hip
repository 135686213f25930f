// ltc_cache_weigh.hip -- positions' weights from scores that the attention wrote
// down.
#include "ltc_cache_device.h"

namespace ltc {
namespace {

constexpr int kWeighLanes = 256, kWeighEach = 4 * kWeighLanes;  // positions of a workgroup at a time

// 2^(score - lse), summed over the rows that see a position and the head's query
// heads, in order.  A lane takes four positions.  Bound by memory: four bytes for
// each score, eight for each position's weight.  40 rows at 500-5,000 positions (8
// heads, 32 query heads: 23 MB) 9.7 us.
__global__ __launch_bounds__(kWeighLanes) void k_weigh_scores(CacheView c, SeqView s, AttendArgs a, float* weights, uint32_t splits) {
  constexpr int AHEAD = 8;  // rows whose scores are in flight
  const uint32_t id = blockIdx.x + gridDim.x * blockIdx.y, split = id % splits, head = id / splits % c.heads;
  const uint32_t seq = id / splits / c.heads;
  if (seq >= s.seqs) return;
  const Span sp = load_span(c, s, seq);
  if (!sp.ok || !sp.n || c.pages == 0) return;
  const uint32_t G = a.q_heads / c.heads, rows = sp.n * G, mask = (1u << c.page_log) - 1;
  const int start = (int)sp.start, len = (int)sp.len, window = (int)a.window;
  const int lo = window && start + 1 > window ? start + 1 - window : 0;
  const int32_t* table = s.table + seq * s.table_stride;
  const int from = (int)score_first(sp.start, a.window);
  const uint64_t first = (uint64_t)sp.row0 * a.q_heads + head * G;
  // from the first position that a row sees: those before it are not touched
  for (int t = lo / 4 * 4 + (int)split * kWeighEach + 4 * (int)threadIdx.x; t < len; t += (int)splits * kWeighEach) {
    const uint32_t page = (uint32_t)table[(uint32_t)t >> c.page_log];
    if (page >= c.pages) continue;
    float* at = weights + (((uint64_t)page * c.heads + head) << c.page_log) + ((uint32_t)t & mask);
    const float4v before = *reinterpret_cast<const float4v*>(at);
    float4v sum = {0, 0, 0, 0};
    for (uint32_t r0 = 0; r0 < rows; r0 += AHEAD) {
      float4v x[AHEAD];
      float lse[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const uint32_t r = min(r0 + i, rows - 1);
        const uint64_t row = first + (uint64_t)(r / G) * a.q_heads + r % G;
        x[i] = *reinterpret_cast<const float4v*>(a.scores + row * a.scores_stride + (t - from));
        lse[i] = a.lse[row];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int hi = r0 + i < rows ? start + (int)((r0 + i) / G) + 1 : 0, low = window ? hi - window : 0;
        for (int j = 0; j < 4; ++j)
          sum[j] += t + j < hi && t + j >= low ? __builtin_amdgcn_exp2f(x[i][j] - lse[i]) : 0.0f;
      }
    }
    float4v now;
    for (int j = 0; j < 4; ++j) now[j] = (t + j < start ? before[j] : 0.0f) + sum[j];
    if (t >= lo && t + 4 <= len) {
      *reinterpret_cast<float4v*>(at) = now;
    } else {
      for (int j = 0; j < 4; ++j)
        if (t + j >= lo && t + j < len) at[j] = now[j];
    }
  }
}

}  // namespace

hipError_t launch_weigh_scores(const CacheView& c, const SeqView& s, const AttendArgs& a, float* weights, hipStream_t st) {
  const uint64_t base = (uint64_t)s.seqs * c.heads, most = (a.scores_stride + kWeighEach - 1) / kWeighEach;
  const uint64_t want = (2048 + base - 1) / base, splits = want < most ? want : most;
  const uint64_t groups = base * splits;
  constexpr uint64_t kWide = 1u << 20;
  const dim3 grid((uint32_t)(groups < kWide ? groups : kWide), (uint32_t)((groups + kWide - 1) / kWide));
  k_weigh_scores<<<grid, kWeighLanes, 0, st>>>(c, s, a, weights, (uint32_t)splits);
  return hipGetLastError();
}

}  // namespace ltc
