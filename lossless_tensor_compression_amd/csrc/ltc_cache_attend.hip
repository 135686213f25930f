// ltc_cache_attend.hip -- attention over E4M3 codes; which code type's a call takes.
#include "ltc_cache_attend.h"

namespace ltc {

// built in files of their own
extern template hipError_t launch_attend<LTC_INT8>(const CacheView&, const SeqView&, bool, const AttendArgs&, hipStream_t);
extern template hipError_t launch_attend<LTC_E2M1>(const CacheView&, const SeqView&, bool, const AttendArgs&, hipStream_t);
template hipError_t launch_attend<LTC_E4M3>(const CacheView&, const SeqView&, bool, const AttendArgs&, hipStream_t);

uint64_t cache_attend_workspace(const CacheView& c, const SeqView& s, int codes, int dtype, uint32_t q_heads, uint32_t window) {
  if (!s.rows) return 0;
  const Plan p = plan_rows(c, s, q_heads, window, codes == LTC_E2M1);
  if (p.tiles) return may_scale(codes, (int)c.dim, dtype == LTC_BF16) ? kCounterBytes + (uint64_t)p.units * c.heads : 0;  // marks
  return p.splits == 1 ? 0 : kCounterBytes + (uint64_t)p.units * c.heads * p.splits * 16 * p.nc * (c.dim + 2) * sizeof(float);
}

uint64_t cache_scores_stride(const CacheView& c, const SeqView& s, int codes, uint32_t q_heads, uint32_t window) {
  return s.rows ? scores_stride(plan_rows(c, s, q_heads, window, codes == LTC_E2M1), c, s, q_heads, window) : 0;
}

hipError_t launch_cache_attend(const CacheView& c, const SeqView& s, int codes, int dtype, const AttendArgs& a,
                               hipStream_t st) {
  const bool bf16 = dtype == LTC_BF16;
  switch (codes) {
    case LTC_E4M3: return launch_attend<LTC_E4M3>(c, s, bf16, a, st);
    case LTC_INT8: return launch_attend<LTC_INT8>(c, s, bf16, a, st);
    case LTC_E2M1: return launch_attend<LTC_E2M1>(c, s, bf16, a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace ltc
