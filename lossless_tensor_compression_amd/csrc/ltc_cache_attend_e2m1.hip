// ltc_cache_attend_e2m1.hip -- attention over E2M1 codes.
#include "ltc_cache_attend.h"

namespace ltc {

template hipError_t launch_attend<LTC_E2M1>(const CacheView&, const SeqView&, bool, const AttendArgs&, hipStream_t);

}  // namespace ltc
