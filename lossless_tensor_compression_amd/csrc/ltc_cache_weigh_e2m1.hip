// ltc_cache_weigh_e2m1.hip -- positions' weights over E2M1 codes.
#include "ltc_cache_weigh.h"

namespace ltc {

template hipError_t launch_weigh<LTC_E2M1>(const CacheView&, const SeqView&, int, const AttendArgs&, float*, hipStream_t);

}  // namespace ltc
