// ltc_cache_weigh_e4m3.hip -- positions' weights over E4M3 codes.
#include "ltc_cache_weigh.h"

namespace ltc {

template hipError_t launch_weigh<LTC_E4M3>(const CacheView&, const SeqView&, int, const AttendArgs&, float*, hipStream_t);

}  // namespace ltc
