// ltc_cache_weigh_int8.hip -- positions' weights over INT8 codes.
#include "ltc_cache_weigh.h"

namespace ltc {

template hipError_t launch_weigh<LTC_INT8>(const CacheView&, const SeqView&, int, const AttendArgs&, float*, hipStream_t);

}  // namespace ltc
