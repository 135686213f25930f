// ltc_cache_attend_int8.hip -- attention over INT8 codes.
#include "ltc_cache_attend.h"

namespace ltc {

template hipError_t launch_attend<LTC_INT8>(const CacheView&, const SeqView&, bool, const AttendArgs&, hipStream_t);

}  // namespace ltc
