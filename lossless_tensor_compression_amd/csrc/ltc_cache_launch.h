// ltc_cache_launch.h -- host-side launchers of the cache's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ltc_cache.h"

namespace ltc {

// 16-bit rows of the call: element [row][head][i] at base[row * row_stride + head * head_stride + i]
struct RowsView {
  const uint16_t* base;
  uint64_t row_stride, head_stride;
};

hipError_t launch_cache_write(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const RowsView& k,
                              const RowsView& v, hipStream_t st);

hipError_t launch_cache_read(const CacheView& c, const SeqView& s, bool e4m3, int dtype, uint16_t* k, uint16_t* v,
                             hipStream_t st);

struct AttendArgs {
  RowsView q;
  uint16_t* out;  // [rows][q_heads][dim]
  uint32_t q_heads;
  uint32_t window;  // 0: all positions up to the row's own
  float scale;      // of the products before the softmax
  void* ws;
};

uint64_t cache_attend_workspace(const CacheView& c, const SeqView& s, uint32_t q_heads, uint32_t window);

hipError_t launch_cache_attend(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const AttendArgs& a,
                               hipStream_t st);

}  // namespace ltc
