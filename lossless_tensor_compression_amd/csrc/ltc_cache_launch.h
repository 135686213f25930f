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

// codes of 8 bits, and of 4
hipError_t launch_cache_write(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const RowsView& k,
                              const RowsView& v, hipStream_t st);

hipError_t launch_cache_read(const CacheView& c, const SeqView& s, bool e4m3, int dtype, uint16_t* k, uint16_t* v,
                             hipStream_t st);

hipError_t launch_cache4_write(const CacheView& c, const SeqView& s, int dtype, const RowsView& k, const RowsView& v,
                               hipStream_t st);

hipError_t launch_cache4_read(const CacheView& c, const SeqView& s, int dtype, uint16_t* k, uint16_t* v, hipStream_t st);

struct AttendArgs {
  RowsView q;
  uint16_t* out;  // [rows][q_heads][dim]
  uint32_t q_heads;
  uint32_t window;  // 0: all positions up to the row's own
  float scale;      // of the products before the softmax
  void* ws;
  float* lse;  // [rows][q_heads] log2 of the softmax's sum, or null
  float* scores;  // [rows][q_heads][scores_stride] in units of log2, by position from score_first on, or null
  uint64_t scores_stride;
};

uint64_t cache_attend_workspace(const CacheView& c, const SeqView& s, int codes, int dtype, uint32_t q_heads, uint32_t window);

// 0: an attention that weighs does without scores
uint64_t cache_scores_stride(const CacheView& c, const SeqView& s, int codes, uint32_t q_heads, uint32_t window);

hipError_t launch_cache_attend(const CacheView& c, const SeqView& s, int codes, int dtype, const AttendArgs& a,
                               hipStream_t st);

// add to weights [pages][heads][page] what the rows give the positions they see;
// a.lse is known, and for the second a.scores
template <int CODES>
hipError_t launch_weigh(const CacheView& c, const SeqView& s, int dtype, const AttendArgs& a, float* weights, hipStream_t st);

hipError_t launch_weigh_scores(const CacheView& c, const SeqView& s, const AttendArgs& a, float* weights, hipStream_t st);

struct EvictArgs {
  float* weights;  // [pages][heads][page]
  const int32_t* to;
  uint64_t to_stride;
  uint32_t keep, recent;
  int32_t *lengths, *positions;
  uint32_t* ws;
};

uint64_t cache_evict_workspace(const CacheView& c, const SeqView& s);

hipError_t launch_cache_evict(const CacheView& c, const SeqView& s, int codes, const EvictArgs& a, hipStream_t st);

// of one code type; each is built in a file of its own
template <int CODES>
hipError_t launch_attend(const CacheView& c, const SeqView& s, bool bf16, const AttendArgs& a, hipStream_t st);

}  // namespace ltc
