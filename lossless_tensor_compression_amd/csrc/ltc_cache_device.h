// ltc_cache_device.h -- device helpers shared by the cache's kernels.
#pragma once

#include "ltc_cache_launch.h"
#include "ltc_internal.h"

namespace ltc {

template <int DT> __device__ __forceinline__ float widen(uint32_t bits16) {
  if constexpr (DT == LTC_BF16) return __builtin_bit_cast(float, bits16 << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

template <int DT> __device__ __forceinline__ uint16_t narrow(float x) {
  if constexpr (DT == LTC_BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  else return __builtin_bit_cast(uint16_t, (_Float16)x);
}

template <bool E4M3> __device__ __forceinline__ float code_value(uint32_t c) {
  if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
  else return (float)(int8_t)c;
}

// Codes of numbers already divided by their scale: rounded to the nearest
// code, ties to even; what is past the top (only an infinity can be)
// saturates.  A NaN keeps its place in E4M3, which has one; INT8 has none and
// stores 0.
template <bool E4M3> __device__ __forceinline__ uint32_t to_code(float x) {
  if constexpr (E4M3) {
    x = x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff;
  } else {
    x = x != x ? 0.0f : fminf(fmaxf(x, -127.0f), 127.0f);
    return (uint32_t)(int)rintf(x) & 0xff;
  }
}

// At how many of the 64 places that find_sequence names units begin at or
// before `unit`, asked by the wave's lanes at once.
struct WaveCount {
  const SeqView& s;
  const UnitMap& m;
  uint64_t unit;
  __device__ __forceinline__ uint32_t operator()(uint32_t lo, uint32_t step, uint32_t n) const {
    const uint32_t o = (threadIdx.x & 63) * step;
    return (uint32_t)__popcll(__ballot(o < n && unit_first(m, s, lo + o) <= unit));
  }
};

__device__ __forceinline__ void report(const CacheView& c, uint32_t bit) { atomicOr(c.status, bit); }

}  // namespace ltc
