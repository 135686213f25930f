// ltc_cache_device.h -- device helpers shared by the cache's kernels.
#pragma once

#include <type_traits>

#include "ltc_cache_launch.h"
#include "ltc_internal.h"

namespace ltc {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <int DT> __device__ __forceinline__ float widen(uint32_t bits16) {
  if constexpr (DT == LTC_BF16) return __builtin_bit_cast(float, bits16 << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

// two numbers rounded to 16 bits, a in the low half
template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  const float2v x = {a, b};
  if constexpr (DT == LTC_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf2v));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, half2v));
}

// Four codes as numbers, the lowest byte first.
template <bool E4M3> __device__ __forceinline__ float4v code_values(uint32_t c) {
  if constexpr (E4M3) {
    const float2v lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    return float4v{lo[0], lo[1], hi[0], hi[1]};
  } else {
    return float4v{(float)(int8_t)c, (float)(int8_t)(c >> 8), (float)(int8_t)(c >> 16), (float)(int8_t)(c >> 24)};
  }
}

// Codes of four numbers already divided by their scale, none past the codes'
// top: rounded to the nearest code, ties to even.
template <bool E4M3> __device__ __forceinline__ uint32_t to_codes(float4v x) {
  if constexpr (E4M3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  } else {
    // 1.5 * 2^23 + x rounds x to a whole number, whose low byte is the sum's
    uint32_t u[4];
    for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(uint32_t, x[i] + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u);
    return lo | hi << 16;
  }
}

// For numbers that may be infinities, which saturate, and NaN, which keeps its
// place in E4M3 and is 0 in INT8.
template <bool E4M3> __device__ __forceinline__ float4v tame(float4v x) {
  constexpr float top = E4M3 ? 448.0f : 127.0f;
  for (int i = 0; i < 4; ++i) x[i] = x[i] != x[i] ? (E4M3 ? x[i] : 0.0f) : fminf(fmaxf(x[i], -top), top);
  return x;
}

// Of the bytes at positions t..t+3, those in [lo, hi) as 0xff.
__device__ __forceinline__ uint32_t byte_mask(int t, int lo, int hi) {
  const int a = min(max(lo - t, 0), 4), b = min(max(hi - t, 0), 4);
  const uint32_t below_b = (uint32_t)((1ull << (8 * b)) - 1), below_a = (uint32_t)((1ull << (8 * a)) - 1);
  return below_b & ~below_a;
}

// The 4x4 transposition of x[i] over the wave's four rows of 16 lanes: lane
// 16 g + n gets x[g] of lanes n, 16 + n, 32 + n, 48 + n.
__device__ __forceinline__ void transpose_rows(uint32_t (&x)[4]) {
  for (int i = 0; i < 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(x[i], x[i + 2], false, false);
    x[i] = r[0];
    x[i + 2] = r[1];
  }
  for (int i = 0; i < 4; i += 2) {
    const auto r = __builtin_amdgcn_permlane16_swap(x[i], x[i + 1], false, false);
    x[i] = r[0];
    x[i + 1] = r[1];
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

// Zeros for the rows of no sequence: `numbers` (a multiple of 8) at out +
// row * stride, by worker's workgroup of `workers`.
__device__ __forceinline__ void clear_unnamed(const Unnamed& u, uint16_t* out, uint64_t stride, uint32_t numbers,
                                              uint64_t worker, uint64_t workers) {
  const uint32_t parts = numbers / 8;
  for (uint64_t i = worker * blockDim.x + threadIdx.x; i < (uint64_t)u.n * parts; i += workers * blockDim.x)
    *reinterpret_cast<uint4v*>(out + unnamed_row(u, (uint32_t)(i / parts)) * stride + i % parts * 8) = uint4v{0, 0, 0, 0};
}

// A wave's share of keys: token lane & 15, dims of part 4 j + lane / 16.
// A wave's share of values: tokens 4 (lane / 16) + i, dims 64 j + 4 (lane & 15) + 0..3.
template <int D> struct Share {
  static constexpr int J = (D + 63) / 64;
  // of the last 64 dims, D = 96 has only the first 32
  static __device__ __forceinline__ bool k_has(int j, int lane) { return D % 64 == 0 || j < J - 1 || lane < 32; }
  static __device__ __forceinline__ bool v_has(int j, int lane) { return D % 64 == 0 || j < J - 1 || (lane & 15) < 8; }
};

typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

// largest magnitudes (as bits) of the pairs' halves
__device__ __forceinline__ ushort2v max_bits(ushort2v top, uint32_t pair) {
  return __builtin_elementwise_max(top, __builtin_bit_cast(ushort2v, pair & 0x7fff7fffu));
}

// the same without infinities and NaN
template <uint32_t kInf> __device__ __forceinline__ uint32_t max_finite_bits(uint32_t top, uint32_t pair) {
  uint32_t mask = 0x7fffu;
  asm("" : "+v"(mask));  // no common subexpressions with max_bits: they would be kept in registers for this rare case
  const uint32_t lo = pair & mask, hi = pair >> 16 & mask;
  return max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
}

template <int DT> __device__ __forceinline__ float4v widen4(uint2v x) {
  return float4v{widen<DT>(x[0] & 0xffffu), widen<DT>(x[0] >> 16), widen<DT>(x[1] & 0xffffu), widen<DT>(x[1] >> 16)};
}

template <int BYTES> __device__ __forceinline__ uint32_t load_drops(const uint8_t* at) {
  if constexpr (BYTES == 4) return *reinterpret_cast<const uint32_t*>(at);
  else if constexpr (BYTES == 2) return *reinterpret_cast<const uint16_t*>(at);
  else return *at;
}

template <int BYTES> __device__ __forceinline__ void store_drops(uint8_t* at, uint32_t drops) {
  if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(at) = drops;
  else if constexpr (BYTES == 2) *reinterpret_cast<uint16_t*>(at) = (uint16_t)drops;
  else *at = (uint8_t)drops;
}

__device__ __forceinline__ void report(const CacheView& c, uint32_t bit) { atomicOr(c.status, bit); }

// ---- on the host

inline UnitMap page_units(const CacheView& c, const SeqView& s) {
  if (!s.cu) return UnitMap{0, 1, 1};  // one row, one page
  return UnitMap{1, 1u << c.page_log, 2};
}

// f with the numbers' and the head's types as constants
template <class F> hipError_t for_numbers(int dtype, uint32_t dim, F f) {
  auto with_dim = [&](auto type) {
    switch (dim) {
      case 64: return f(type, std::integral_constant<int, 64>()), hipGetLastError();
      case 96: return f(type, std::integral_constant<int, 96>()), hipGetLastError();
      case 128: return f(type, std::integral_constant<int, 128>()), hipGetLastError();
      case 192: return f(type, std::integral_constant<int, 192>()), hipGetLastError();
      case 256: return f(type, std::integral_constant<int, 256>()), hipGetLastError();
    }
    return hipErrorInvalidValue;
  };
  return dtype == LTC_BF16 ? with_dim(std::integral_constant<int, LTC_BF16>())
                           : with_dim(std::integral_constant<int, LTC_FP16>());
}

}  // namespace ltc
