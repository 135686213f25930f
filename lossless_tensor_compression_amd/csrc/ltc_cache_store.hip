// ltc_cache_store.hip -- writing keys and values into the 8-bit cache and
// reading them back.
#include "ltc_cache_device.h"

namespace ltc {
namespace {

// One workgroup for a touched page and head.  Its new rows set the scale; a
// page that already holds tokens of the sequence keeps the larger of its
// scale and theirs, and if that grew, its tokens are coded again.
template <bool E4M3, int DT>
__global__ __launch_bounds__(256) void k_cache_write(CacheView c, SeqView s, UnitMap map, RowsView k, RowsView v) {
  __shared__ uint32_t largest_bits;
  uint32_t seq;
  Span sp;
  uint64_t j;
  const bool mine = locate_unit(c, s, map, blockIdx.x, WaveCount{s, map, blockIdx.x}, &seq, &sp, &j);
  if (!sp.ok && threadIdx.x == 0) report(c, kCacheBadSeq);
  if (!mine || !sp.ok) return;
  j += sp.start >> c.page_log;
  if (j > ((sp.len - 1) >> c.page_log)) return;
  uint32_t page;
  if (!page_at(s, seq, (uint32_t)j, c.pages, &page)) {
    if (threadIdx.x == 0) report(c, kCacheBadPage);
    return;
  }
  const uint32_t P = 1u << c.page_log, head = blockIdx.y;
  const uint32_t first = (uint32_t)j << c.page_log;  // position of the page's token 0
  const uint32_t t0 = sp.start > first ? sp.start - first : 0;
  const uint32_t t1 = sp.len - first < P ? sp.len - first : P;
  for (int kind = 0; kind < 2; ++kind) {
    const RowsView& x = kind ? v : k;
    uint8_t* codes = (kind ? c.v : c.k) + head_offset(c, page, head);
    uint8_t* scale = c.scales + ((uint64_t)page * c.heads + head) * 2 + kind;
    const uint32_t before = *scale;
    if (threadIdx.x == 0) largest_bits = 0;
    __syncthreads();
    const uint32_t cells = (t1 - t0) * c.dim;
    auto value = [&](uint32_t i) {
      const uint32_t t = t0 + i / c.dim, d = i % c.dim;
      const uint64_t row = sp.row0 + (first + t - sp.start);
      return widen<DT>(x.base[row * x.row_stride + head * x.head_stride + d]);
    };
    float largest = 0.0f;
    for (uint32_t i = threadIdx.x; i < cells; i += 256) {
      const float a = fabsf(value(i));
      if (a < INFINITY) largest = fmaxf(largest, a);
    }
    atomicMax(&largest_bits, __builtin_bit_cast(uint32_t, largest));
    __syncthreads();
    uint32_t after = scale_byte(__builtin_bit_cast(float, largest_bits), E4M3);
    if (t0 > 0 && before > after) after = before;
    if (t0 > 0 && after > before) {
      const int drop = (int)before - (int)after;
      const float shrink = power_of_two(drop < -126 ? -126 : drop);
      for (uint32_t i = threadIdx.x; i < t0 * c.dim; i += 256) {
        const uint32_t t = i / c.dim, d = i % c.dim;
        uint8_t* at = codes + (kind ? v_code(t, d, c.dim) : k_code(t, d, c.dim));
        *at = (uint8_t)to_code<E4M3>(code_value<E4M3>(*at) * shrink);
      }
    }
    const float unscale = power_of_two(127 - (int)after);
    for (uint32_t i = threadIdx.x; i < cells; i += 256) {
      const uint32_t t = t0 + i / c.dim, d = i % c.dim;
      codes[kind ? v_code(t, d, c.dim) : k_code(t, d, c.dim)] = (uint8_t)to_code<E4M3>(value(i) * unscale);
    }
    __syncthreads();
    if (threadIdx.x == 0) *scale = (uint8_t)after;
  }
}

// One workgroup for a touched page and head: its tokens that the call asks
// for, code times scale, rounded once.
template <bool E4M3, int DT>
__global__ __launch_bounds__(256) void k_cache_read(CacheView c, SeqView s, UnitMap map, uint16_t* k, uint16_t* v) {
  uint32_t seq;
  Span sp;
  uint64_t j;
  const bool mine = locate_unit(c, s, map, blockIdx.x, WaveCount{s, map, blockIdx.x}, &seq, &sp, &j);
  if (!sp.ok && threadIdx.x == 0) report(c, kCacheBadSeq);
  if (!mine) return;
  j += sp.start >> c.page_log;
  const uint32_t P = 1u << c.page_log, head = blockIdx.y;
  // a refused sequence has start 0 here: its rows get zeros
  const uint32_t last = sp.start + sp.n - 1;
  if (j > (last >> c.page_log)) return;
  uint32_t page = 0;
  const bool have = sp.ok && page_at(s, seq, (uint32_t)j, c.pages, &page);
  if (sp.ok && !have && threadIdx.x == 0) report(c, kCacheBadPage);
  const uint32_t first = (uint32_t)j << c.page_log;
  const uint32_t t0 = sp.start > first ? sp.start - first : 0;
  const uint32_t t1 = last - first < P ? last - first + 1 : P;
  for (int kind = 0; kind < 2; ++kind) {
    const uint8_t* codes = (kind ? c.v : c.k) + head_offset(c, page, head);
    const float scale = have ? power_of_two((int)c.scales[((uint64_t)page * c.heads + head) * 2 + kind] - 127) : 0.0f;
    for (uint32_t i = threadIdx.x; i < (t1 - t0) * c.dim; i += 256) {
      const uint32_t t = t0 + i / c.dim, d = i % c.dim;
      const uint64_t row = sp.row0 + (first + t - sp.start);
      const float x = have ? code_value<E4M3>(codes[kind ? v_code(t, d, c.dim) : k_code(t, d, c.dim)]) * scale : 0.0f;
      (kind ? v : k)[(row * c.heads + head) * c.dim + d] = narrow<DT>(x);
    }
  }
}

UnitMap page_units(const CacheView& c, const SeqView& s) {
  if (!s.cu) return UnitMap{0, 1, 1};  // one row, one page
  return UnitMap{1, 1u << c.page_log, 2};
}

}  // namespace

hipError_t launch_cache_write(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const RowsView& k,
                              const RowsView& v, hipStream_t st) {
  const UnitMap m = page_units(c, s);
  const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
  if (e4m3) {
    if (dtype == LTC_BF16) k_cache_write<true, LTC_BF16><<<grid, 256, 0, st>>>(c, s, m, k, v);
    else k_cache_write<true, LTC_FP16><<<grid, 256, 0, st>>>(c, s, m, k, v);
  } else {
    if (dtype == LTC_BF16) k_cache_write<false, LTC_BF16><<<grid, 256, 0, st>>>(c, s, m, k, v);
    else k_cache_write<false, LTC_FP16><<<grid, 256, 0, st>>>(c, s, m, k, v);
  }
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheView& c, const SeqView& s, bool e4m3, int dtype, uint16_t* k, uint16_t* v,
                             hipStream_t st) {
  const UnitMap m = page_units(c, s);
  const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
  if (e4m3) {
    if (dtype == LTC_BF16) k_cache_read<true, LTC_BF16><<<grid, 256, 0, st>>>(c, s, m, k, v);
    else k_cache_read<true, LTC_FP16><<<grid, 256, 0, st>>>(c, s, m, k, v);
  } else {
    if (dtype == LTC_BF16) k_cache_read<false, LTC_BF16><<<grid, 256, 0, st>>>(c, s, m, k, v);
    else k_cache_read<false, LTC_FP16><<<grid, 256, 0, st>>>(c, s, m, k, v);
  }
  return hipGetLastError();
}

}  // namespace ltc
