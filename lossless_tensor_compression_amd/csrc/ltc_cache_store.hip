// ltc_cache_store.hip -- writing keys and values into the 8-bit cache and
// reading them back.
#include "ltc_cache_device.h"

namespace ltc {
namespace {

// What bounds both: the bytes (6 a number pair) at memory's rate, and for a
// few tokens the chain of loads span -> table -> scale.  A workgroup takes a
// page and head, a wave 16 of its tokens, keys and values both, so that 16
// tokens' values leave and arrive as the 16 bytes of a dim.  With narrow
// accesses instead: write of 18,000 tokens 134 us, read of 65,537 tokens 209 us,
// 8 heads of 128.  So 28 us, 4.4 TB/s, and 84 us, 4.8
// TB/s, where a 2 GiB copy runs at 4.9; a token of each of 48 sequences 6 us.

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

// The page's new rows set the scale; a page that already holds tokens of the
// sequence keeps the larger of its scale and theirs, and if that grew, its
// tokens are coded again.
template <bool E4M3, int DT, int D>
__global__ __launch_bounds__(1024) void k_cache_write(CacheView c, SeqView s, UnitMap map, RowsView k, RowsView v) {
  using S = Share<D>;
  constexpr int J = S::J;
  constexpr uint32_t kInf = DT == LTC_BF16 ? 0x7f80 : 0x7c00;
  __shared__ uint32_t tops[2][16];
  __shared__ uint32_t befores[2];
  uint32_t seq;
  Span sp;
  uint64_t j64;
  const Early early = load_early(s, blockIdx.x);
  const bool mine = locate_unit(c, s, map, blockIdx.x, WaveCount{s, map, blockIdx.x}, &seq, &sp, &j64);
  if (!(sp.ok && check_sequence(c, s, early)) && threadIdx.x == 0) report(c, kCacheBadSeq);
  if (!mine || !sp.ok) return;
  j64 += sp.start >> c.page_log;
  if (j64 > ((sp.len - 1) >> c.page_log)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const uint32_t head = blockIdx.y, P = 1u << c.page_log, first = (uint32_t)j64 << c.page_log;
  const int t0 = sp.start > first ? (int)(sp.start - first) : 0;               // tokens [t0, t1) are new
  const int t1 = (int)(sp.len - first < P ? sp.len - first : P);
  const int kt = wave * 16 + (lane & 15), vt = wave * 16 + (lane >> 4) * 4;  // of the page
  // the rows' loads need no page: they go first
  const uint64_t row = (uint64_t)sp.row0 + first - sp.start;  // row of token 0, if it were new
  uint4v kr[J][2];
  uint2v vr[J][4];
  ushort2v most_k = {0, 0}, most_v = {0, 0};
  for (int j = 0; j < J; ++j) {
    const bool want = kt >= t0 && kt < t1 && S::k_has(j, lane);
    const uint4v* p = reinterpret_cast<const uint4v*>(k.base + (row + kt) * k.row_stride + head * k.head_stride +
                                                      j * 64 + (lane >> 4) * 16);
    for (int i = 0; i < 2; ++i) kr[j][i] = want ? p[i] : uint4v{0, 0, 0, 0};
  }
  for (int j = 0; j < J; ++j)
    for (int i = 0; i < 4; ++i) {
      const bool want = vt + i >= t0 && vt + i < t1 && S::v_has(j, lane);
      vr[j][i] = want ? *reinterpret_cast<const uint2v*>(v.base + (row + vt + i) * v.row_stride + head * v.head_stride +
                                                         j * 64 + (lane & 15) * 4)
                      : uint2v{0, 0};
    }
  uint32_t page;
  if (!page_at(s, seq, (uint32_t)j64, c.pages, &page)) {
    if (threadIdx.x == 0) report(c, kCacheBadPage);
    return;
  }
  uint8_t* scales = c.scales + ((uint64_t)page * c.heads + head) * 2;
  if (threadIdx.x == 0) {
    befores[0] = scales[0];
    befores[1] = scales[1];
  }
  for (int j = 0; j < J; ++j) {
    for (int i = 0; i < 2; ++i)
      for (int w = 0; w < 4; ++w) most_k = max_bits(most_k, kr[j][i][w]);
    for (int i = 0; i < 4; ++i)
      for (int w = 0; w < 2; ++w) most_v = max_bits(most_v, vr[j][i][w]);
  }
  uint32_t top_k = max(most_k[0], most_k[1]), top_v = max(most_v[0], most_v[1]);
  // infinities and NaN do not count: without them once more
  const bool special_k = __any(top_k >= kInf), special_v = __any(top_v >= kInf);
  if (special_k) {
    top_k = 0;
    for (int j = 0; j < J; ++j)
      for (int i = 0; i < 8; ++i) top_k = max_finite_bits<kInf>(top_k, kr[j][i >> 2][i & 3]);
  }
  if (special_v) {
    top_v = 0;
    for (int j = 0; j < J; ++j)
      for (int i = 0; i < 8; ++i) top_v = max_finite_bits<kInf>(top_v, vr[j][i >> 1][i & 1]);
  }
  for (int w = 32; w; w >>= 1) {
    top_k = max(top_k, (uint32_t)__shfl_xor((int)top_k, w));
    top_v = max(top_v, (uint32_t)__shfl_xor((int)top_v, w));
  }
  if (lane == 0) {
    tops[0][wave] = top_k;
    tops[1][wave] = top_v;
  }
  __syncthreads();
  for (int w = 0; w < waves; ++w) {
    top_k = max(top_k, tops[0][w]);
    top_v = max(top_v, tops[1][w]);
  }
  int after[2] = {(int)scale_byte(widen<DT>(top_k), E4M3), (int)scale_byte(widen<DT>(top_v), E4M3)};
  float shrink[2];
  bool grown[2];
  for (int i = 0; i < 2; ++i) {
    const int before = (int)befores[i];
    if (t0 > 0) after[i] = max(after[i], before);
    grown[i] = t0 > 0 && after[i] > before;
    shrink[i] = power_of_two(max(before - after[i], -126));
  }
  if (threadIdx.x == 0) {
    scales[0] = (uint8_t)after[0];
    scales[1] = (uint8_t)after[1];
  }
  const uint64_t base = head_offset(c, page, head) + (uint32_t)wave * (16 * D);
  {
    // keys: a lane's token is new, or old and coded again, or left
    const float un = power_of_two(127 - after[0]);
    for (int j = 0; j < J; ++j) {
      uint4v* at = reinterpret_cast<uint4v*>(c.k + base + j * 1024 + (lane >> 4) * 256 + (lane & 15) * 16);
      __builtin_amdgcn_sched_barrier(0);  // one part at a time: registers
      if (!S::k_has(j, lane)) continue;
      if (kt >= t0 && kt < t1) {
        uint4v o;
        for (int i = 0; i < 4; ++i) {
          float4v x = widen4<DT>(uint2v{kr[j][i >> 1][(i & 1) * 2], kr[j][i >> 1][(i & 1) * 2 + 1]}) * un;
          if (special_k) x = tame<E4M3>(x);
          o[i] = to_codes<E4M3>(x);
        }
        *at = o;
      } else if (grown[0] && kt < t0) {
        uint4v o = *at;
        for (int i = 0; i < 4; ++i) o[i] = to_codes<E4M3>(code_values<E4M3>(o[i]) * shrink[0]);
        *at = o;
      }
    }
  }
  // values: a lane's dim is 16 tokens, of which old ones may be among new
  const int b0 = wave * 16;
  if (b0 >= t1 || (b0 + 16 <= t0 && !grown[1])) return;
  const float un = power_of_two(127 - after[1]);
  for (int j = 0; j < J; ++j) {
    __builtin_amdgcn_sched_barrier(0);
    uint32_t x[4];  // dim i, this lane's four tokens
    for (int i = 0; i < 4; ++i) {
      float4v y;
      for (int t = 0; t < 4; ++t) y[t] = widen<DT>(vr[j][t][i >> 1] >> (16 * (i & 1)) & 0xffffu) * un;
      if (special_v) y = tame<E4M3>(y);
      x[i] = to_codes<E4M3>(y);
    }
    transpose_rows(x);  // dim 4 (lane & 15) + lane / 16, tokens 4 i + 0..3
    if (!S::v_has(j, lane)) continue;
    uint4v* at = reinterpret_cast<uint4v*>(c.v + base + (j * 64 + (lane & 15) * 4 + (lane >> 4)) * 16);
    uint4v o = {x[0], x[1], x[2], x[3]};
    if (b0 < t0 || b0 + 16 > t1) {
      const uint4v old = *at;
      for (int i = 0; i < 4; ++i) {
        const uint32_t fresh = byte_mask(b0 + 4 * i, t0, t1), begun = byte_mask(b0 + 4 * i, 0, t0);
        uint32_t kept = old[i];
        if (grown[1]) kept = (to_codes<E4M3>(code_values<E4M3>(kept) * shrink[1]) & begun) | (kept & ~begun);
        o[i] = (o[i] & fresh) | (kept & ~fresh);
      }
    }
    *at = o;
  }
}

// Code times scale, exact in 32 bits, rounded once.
template <bool E4M3, int DT, int D>
__global__ __launch_bounds__(1024) void k_cache_read(CacheView c, SeqView s, UnitMap map, uint16_t* k, uint16_t* v) {
  using S = Share<D>;
  constexpr int J = S::J;
  uint32_t seq;
  Span sp;
  uint64_t j64;
  const Early early = load_early(s, blockIdx.x);
  const bool mine = locate_unit(c, s, map, blockIdx.x, WaveCount{s, map, blockIdx.x}, &seq, &sp, &j64);
  const Unnamed none = unnamed_rows(s, early);
  if (none.n)
    for (uint16_t* out : {k, v})
      clear_unnamed(none, out + blockIdx.y * D, (uint64_t)c.heads * D, D, blockIdx.x, gridDim.x);
  if (!(sp.ok && check_sequence(c, s, early)) && threadIdx.x == 0) report(c, kCacheBadSeq);
  if (!mine) return;
  j64 += sp.start >> c.page_log;
  // a refused sequence has start 0 here: its rows get zeros
  const uint32_t last = sp.start + sp.n - 1;
  if (j64 > (last >> c.page_log)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t head = blockIdx.y, P = 1u << c.page_log, first = (uint32_t)j64 << c.page_log;
  const int t0 = sp.start > first ? (int)(sp.start - first) : 0;
  const int t1 = (int)(last - first < P ? last - first + 1 : P);
  if (wave * 16 >= t1 || wave * 16 + 16 <= t0) return;
  uint32_t page = 0;
  const bool have = sp.ok && page_at(s, seq, (uint32_t)j64, c.pages, &page);
  if (sp.ok && !have && lane == 0) report(c, kCacheBadPage);
  uint2v kr[J][2];
  uint4v vr[J];
  float ks = 0.0f, vs = 0.0f;
  for (int j = 0; j < J; ++j) {
    kr[j][0] = kr[j][1] = uint2v{0, 0};
    vr[j] = uint4v{0, 0, 0, 0};
  }
  // keys here: token 8 i + lane / 8, 8 dims, so that a row's 64 dims leave as one line
  const int kd = (lane & 7) * 8, ktok = lane >> 3;
  if (have) {
    const uint64_t base = head_offset(c, page, head) + (uint32_t)wave * (16 * D);
    const uint8_t* scales = c.scales + ((uint64_t)page * c.heads + head) * 2;
    for (int j = 0; j < J; ++j) {
      if (j * 64 + kd < D)
        for (int i = 0; i < 2; ++i)
          kr[j][i] = *reinterpret_cast<const uint2v*>(c.k + base + j * 1024 + (kd >> 4) * 256 + (i * 8 + ktok) * 16 + (kd & 8));
      if (S::v_has(j, lane))
        vr[j] = *reinterpret_cast<const uint4v*>(c.v + base + (j * 64 + (lane & 15) * 4 + (lane >> 4)) * 16);
    }
    ks = power_of_two((int)scales[0] - 127);
    vs = power_of_two((int)scales[1] - 127);
  }
  const uint64_t row = (uint64_t)sp.row0 + first - sp.start;  // row of token 0 of the page, if asked for
  const uint64_t stride = (uint64_t)c.heads * D;
  for (int j = 0; j < J; ++j)
    for (int i = 0; i < 2; ++i) {
      const int t = wave * 16 + i * 8 + ktok;
      const float4v a = code_values<E4M3>(kr[j][i][0]) * ks, b = code_values<E4M3>(kr[j][i][1]) * ks;
      const uint4v o = {pack2<DT>(a[0], a[1]), pack2<DT>(a[2], a[3]), pack2<DT>(b[0], b[1]), pack2<DT>(b[2], b[3])};
      if (t >= t0 && t < t1 && j * 64 + kd < D)
        *reinterpret_cast<uint4v*>(k + (row + t) * stride + head * D + j * 64 + kd) = o;
    }
  for (int j = 0; j < J; ++j) {
    uint32_t x[4] = {vr[j][0], vr[j][1], vr[j][2], vr[j][3]};  // tokens 4 i + 0..3 of one dim
    transpose_rows(x);                                          // dim 4 (lane & 15) + i, tokens 4 (lane / 16) + 0..3
    float4v y[4];
    for (int i = 0; i < 4; ++i) y[i] = code_values<E4M3>(x[i]) * vs;
    for (int i = 0; i < 4; ++i) {
      const int t = wave * 16 + (lane >> 4) * 4 + i;
      const uint2v o = {pack2<DT>(y[0][i], y[1][i]), pack2<DT>(y[2][i], y[3][i])};
      if (t >= t0 && t < t1 && S::v_has(j, lane))
        *reinterpret_cast<uint2v*>(v + (row + t) * stride + head * D + j * 64 + (lane & 15) * 4) = o;
    }
  }
}

UnitMap page_units(const CacheView& c, const SeqView& s) {
  if (!s.cu) return UnitMap{0, 1, 1};  // one row, one page
  return UnitMap{1, 1u << c.page_log, 2};
}

template <bool E4M3, int DT, int D>
void launch_write(const CacheView& c, const SeqView& s, const RowsView& k, const RowsView& v, hipStream_t st) {
  const UnitMap m = page_units(c, s);
  const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
  k_cache_write<E4M3, DT, D><<<grid, 4u << c.page_log, 0, st>>>(c, s, m, k, v);
}

template <bool E4M3, int DT, int D>
void launch_read(const CacheView& c, const SeqView& s, uint16_t* k, uint16_t* v, hipStream_t st) {
  const UnitMap m = page_units(c, s);
  const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
  k_cache_read<E4M3, DT, D><<<grid, 4u << c.page_log, 0, st>>>(c, s, m, k, v);
}

// f with the codes', the numbers' and the head's types as constants
template <class F> hipError_t for_types(bool e4m3, int dtype, uint32_t dim, F f) {
  auto with_dim = [&](auto codes, auto type) {
    switch (dim) {
      case 64: return f(codes, type, std::integral_constant<int, 64>()), hipGetLastError();
      case 96: return f(codes, type, std::integral_constant<int, 96>()), hipGetLastError();
      case 128: return f(codes, type, std::integral_constant<int, 128>()), hipGetLastError();
      case 192: return f(codes, type, std::integral_constant<int, 192>()), hipGetLastError();
      case 256: return f(codes, type, std::integral_constant<int, 256>()), hipGetLastError();
    }
    return hipErrorInvalidValue;
  };
  auto with_type = [&](auto codes) {
    return dtype == LTC_BF16 ? with_dim(codes, std::integral_constant<int, LTC_BF16>())
                             : with_dim(codes, std::integral_constant<int, LTC_FP16>());
  };
  return e4m3 ? with_type(std::true_type()) : with_type(std::false_type());
}

}  // namespace

hipError_t launch_cache_write(const CacheView& c, const SeqView& s, bool e4m3, int dtype, const RowsView& k,
                              const RowsView& v, hipStream_t st) {
  return for_types(e4m3, dtype, c.dim, [&](auto codes, auto type, auto dim) {
    launch_write<decltype(codes)::value, decltype(type)::value, decltype(dim)::value>(c, s, k, v, st);
  });
}

hipError_t launch_cache_read(const CacheView& c, const SeqView& s, bool e4m3, int dtype, uint16_t* k, uint16_t* v,
                             hipStream_t st) {
  return for_types(e4m3, dtype, c.dim, [&](auto codes, auto type, auto dim) {
    launch_read<decltype(codes)::value, decltype(type)::value, decltype(dim)::value>(c, s, k, v, st);
  });
}

}  // namespace ltc
