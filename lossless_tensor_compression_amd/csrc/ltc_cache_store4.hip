// ltc_cache_store4.hip -- writing keys and values into a cache of 4-bit codes
// and reading them back.
//
// Every token has a scale of its own, 2^e with the least e >= -100 for which its
// largest number fits the codes (6), and 32 dims of a key one that is 2^drop
// below it, as many as they leave unused: so a write changes nothing but its
// own tokens, and one channel of keys that is always large costs its 32
// neighbours precision and no other.
#include "ltc_cache_device.h"

namespace ltc {
namespace {

// What bounds both: the bytes at memory's rate, and for a few tokens the chain of
// loads span -> table -> codes.  8 heads of 128: 18,617 tokens written 19.8 us, 4.9
// TB/s, where a 1 GiB copy runs at 5.1; a token of each of 48 sequences 5.8 us; 19
// spans of 20-901 tokens of 5 heads of 96 read 9 us.
// A workgroup takes a page and head, a wave 16 of its tokens, keys and values
// both.  Of keys a lane has 32 dims of a token, the 16 bytes that share a scale;
// of values 4 tokens' 4 dims, whose codes make 16 bits of each dim and change
// places with those of the wave's other lane rows (transpose_rows).

// Eight numbers already divided by their scale, none past the codes' top: rounded
// to the nearest code, ties to even, the first one in the lowest bits.
__device__ __forceinline__ uint32_t to_e2m1(float4v a, float4v b) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a[0], a[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], 1.0f, 3);
}
__device__ __forceinline__ uint32_t to_e2m1(float4v a) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a[0], a[1], 1.0f, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], 1.0f, 1) & 0xffffu;
}

// Infinities saturate, and a NaN is 0: E2M1 has neither.
__device__ __forceinline__ float4v tame4(float4v x) {
  for (int i = 0; i < 4; ++i) x[i] = x[i] != x[i] ? 0.0f : fminf(fmaxf(x[i], -6.0f), 6.0f);
  return x;
}

// The code's value times 2^e for codes 2 SEL and 2 SEL + 1 of c.
template <int SEL> __device__ __forceinline__ float2v two_values(uint32_t c, float scale) {
  return __builtin_bit_cast(float2v, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, SEL));
}

// Of the four bits each of tokens t..t+7, those of tokens in [lo, hi).
__device__ __forceinline__ uint32_t nibble_mask(int t, int lo, int hi) {
  const int a = min(max(lo - t, 0), 8), b = min(max(hi - t, 0), 8);
  const uint32_t below_b = (uint32_t)((1ull << (4 * b)) - 1), below_a = (uint32_t)((1ull << (4 * a)) - 1);
  return below_b & ~below_a;
}

template <int DT, int D>
__global__ __launch_bounds__(1024) void k_cache4_write(CacheView c, SeqView s, UnitMap map, RowsView k, RowsView v) {
  using S = Share<D>;
  constexpr int J = S::J, BLOCKS = D / 32, JB = (BLOCKS + 3) / 4, DROPS = (int)drop_bytes(D);
  constexpr uint32_t kInf = DT == LTC_BF16 ? 0x7f80 : 0x7c00;
  uint32_t seq;
  Span sp;
  uint64_t j64;
  const Early early = load_early(s, blockIdx.x);
  const bool mine = locate_unit(c, s, map, blockIdx.x, WaveCount{s, map, blockIdx.x}, &seq, &sp, &j64);
  if (!(sp.ok && check_sequence(c, s, early)) && threadIdx.x == 0) report(c, kCacheBadSeq);
  if (!mine || !sp.ok) return;
  j64 += sp.start >> c.page_log;
  if (j64 > ((sp.len - 1) >> c.page_log)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const uint32_t head = blockIdx.y, P = 1u << c.page_log, first = (uint32_t)j64 << c.page_log;
  const int t0 = sp.start > first ? (int)(sp.start - first) : 0;  // tokens [t0, t1) are new
  const int t1 = (int)(sp.len - first < P ? sp.len - first : P);
  const int b0 = wave * 16, kt = b0 + n, vt = b0 + g * 4;  // of the page
  if (b0 >= t1 || b0 + 16 <= t0) {
    uint32_t page;
    if (threadIdx.x == 0 && !page_at(s, seq, (uint32_t)j64, c.pages, &page)) report(c, kCacheBadPage);
    return;
  }
  // the rows' loads need no page: they go first
  const uint64_t row = (uint64_t)sp.row0 + first - sp.start;  // row of token 0, if it were new
  const bool fresh = kt >= t0 && kt < t1;
  uint4v kr[JB][4];
  uint2v vr[J][4];
  for (int j = 0; j < JB; ++j) {
    const uint4v* p = reinterpret_cast<const uint4v*>(k.base + (row + kt) * k.row_stride + head * k.head_stride + (4 * j + g) * 32);
    for (int i = 0; i < 4; ++i) kr[j][i] = fresh && 4 * j + g < BLOCKS ? p[i] : uint4v{0, 0, 0, 0};
  }
  for (int j = 0; j < J; ++j)
    for (int i = 0; i < 4; ++i) {
      const bool want = vt + i >= t0 && vt + i < t1 && S::v_has(j, lane);
      vr[j][i] = want ? *reinterpret_cast<const uint2v*>(v.base + (row + vt + i) * v.row_stride + head * v.head_stride +
                                                         j * 64 + n * 4)
                      : uint2v{0, 0};
    }
  uint32_t page;
  if (!page_at(s, seq, (uint32_t)j64, c.pages, &page)) {
    if (threadIdx.x == 0) report(c, kCacheBadPage);
    return;
  }
  uint8_t* scales = c.scales + token_scales(c, page, head);
  const uint64_t base = head_offset(c, page, head) / 2 + (uint32_t)wave * (8 * D);

  {  // ---- keys
    uint32_t top[JB], most = 0;
    bool special = false;
    for (int j = 0; j < JB; ++j) {
      ushort2v m = {0, 0};
      for (int i = 0; i < 16; ++i) m = max_bits(m, kr[j][i >> 2][i & 3]);
      top[j] = max(m[0], m[1]);
      if (top[j] >= kInf) {  // infinities and NaN do not count: without them once more
        special = true;
        top[j] = 0;
        for (int i = 0; i < 16; ++i) top[j] = max_finite_bits<kInf>(top[j], kr[j][i >> 2][i & 3]);
      }
      most = max(most, top[j]);
    }
    most = max(most, (uint32_t)__shfl_xor((int)most, 16));
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    const int e = max(e2m1_exponent(widen<DT>(most)), kLowestScale);
    uint32_t drops = 0;
    for (int j = 0; j < JB; ++j) {
      const int block = 4 * j + g, drop = min(e - e2m1_exponent(widen<DT>(top[j])), kMostDrop);
      if (block < BLOCKS) drops |= (uint32_t)drop << (4 * block);
      const float un = power_of_two(drop - e);
      uint4v o;
      for (int i = 0; i < 4; ++i) {
        float4v a = widen4<DT>(uint2v{kr[j][i][0], kr[j][i][1]}) * un, b = widen4<DT>(uint2v{kr[j][i][2], kr[j][i][3]}) * un;
        if (special) {
          a = tame4(a);
          b = tame4(b);
        }
        o[i] = to_e2m1(a, b);
      }
      if (fresh && block < BLOCKS) *reinterpret_cast<uint4v*>(c.k + base + block * 256 + n * 16) = o;
    }
    drops |= (uint32_t)__shfl_xor((int)drops, 16);
    drops |= (uint32_t)__shfl_xor((int)drops, 32);
    if (fresh && g == 0) {
      scales[kt] = (uint8_t)(e + 127);
      store_drops<DROPS>(scales + 2 * P + kt * DROPS, drops);
    }
  }
  // ---- values
  uint32_t top[4];
  bool special = false;
  for (int i = 0; i < 4; ++i) {
    ushort2v m = {0, 0};
    for (int j = 0; j < J; ++j)
      for (int w = 0; w < 2; ++w) m = max_bits(m, vr[j][i][w]);
    top[i] = max(m[0], m[1]);
    if (top[i] >= kInf) {
      special = true;
      top[i] = 0;
      for (int j = 0; j < J; ++j)
        for (int w = 0; w < 2; ++w) top[i] = max_finite_bits<kInf>(top[i], vr[j][i][w]);
    }
    for (int w = 8; w; w >>= 1) top[i] = max(top[i], (uint32_t)__shfl_xor((int)top[i], w));
  }
  float un[4];
  for (int i = 0; i < 4; ++i) {
    const int e = max(e2m1_exponent(widen<DT>(top[i])), kLowestScale);
    un[i] = power_of_two(-e);
    if (n == i && vt + i >= t0 && vt + i < t1) scales[P + vt + i] = (uint8_t)(e + 127);
  }
  for (int j = 0; j < J; ++j) {
    uint32_t x[4];  // dim i, this lane's four tokens
    for (int i = 0; i < 4; ++i) {
      float4v y;
      for (int t = 0; t < 4; ++t) y[t] = widen<DT>(vr[j][t][i >> 1] >> (16 * (i & 1)) & 0xffffu) * un[t];
      if (special) y = tame4(y);
      x[i] = to_e2m1(y);
    }
    transpose_rows(x);  // dim 4 n + g, tokens 4 i + 0..3
    if (!S::v_has(j, lane)) continue;
    uint2v* at = reinterpret_cast<uint2v*>(c.v + base + (j * 64 + n * 4 + g) * 8);
    uint2v o = {x[0] | x[1] << 16, x[2] | x[3] << 16};
    if (b0 < t0 || b0 + 16 > t1) {
      const uint2v old = *at;
      for (int i = 0; i < 2; ++i) {
        const uint32_t mask = nibble_mask(b0 + 8 * i, t0, t1);
        o[i] = (o[i] & mask) | (old[i] & ~mask);
      }
    }
    *at = o;
  }
}

// Code times scale, exact in 32 bits, rounded once.
template <int DT, int D>
__global__ __launch_bounds__(1024) void k_cache4_read(CacheView c, SeqView s, UnitMap map, uint16_t* k, uint16_t* v) {
  using S = Share<D>;
  constexpr int J = S::J, DROPS = (int)drop_bytes(D);
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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const uint32_t head = blockIdx.y, P = 1u << c.page_log, first = (uint32_t)j64 << c.page_log;
  const int t0 = sp.start > first ? (int)(sp.start - first) : 0;
  const int t1 = (int)(last - first < P ? last - first + 1 : P);
  if (wave * 16 >= t1 || wave * 16 + 16 <= t0) return;
  uint32_t page = 0;
  const bool have = sp.ok && page_at(s, seq, (uint32_t)j64, c.pages, &page);
  if (sp.ok && !have && lane == 0) report(c, kCacheBadPage);
  // keys here: token 8 i + lane / 8, 8 dims, so that a row's 64 dims leave as one line
  const int kd = (lane & 7) * 8, ktok = lane >> 3;
  uint32_t kr[J][2], drops[2] = {0, 0}, ke[2] = {0, 0}, ve = 0;
  uint2v vr[J];
  for (int j = 0; j < J; ++j) {
    kr[j][0] = kr[j][1] = 0;
    vr[j] = uint2v{0, 0};
  }
  if (have) {
    const uint64_t base = head_offset(c, page, head) / 2 + (uint32_t)wave * (8 * D);
    const uint8_t* scales = c.scales + token_scales(c, page, head);
    for (int j = 0; j < J; ++j) {
      const int d = j * 64 + kd;
      if (d < D)
        for (int i = 0; i < 2; ++i)
          kr[j][i] = *reinterpret_cast<const uint32_t*>(c.k + base + (d >> 5) * 256 + (i * 8 + ktok) * 16 + (d & 31) / 2);
      if (S::v_has(j, lane)) vr[j] = *reinterpret_cast<const uint2v*>(c.v + base + (j * 64 + n * 4 + g) * 8);
    }
    for (int i = 0; i < 2; ++i) {
      const int t = wave * 16 + i * 8 + ktok;
      ke[i] = scales[t];
      drops[i] = load_drops<DROPS>(scales + 2 * P + t * DROPS);
    }
    ve = *reinterpret_cast<const uint32_t*>(scales + P + wave * 16 + g * 4);
  }
  const uint64_t row = (uint64_t)sp.row0 + first - sp.start;  // row of token 0 of the page, if asked for
  const uint64_t stride = (uint64_t)c.heads * D;
  for (int j = 0; j < J; ++j)
    for (int i = 0; i < 2; ++i) {
      const int t = wave * 16 + i * 8 + ktok, d = j * 64 + kd;
      if (!(t >= t0 && t < t1 && d < D)) continue;
      const float scale = __builtin_amdgcn_ldexpf(1.0f, (int)ke[i] - 127 - (int)(drops[i] >> (4 * (d >> 5)) & 15));
      const float2v a = two_values<0>(kr[j][i], 1.0f) * scale, b = two_values<1>(kr[j][i], 1.0f) * scale;
      const float2v x = two_values<2>(kr[j][i], 1.0f) * scale, y = two_values<3>(kr[j][i], 1.0f) * scale;
      *reinterpret_cast<uint4v*>(k + (row + t) * stride + head * D + d) =
          uint4v{pack2<DT>(a[0], a[1]), pack2<DT>(b[0], b[1]), pack2<DT>(x[0], x[1]), pack2<DT>(y[0], y[1])};
    }
  float vs[4];
  for (int i = 0; i < 4; ++i) vs[i] = power_of_two((int)(ve >> (8 * i) & 0xff) - 127);
  for (int j = 0; j < J; ++j) {
    uint32_t x[4] = {vr[j][0] & 0xffffu, vr[j][0] >> 16, vr[j][1] & 0xffffu, vr[j][1] >> 16};  // tokens 4 i + 0..3 of one dim
    transpose_rows(x);                                                                          // dim 4 n + i, tokens 4 g + 0..3
    float4v y[4];
    for (int i = 0; i < 4; ++i) {
      const float2v a = two_values<0>(x[i], 1.0f), b = two_values<1>(x[i], 1.0f);
      y[i] = float4v{a[0] * vs[0], a[1] * vs[1], b[0] * vs[2], b[1] * vs[3]};
    }
    for (int i = 0; i < 4; ++i) {
      const int t = wave * 16 + g * 4 + i;
      const uint2v o = {pack2<DT>(y[0][i], y[1][i]), pack2<DT>(y[2][i], y[3][i])};
      if (t >= t0 && t < t1 && S::v_has(j, lane))
        *reinterpret_cast<uint2v*>(v + (row + t) * stride + head * D + j * 64 + n * 4) = o;
    }
  }
}

}  // namespace

hipError_t launch_cache4_write(const CacheView& c, const SeqView& s, int dtype, const RowsView& k, const RowsView& v,
                               hipStream_t st) {
  return for_numbers(dtype, c.dim, [&](auto type, auto dim) {
    const UnitMap m = page_units(c, s);
    const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
    k_cache4_write<decltype(type)::value, decltype(dim)::value><<<grid, 4u << c.page_log, 0, st>>>(c, s, m, k, v);
  });
}

hipError_t launch_cache4_read(const CacheView& c, const SeqView& s, int dtype, uint16_t* k, uint16_t* v, hipStream_t st) {
  return for_numbers(dtype, c.dim, [&](auto type, auto dim) {
    const UnitMap m = page_units(c, s);
    const dim3 grid((uint32_t)unit_count(m, s.rows, s.seqs), c.heads);
    k_cache4_read<decltype(type)::value, decltype(dim)::value><<<grid, 4u << c.page_log, 0, st>>>(c, s, m, k, v);
  });
}

}  // namespace ltc
