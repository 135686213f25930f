// ltc_rotate.hip -- queries and keys on their way to the cache: the norm of each
// head, and the rotation by the row's position, in one pass; argument checks and
// entry point.
#include "ltc.h"
#include "ltc_cache_device.h"

namespace ltc {
namespace {

struct RotateArgs {
  RowsView q, k;
  uint16_t *q_out, *k_out;
  const uint16_t *q_weight, *k_weight;  // null: no norm
  const uint64_t* turns;
  uint32_t* status;
  uint32_t q_heads, k_heads, rotary, pairs;
  float eps;
};

constexpr uint64_t kMostPositions = 0x7fffffff;
constexpr int kRotateWaves = 4;

// Lanes of a head: eight numbers each.  Their sum over the head's lanes, which
// are a power of two, or three times one, and begin at a multiple of it.
template <int L> __device__ __forceinline__ float sum_lanes(float x, int lane) {
  constexpr int P = L & -L;
  for (int w = 1; w < P; w <<= 1) x += __shfl_xor(x, w);
  if constexpr (P < L) {
    const int o = lane % L, base = lane - o;
    const float a = __shfl(x, base + (o + P) % L), b = __shfl(x, base + (o + 2 * P) % L);
    x += a + b;
  }
  return x;
}

template <int DT> __device__ __forceinline__ void widen8(uint4v x, float (&y)[8]) {
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = widen<DT>(x[i] & 0xffffu);
    y[2 * i + 1] = widen<DT>(x[i] >> 16);
  }
}

// A workgroup takes a row, its waves the heads in turn, 64 / (D / 8) at a time.
// A row's angles are the same for all its heads.  An angle is a number of turns
// in 64 bits of fraction: the position times the turns of one position, modulo 1
// by the product's overflow, so far positions lose nothing.
template <int DT, int D>
__global__ __launch_bounds__(64 * kRotateWaves) void k_norm_rotate(SeqView s, RotateArgs a) {
  constexpr int L = D / 8, HEADS = 64 / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t row = blockIdx.x;
  const UnitMap map = {1, 1, 0};
  const uint32_t seq = find_sequence(s.seqs, WaveCount{s, map, row});
  auto span = [&](uint32_t i) {
    const int32_t c0 = s.cu ? s.cu[i] : (int32_t)i, c1 = s.cu ? s.cu[i + 1] : (int32_t)i + 1;
    return span_of(c0, c1, s.lengths[i], s.rows, kMostPositions);
  };
  const Span sp = span(seq);
  if (threadIdx.x == 0 && (!sp.ok || (row < s.seqs && !span(row).ok))) atomicOr(a.status, kCacheBadSeq);
  if (row >= s.rows) return;
  const bool named = sp.ok && row >= sp.row0 && row - sp.row0 < sp.n;
  const int o = lane % L, slot = lane / L;
  // the lane's numbers and those that they are turned with: 8 of the same lane, in
  // pairs, or of the one that is half of the turned dims away
  const int far = a.pairs ? o : o * 8 < (int)a.rotary / 2 ? o + (int)a.rotary / 16 : o - (int)a.rotary / 16;
  const bool turned = o * 8 < (int)a.rotary;
  const int from = turned ? lane - o + far : lane;
  float cos[8], sin[8];
  for (int i = 0; i < 8; ++i) {
    cos[i] = 1.0f;
    sin[i] = 0.0f;
  }
  if (turned) {
    const uint64_t position = sp.start + (row - sp.row0);
    const int n = a.pairs ? 4 : 8, first = a.pairs ? o * 4 : o * 8 % ((int)a.rotary / 2);
    for (int i = 0; i < n; ++i) {
      // half turns in [-1, 1)
      const int32_t turn = (int32_t)(position * a.turns[first + i] >> 32);
      float c, sn;
      sincospif((float)turn * 0x1p-31f, &sn, &c);
      if (a.pairs) {
        cos[2 * i] = cos[2 * i + 1] = c;
        sin[2 * i] = -sn;
        sin[2 * i + 1] = sn;
      } else {
        cos[i] = c;
        sin[i] = o * 8 < (int)a.rotary / 2 ? -sn : sn;
      }
    }
  }
  for (int kind = 0; kind < 2; ++kind) {
    const RowsView& in = kind ? a.k : a.q;
    const uint16_t* weight = kind ? a.k_weight : a.q_weight;
    const uint32_t heads = kind ? a.k_heads : a.q_heads;
    uint16_t* out = kind ? a.k_out : a.q_out;
    float w[8], far_w[8];  // the weights of the lane's dims and of those that they are turned with
    for (int i = 0; i < 8; ++i) w[i] = far_w[i] = 1.0f;
    if (weight && slot < HEADS) {
      widen8<DT>(*reinterpret_cast<const uint4v*>(weight + o * 8), w);
      widen8<DT>(*reinterpret_cast<const uint4v*>(weight + (turned ? far : o) * 8), far_w);
    }
    for (uint32_t h0 = wave * HEADS; h0 < heads; h0 += kRotateWaves * HEADS) {
      const uint32_t head = h0 + slot;
      const bool live = slot < HEADS && head < heads;
      uint4v raw = {0, 0, 0, 0}, far_raw;
      if (live && named)
        raw = *reinterpret_cast<const uint4v*>(in.base + (uint64_t)row * in.row_stride + (uint64_t)head * in.head_stride + o * 8);
      for (int i = 0; i < 4; ++i) far_raw[i] = (uint32_t)__shfl((int)raw[i], from);
      float x[8], y[8];
      widen8<DT>(raw, x);
      widen8<DT>(far_raw, y);
      float r = 1.0f;
      if (weight) {
        float sum = 0.0f;
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
        sum = sum_lanes<L>(sum, lane);
        r = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
      }
      uint4v o4;
      for (int i = 0; i < 8; i += 2) {
        float z[2];
        for (int j = 0; j < 2; ++j) {
          const int e = i + j;
          const float mine = x[e] * r * w[e];
          const float other = a.pairs ? x[e ^ 1] * r * w[e ^ 1] : y[e] * r * far_w[e];
          z[j] = turned ? fmaf(mine, cos[e], other * sin[e]) : mine;
        }
        o4[i / 2] = pack2<DT>(z[0], z[1]);
      }
      if (!named) o4 = uint4v{0, 0, 0, 0};
      if (live) *reinterpret_cast<uint4v*>(out + ((uint64_t)row * heads + head) * D + o * 8) = o4;
    }
  }
}

bool aligned(const void* p, uintptr_t to) { return p && reinterpret_cast<uintptr_t>(p) % to == 0; }

bool take_rows(const ltc_cache_rows* r, RowsView* out) {
  if (!r || !aligned(r->d_base, 16) || r->row_stride % 8 || r->head_stride % 8) return false;
  *out = RowsView{static_cast<const uint16_t*>(r->d_base), r->row_stride, r->head_stride};
  return true;
}

}  // namespace
}  // namespace ltc

using namespace ltc;

extern "C" int ltc_norm_rotate(const ltc_rotation* rotation, const ltc_cache_seqs* seqs, int dtype, const ltc_cache_rows* q,
                               uint32_t q_heads, const void* d_q_weight, const ltc_cache_rows* k, uint32_t k_heads,
                               const void* d_k_weight, float eps, void* d_q_out, void* d_k_out, hipStream_t stream) {
  if (!rotation || !seqs || seqs->reserved) return LTC_ERR_INVALID_ARGUMENT;
  if (dtype != LTC_BF16 && dtype != LTC_FP16) return LTC_ERR_UNSUPPORTED_DTYPE;
  const uint32_t dim = rotation->dim;
  if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return LTC_ERR_INVALID_ARGUMENT;
  if (rotation->rotary > dim || rotation->rotary % 16 || rotation->pairs > 1) return LTC_ERR_INVALID_ARGUMENT;
  if (!aligned(rotation->d_status, 4) || (rotation->rotary && !aligned(rotation->d_turns, 8))) return LTC_ERR_INVALID_ARGUMENT;
  if (seqs->rows > (1u << 24) || seqs->seqs > (1u << 20)) return LTC_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.0f && eps < 1e30f) || q_heads > 65535 || k_heads > 65535) return LTC_ERR_INVALID_ARGUMENT;
  if (!seqs->seqs) return seqs->rows ? LTC_ERR_INVALID_ARGUMENT : LTC_OK;
  if (!aligned(seqs->d_lengths, 4) || (seqs->d_cu ? !aligned(seqs->d_cu, 4) : seqs->rows != seqs->seqs))
    return LTC_ERR_INVALID_ARGUMENT;
  if (!seqs->rows) return LTC_OK;
  RotateArgs a = {};
  if (q_heads && (!take_rows(q, &a.q) || !aligned(d_q_out, 16))) return LTC_ERR_INVALID_ARGUMENT;
  if (k_heads && (!take_rows(k, &a.k) || !aligned(d_k_out, 16))) return LTC_ERR_INVALID_ARGUMENT;
  if ((d_q_weight && !aligned(d_q_weight, 16)) || (d_k_weight && !aligned(d_k_weight, 16))) return LTC_ERR_INVALID_ARGUMENT;
  SeqView s = {};
  s.lengths = seqs->d_lengths;
  s.cu = seqs->d_cu;
  s.seqs = seqs->seqs;
  s.rows = seqs->rows;
  a.q_out = static_cast<uint16_t*>(d_q_out);
  a.k_out = static_cast<uint16_t*>(d_k_out);
  a.q_weight = static_cast<const uint16_t*>(d_q_weight);
  a.k_weight = static_cast<const uint16_t*>(d_k_weight);
  a.turns = rotation->d_turns;
  a.status = rotation->d_status;
  a.q_heads = q_heads;
  a.k_heads = k_heads;
  a.rotary = rotation->rotary;
  a.pairs = rotation->pairs;
  a.eps = eps;
  // a workgroup for each row, and for each sequence, which it checks
  const uint32_t units = s.rows > s.seqs ? s.rows : s.seqs;
  const hipError_t e = for_numbers(dtype, dim, [&](auto type, auto d) {
    k_norm_rotate<decltype(type)::value, decltype(d)::value><<<units, 64 * kRotateWaves, 0, stream>>>(s, a);
  });
  return e == hipSuccess ? LTC_OK : LTC_ERR_HIP;
}
