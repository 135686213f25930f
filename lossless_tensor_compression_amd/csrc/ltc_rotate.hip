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

// A workgroup takes a row, its waves the heads in turn, 64 / (D / 8) at a time,
// queries' and keys' in one list.  An angle is a number of turns in 64 bits of
// fraction: the position times the turns of one position, modulo 1 by the product's
// overflow, so far positions lose nothing but what fp32 does of any (2^-26 of a turn).
// A row's angles are the same for all its heads: each of a wave's lanes makes one or
// two, while the row's first numbers are on their way, and finds its dims' in shared
// memory.  (With every lane making its own eight, 15,413 rows of 40 heads took 105 us;
// 70 us so, 4.5 TB/s, where a 1 GiB copy runs at 5.1.)  A head's sum of squares goes
// over its lanes; the numbers that a lane's are turned with come from the lane half of
// the dims away.
template <int DT, int D, int W>
__global__ __launch_bounds__(64 * W) void k_norm_rotate(SeqView s, RotateArgs a) {
  constexpr int L = D / 8, HEADS = 64 / L, AHEAD = 3;
  __shared__ float2v angles[W][D / 2];  // cosine and sine
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t row = blockIdx.x, heads = a.q_heads + a.k_heads;
  const int o = lane % L, slot = lane / L;
  auto load = [&](uint32_t h) -> uint4v {
    if (row >= s.rows || slot >= HEADS || h >= heads) return uint4v{0, 0, 0, 0};
    const bool key = h >= a.q_heads;
    const RowsView& in = key ? a.k : a.q;
    return *reinterpret_cast<const uint4v*>(in.base + (uint64_t)row * in.row_stride +
                                            (uint64_t)(key ? h - a.q_heads : h) * in.head_stride + o * 8);
  };
  const uint32_t h_first = wave * HEADS + slot, h_by = W * HEADS;
  uint4v raw[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) raw[i] = load(h_first + i * h_by);
  uint64_t turns[2];
  const int pairs = (int)a.rotary / 2;
  for (int i = 0; i < 2; ++i) turns[i] = lane + 64 * i < pairs ? a.turns[lane + 64 * i] : 0;
  // the lane's numbers and those that they are turned with: of the same lane, in pairs,
  // or of the one that is half of the turned dims away
  const bool turned = o * 8 < (int)a.rotary;
  const int far = !turned || a.pairs ? o : o * 8 < pairs ? o + pairs / 8 : o - pairs / 8;
  uint4v weights[2][2] = {};  // of queries and keys: the lane's dims, and those that they are turned with
  for (int kind = 0; kind < 2; ++kind) {
    const uint16_t* weight = kind ? a.k_weight : a.q_weight;
    if (!weight) continue;
    weights[kind][0] = *reinterpret_cast<const uint4v*>(weight + o * 8);
    weights[kind][1] = *reinterpret_cast<const uint4v*>(weight + far * 8);
  }
  const UnitMap map = {1, 1, 0};
  const uint32_t seq = s.cu ? find_sequence(s.seqs, WaveCount{s, map, row}) : min(row, s.seqs - 1);
  auto span = [&](uint32_t i) {
    const int32_t c0 = s.cu ? s.cu[i] : (int32_t)i, c1 = s.cu ? s.cu[i + 1] : (int32_t)i + 1;
    return span_of(c0, c1, s.lengths[i], s.rows, kMostPositions);
  };
  const Span sp = span(seq);
  if (threadIdx.x == 0 && (!sp.ok || (s.cu && row < s.seqs && !span(row).ok))) atomicOr(a.status, kCacheBadSeq);
  if (row >= s.rows) return;
  const bool named = sp.ok && row >= sp.row0 && row - sp.row0 < sp.n;
  const uint64_t position = named ? sp.start + (row - sp.row0) : 0;
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < pairs) {
      const int32_t turn = (int32_t)(position * turns[i] >> 32);
      float cos, sin;
      sincospif((float)turn * 0x1p-31f, &sin, &cos);  // half turns in [-1, 1)
      angles[wave][lane + 64 * i] = float2v{cos, sin};
    }
  // written and read by one wave, whose accesses stay in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  float cos[8], sin[8];
  for (int i = 0; i < 8; ++i) {
    cos[i] = 1.0f;
    sin[i] = 0.0f;
  }
  if (turned) {
    if (a.pairs) {
      for (int i = 0; i < 4; ++i) {
        const float2v x = angles[wave][o * 4 + i];
        cos[2 * i] = cos[2 * i + 1] = x[0];
        sin[2 * i] = -x[1];
        sin[2 * i + 1] = x[1];
      }
    } else {
      const bool low = o * 8 < pairs;
      for (int i = 0; i < 8; ++i) {
        const float2v x = angles[wave][(low ? o * 8 : o * 8 - pairs) + i];
        cos[i] = x[0];
        sin[i] = low ? -x[1] : x[1];
      }
    }
  }
  const int from = lane - o + far;
  for (uint32_t h0 = 0; h0 < heads; h0 += AHEAD * h_by) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const uint32_t h = h0 + k * h_by + h_first;
      if (h0 + k * h_by + wave * HEADS >= heads) break;  // none of the wave's
      const bool live = slot < HEADS && h < heads, key = h >= a.q_heads;
      const bool norm = key ? a.k_weight != nullptr : a.q_weight != nullptr;
      const uint4v mine = raw[k];
      raw[k] = load(h + AHEAD * h_by);
      uint4v other;
      for (int i = 0; i < 4; ++i) other[i] = (uint32_t)__shfl((int)mine[i], from);
      float x[8], y[8];
      widen8<DT>(mine, x);
      widen8<DT>(other, y);
      float sum = 0.0f;
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
      sum = sum_lanes<L>(sum, lane);
      if (norm) {
        const float r = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
        float w[8], v[8];
        widen8<DT>(weights[key][0], w);
        widen8<DT>(weights[key][1], v);
        for (int i = 0; i < 8; ++i) {
          x[i] *= r * w[i];
          y[i] *= r * v[i];
        }
      }
      uint4v out;
      for (int i = 0; i < 8; i += 2) {
        float z[2];
        for (int j = 0; j < 2; ++j) {
          const int e = i + j;
          z[j] = turned ? fmaf(x[e], cos[e], (a.pairs ? x[e ^ 1] : y[e]) * sin[e]) : x[e];
        }
        out[i / 2] = pack2<DT>(z[0], z[1]);
      }
      if (!named) out = uint4v{0, 0, 0, 0};
      if (live) {
        uint16_t* to = key ? a.k_out + ((uint64_t)row * a.k_heads + (h - a.q_heads)) * D
                           : a.q_out + ((uint64_t)row * a.q_heads + h) * D;
        *reinterpret_cast<uint4v*>(to + o * 8) = out;
      }
    }
  }
}

bool aligned(const void* p, uintptr_t to) { return p && reinterpret_cast<uintptr_t>(p) % to == 0; }

bool take_rows(const ltc_cache_rows& r, RowsView* out) {
  if (!aligned(r.d_base, 16) || r.row_stride % 8 || r.head_stride % 8) return false;
  *out = RowsView{static_cast<const uint16_t*>(r.d_base), r.row_stride, r.head_stride};
  return true;
}

}  // namespace
}  // namespace ltc

using namespace ltc;

extern "C" int ltc_norm_rotate(const ltc_rotation* rotation, const ltc_cache_seqs* seqs, const ltc_rotate_rows* rows,
                               hipStream_t stream) {
  if (!rotation || !seqs || !rows || seqs->reserved || rotation->reserved) return LTC_ERR_INVALID_ARGUMENT;
  if (rows->dtype != LTC_BF16 && rows->dtype != LTC_FP16) return LTC_ERR_UNSUPPORTED_DTYPE;
  const uint32_t dim = rotation->dim;
  if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return LTC_ERR_INVALID_ARGUMENT;
  if (rotation->rotary > dim || rotation->rotary % 16 || rotation->pairs > 1) return LTC_ERR_INVALID_ARGUMENT;
  if (!aligned(rotation->d_status, 4) || (rotation->rotary && !aligned(rotation->d_turns, 8))) return LTC_ERR_INVALID_ARGUMENT;
  if (seqs->rows > (1u << 24) || seqs->seqs > (1u << 20)) return LTC_ERR_INVALID_ARGUMENT;
  if (!(rows->eps >= 0.0f && rows->eps < 1e30f) || rows->q_heads > 65535 || rows->k_heads > 65535)
    return LTC_ERR_INVALID_ARGUMENT;
  if (!seqs->seqs) return seqs->rows ? LTC_ERR_INVALID_ARGUMENT : LTC_OK;
  if (!aligned(seqs->d_lengths, 4) || (seqs->d_cu ? !aligned(seqs->d_cu, 4) : seqs->rows != seqs->seqs))
    return LTC_ERR_INVALID_ARGUMENT;
  if (!seqs->rows) return LTC_OK;
  RotateArgs a = {};
  if (rows->q_heads && (!take_rows(rows->q, &a.q) || !aligned(rows->d_q_out, 16))) return LTC_ERR_INVALID_ARGUMENT;
  if (rows->k_heads && (!take_rows(rows->k, &a.k) || !aligned(rows->d_k_out, 16))) return LTC_ERR_INVALID_ARGUMENT;
  if ((rows->d_q_weight && !aligned(rows->d_q_weight, 16)) || (rows->d_k_weight && !aligned(rows->d_k_weight, 16)))
    return LTC_ERR_INVALID_ARGUMENT;
  SeqView s = {};
  s.lengths = seqs->d_lengths;
  s.cu = seqs->d_cu;
  s.seqs = seqs->seqs;
  s.rows = seqs->rows;
  a.q_out = static_cast<uint16_t*>(rows->d_q_out);
  a.k_out = static_cast<uint16_t*>(rows->d_k_out);
  a.q_weight = static_cast<const uint16_t*>(rows->d_q_weight);
  a.k_weight = static_cast<const uint16_t*>(rows->d_k_weight);
  a.turns = rotation->d_turns;
  a.status = rotation->d_status;
  a.q_heads = rows->q_heads;
  a.k_heads = rows->k_heads;
  a.rotary = rotation->rotary;
  a.pairs = rotation->pairs;
  a.eps = rows->eps;
  // a workgroup for each row, and for each sequence, which it checks
  const uint32_t units = s.rows > s.seqs ? s.rows : s.seqs;
  const hipError_t e = for_numbers(rows->dtype, dim, [&](auto type, auto d) {
    constexpr int DT = decltype(type)::value, D = decltype(d)::value;
    // few rows: more waves share one's heads; many, and there are waves enough: fewer
    // make its angles.  4 / 2 waves: 48 rows of 40 heads 5.1 / 6.5 us, 15,413 of them
    // 77 / 70 us.
    if (units <= 1024) k_norm_rotate<DT, D, 4><<<units, 256, 0, stream>>>(s, a);
    else k_norm_rotate<DT, D, 2><<<units, 128, 0, stream>>>(s, a);
  });
  return e == hipSuccess ? LTC_OK : LTC_ERR_HIP;
}
