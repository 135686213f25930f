// ltc_cache_api.hip -- host side of the key/value cache's C ABI: argument
// checks and launches.  Nothing here allocates or synchronises.
#include "ltc.h"
#include "ltc_cache_launch.h"

namespace ltc {
namespace {

constexpr uint32_t kMaxPages = 1u << 30;   // table entries are 32-bit
constexpr uint32_t kMaxHeads = 65535;      // a grid's second dimension
// grid limits: lanes of a grid's first dimension stay below 2^32, and the
// workgroups of an attention are counted in 32 bits
constexpr uint32_t kMaxRows = 1u << 24;
constexpr uint32_t kMaxSeqs = 1u << 20;
constexpr uint32_t kMaxEvictSeqs = 65535, kMaxEvictPages = 65535;  // a grid's further dimensions
constexpr uint64_t kMaxAttend = 1ull << 31;  // (rows + sequences) * query heads

bool aligned(const void* p, uintptr_t to) { return p && reinterpret_cast<uintptr_t>(p) % to == 0; }

int check_cache(const ltc_cache* c, CacheView* out) {
  if (!c) return LTC_ERR_INVALID_ARGUMENT;
  if (c->dtype != LTC_BF16 && c->dtype != LTC_FP16) return LTC_ERR_UNSUPPORTED_DTYPE;
  if (c->codes != LTC_E4M3 && c->codes != LTC_INT8 && c->codes != LTC_E2M1) return LTC_ERR_UNSUPPORTED_DTYPE;
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return LTC_ERR_INVALID_ARGUMENT;
  if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256)
    return LTC_ERR_INVALID_ARGUMENT;
  if (c->heads < 1 || c->heads > kMaxHeads || c->pages > kMaxPages) return LTC_ERR_INVALID_ARGUMENT;
  if (!aligned(c->d_status, 4)) return LTC_ERR_INVALID_ARGUMENT;
  if (c->pages && (!aligned(c->d_k_codes, 16) || !aligned(c->d_v_codes, 16) ||
                   !aligned(c->d_scales, c->codes == LTC_E2M1 ? 16 : 2)))
    return LTC_ERR_INVALID_ARGUMENT;
  out->k = static_cast<uint8_t*>(c->d_k_codes);
  out->v = static_cast<uint8_t*>(c->d_v_codes);
  out->scales = static_cast<uint8_t*>(c->d_scales);
  out->status = c->d_status;
  out->pages = c->pages;
  out->heads = c->heads;
  out->dim = c->dim;
  out->page_log = (uint32_t)__builtin_ctz(c->page);
  return LTC_OK;
}

int check_seqs(const ltc_cache_seqs* s, SeqView* out) {
  if (!s || s->reserved) return LTC_ERR_INVALID_ARGUMENT;
  if (s->rows > kMaxRows || s->seqs > kMaxSeqs) return LTC_ERR_INVALID_ARGUMENT;
  if (s->seqs) {
    if (!aligned(s->d_lengths, 4) || (s->width && !aligned(s->d_table, 4))) return LTC_ERR_INVALID_ARGUMENT;
    if (s->d_cu ? !aligned(s->d_cu, 4) : s->rows != s->seqs) return LTC_ERR_INVALID_ARGUMENT;
    if (s->table_stride < s->width) return LTC_ERR_INVALID_ARGUMENT;
  } else if (s->rows) {
    return LTC_ERR_INVALID_ARGUMENT;
  }
  out->table = s->d_table;
  out->lengths = s->d_lengths;
  out->cu = s->d_cu;
  out->table_stride = s->table_stride;
  out->seqs = s->seqs;
  out->rows = s->rows;
  out->width = s->width;
  return LTC_OK;
}

int check_rows(const ltc_cache_rows* r, RowsView* out) {
  if (!r || !aligned(r->d_base, 16) || r->row_stride % 8 || r->head_stride % 8) return LTC_ERR_INVALID_ARGUMENT;
  out->base = static_cast<const uint16_t*>(r->d_base);
  out->row_stride = r->row_stride;
  out->head_stride = r->head_stride;
  return LTC_OK;
}

int check_heads(const CacheView& c, const SeqView& s, uint32_t q_heads) {
  if (!q_heads || q_heads % c.heads || q_heads > kMaxHeads) return LTC_ERR_INVALID_ARGUMENT;
  return ((uint64_t)s.rows + s.seqs) * q_heads > kMaxAttend ? LTC_ERR_INVALID_ARGUMENT : LTC_OK;
}

int check_attend(const ltc_cache* cache, const ltc_cache_seqs* seqs, const ltc_cache_rows* q, uint32_t q_heads,
                 uint32_t window, float scale, void* d_out, CacheView* c, SeqView* s, AttendArgs* a) {
  int rc = check_cache(cache, c);
  if (!rc) rc = check_seqs(seqs, s);
  if (!rc) rc = check_heads(*c, *s, q_heads);
  if (rc) return rc;
  if (window > 0x7fffffffu || !(scale > 0.0f && scale < 1e30f)) return LTC_ERR_INVALID_ARGUMENT;
  if (!s->rows) return LTC_OK;
  rc = check_rows(q, &a->q);
  if (rc) return rc;
  if (!aligned(d_out, 16)) return LTC_ERR_INVALID_ARGUMENT;
  a->out = static_cast<uint16_t*>(d_out);
  a->q_heads = q_heads;
  a->window = window;
  a->scale = scale;
  a->ws = nullptr;
  a->lse = a->scores = nullptr;
  a->scores_stride = 0;
  return LTC_OK;
}

// where the rows' sums lie in the workspace of an attention that weighs: behind
// what the attention uses, and never in the bytes that calls leave zero
uint64_t lse_offset(const CacheView& c, const SeqView& s, int codes, int dtype, uint32_t q_heads, uint32_t window) {
  const uint64_t need = cache_attend_workspace(c, s, codes, dtype, q_heads, window);
  return need < LTC_CACHE_WS_ZEROS ? (uint64_t)LTC_CACHE_WS_ZEROS : (need + 255) / 256 * 256;
}

// the scores lie behind them
uint64_t scores_offset(const SeqView& s, uint32_t q_heads, uint64_t lse) {
  return (lse + (uint64_t)s.rows * q_heads * sizeof(float) + 255) / 256 * 256;
}

int launched(hipError_t e) { return e == hipSuccess ? LTC_OK : LTC_ERR_HIP; }

}  // namespace
}  // namespace ltc

using namespace ltc;

extern "C" {

int ltc_cache_write(const ltc_cache* cache, const ltc_cache_seqs* seqs, const ltc_cache_rows* k,
                    const ltc_cache_rows* v, hipStream_t stream) {
  CacheView c;
  SeqView s;
  RowsView kr, vr;
  int rc = check_cache(cache, &c);
  if (!rc) rc = check_seqs(seqs, &s);
  if (rc || !s.rows) return rc;
  if (!rc) rc = check_rows(k, &kr);
  if (!rc) rc = check_rows(v, &vr);
  if (rc) return rc;
  if (cache->codes == LTC_E2M1) return launched(launch_cache4_write(c, s, cache->dtype, kr, vr, stream));
  return launched(launch_cache_write(c, s, cache->codes == LTC_E4M3, cache->dtype, kr, vr, stream));
}

int ltc_cache_read(const ltc_cache* cache, const ltc_cache_seqs* seqs, void* d_k, void* d_v, hipStream_t stream) {
  CacheView c;
  SeqView s;
  int rc = check_cache(cache, &c);
  if (!rc) rc = check_seqs(seqs, &s);
  if (rc || !s.rows) return rc;
  if (!aligned(d_k, 16) || !aligned(d_v, 16)) return LTC_ERR_INVALID_ARGUMENT;
  uint16_t *k = static_cast<uint16_t*>(d_k), *v = static_cast<uint16_t*>(d_v);
  if (cache->codes == LTC_E2M1) return launched(launch_cache4_read(c, s, cache->dtype, k, v, stream));
  return launched(launch_cache_read(c, s, cache->codes == LTC_E4M3, cache->dtype, k, v, stream));
}

uint64_t ltc_cache_attend_workspace_size(const ltc_cache* cache, const ltc_cache_seqs* seqs, uint32_t q_heads,
                                         uint32_t window) {
  CacheView c;
  SeqView s;
  if (check_cache(cache, &c) || check_seqs(seqs, &s) || check_heads(c, s, q_heads)) return 0;
  return cache_attend_workspace(c, s, cache->codes, cache->dtype, q_heads, window);
}

int ltc_cache_attend(const ltc_cache* cache, const ltc_cache_seqs* seqs, const ltc_cache_rows* q, uint32_t q_heads,
                     uint32_t window, float scale, void* d_out, void* d_ws, uint64_t ws_nbytes, hipStream_t stream) {
  CacheView c;
  SeqView s;
  AttendArgs a;
  const int rc = check_attend(cache, seqs, q, q_heads, window, scale, d_out, &c, &s, &a);
  if (rc || !s.rows) return rc;
  const uint64_t need = cache_attend_workspace(c, s, cache->codes, cache->dtype, q_heads, window);
  if (need && (ws_nbytes < need || !aligned(d_ws, 256))) return LTC_ERR_WORKSPACE;
  a.ws = d_ws;
  return launched(launch_cache_attend(c, s, cache->codes, cache->dtype, a, stream));
}

uint64_t ltc_cache_attend_weigh_workspace_size(const ltc_cache* cache, const ltc_cache_seqs* seqs, uint32_t q_heads,
                                               uint32_t window) {
  CacheView c;
  SeqView s;
  if (check_cache(cache, &c) || check_seqs(seqs, &s) || check_heads(c, s, q_heads) || !s.rows) return 0;
  const uint64_t stride = cache_scores_stride(c, s, cache->codes, q_heads, window);
  return scores_offset(s, q_heads, lse_offset(c, s, cache->codes, cache->dtype, q_heads, window)) +
         stride * s.rows * q_heads * sizeof(float);
}

int ltc_cache_attend_weigh(const ltc_cache* cache, const ltc_cache_seqs* seqs, const ltc_cache_rows* q, uint32_t q_heads,
                           uint32_t window, float scale, void* d_out, float* d_weights, void* d_ws, uint64_t ws_nbytes,
                           hipStream_t stream) {
  CacheView c;
  SeqView s;
  AttendArgs a;
  const int rc = check_attend(cache, seqs, q, q_heads, window, scale, d_out, &c, &s, &a);
  if (rc || !s.rows) return rc;
  if (c.pages && !aligned(d_weights, 16)) return LTC_ERR_INVALID_ARGUMENT;
  const uint64_t lse = lse_offset(c, s, cache->codes, cache->dtype, q_heads, window), scores = scores_offset(s, q_heads, lse);
  a.scores_stride = cache_scores_stride(c, s, cache->codes, q_heads, window);
  if (ws_nbytes < scores + a.scores_stride * s.rows * q_heads * sizeof(float) || !aligned(d_ws, 256)) return LTC_ERR_WORKSPACE;
  a.ws = d_ws;
  a.lse = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + lse);
  if (a.scores_stride) a.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + scores);
  hipError_t e = launch_cache_attend(c, s, cache->codes, cache->dtype, a, stream);
  if (e != hipSuccess) return LTC_ERR_HIP;
  if (a.scores) return launched(launch_weigh_scores(c, s, a, d_weights, stream));
  switch (cache->codes) {
    case LTC_E4M3: e = launch_weigh<LTC_E4M3>(c, s, cache->dtype, a, d_weights, stream); break;
    case LTC_INT8: e = launch_weigh<LTC_INT8>(c, s, cache->dtype, a, d_weights, stream); break;
    default: e = launch_weigh<LTC_E2M1>(c, s, cache->dtype, a, d_weights, stream); break;
  }
  return launched(e);
}

uint64_t ltc_cache_evict_workspace_size(const ltc_cache* cache, const ltc_cache_seqs* seqs) {
  CacheView c;
  SeqView s;
  if (check_cache(cache, &c) || check_seqs(seqs, &s)) return 0;
  const uint64_t need = cache_evict_workspace(c, s);
  return need ? LTC_CACHE_WS_ZEROS + need : 0;
}

int ltc_cache_evict(const ltc_cache* cache, const ltc_cache_seqs* seqs, float* d_weights, const int32_t* d_to,
                    uint64_t to_stride, uint32_t to_width, uint32_t keep, uint32_t recent, int32_t* d_lengths,
                    int32_t* d_positions, void* d_ws, uint64_t ws_nbytes, hipStream_t stream) {
  CacheView c;
  SeqView s;
  int rc = check_cache(cache, &c);
  if (!rc) rc = check_seqs(seqs, &s);
  if (rc) return rc;
  if (s.cu || s.seqs > kMaxEvictSeqs) return LTC_ERR_INVALID_ARGUMENT;
  const uint64_t pages = ((uint64_t)keep + cache->page - 1) / cache->page;
  if (!keep || recent > keep || pages > kMaxEvictPages || to_width < pages || to_stride < to_width)
    return LTC_ERR_INVALID_ARGUMENT;
  if (!s.seqs) return LTC_OK;
  if ((c.pages && !aligned(d_weights, 16)) || !aligned(d_to, 4) || !aligned(d_lengths, 4) || !aligned(d_positions, 4))
    return LTC_ERR_INVALID_ARGUMENT;
  const uint64_t need = cache_evict_workspace(c, s);
  if (need && (ws_nbytes < LTC_CACHE_WS_ZEROS + need || !aligned(d_ws, 256))) return LTC_ERR_WORKSPACE;
  // the workgroups of a sequence's heads read its length when one of them may have written the new one
  const uintptr_t from = reinterpret_cast<uintptr_t>(s.lengths), to = reinterpret_cast<uintptr_t>(d_lengths);
  if ((from > to ? from - to : to - from) < s.seqs * sizeof(int32_t)) return LTC_ERR_INVALID_ARGUMENT;
  // behind the bytes that calls leave zero
  uint32_t* ws = need ? reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + LTC_CACHE_WS_ZEROS) : nullptr;
  const EvictArgs a = {d_weights, d_to, to_stride, keep, recent, d_lengths, d_positions, ws};
  return launched(launch_cache_evict(c, s, cache->codes, a, stream));
}

}  // extern "C"
