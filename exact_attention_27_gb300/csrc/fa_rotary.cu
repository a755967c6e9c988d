// Entry points of rotary positions and of appending to a paged cache (fa_rotary.cuh has the
// kernel), and the checks that they share with the norms' (fa_norm.cu).

#include "fa_rotary.cuh"

namespace fa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool good_stride(long long s) { return s >= 0 && s % 8 == 0; }

// Strides of an output must keep the rows apart (a zero stride is for inputs).
bool good_out(long long stride, long long extent) {
  return good_stride(stride) && (stride > 0 || extent == 1);
}

bool put_rows(TurnRows& R, const fa_rotary_rows& r, int B, int N) {
  if (!r.in || !r.out || !aligned16(r.in) || !aligned16(r.out) || r.heads < 1) return false;
  if (!good_stride(r.in_batch) || !good_stride(r.in_head) || !good_stride(r.in_pos)) return false;
  if (!good_out(r.out_batch, B) || !good_out(r.out_head, r.heads) || !good_out(r.out_pos, N))
    return false;
  R = TurnRows{static_cast<const __nv_bfloat16*>(r.in), static_cast<__nv_bfloat16*>(r.out),
           r.in_batch, r.in_head, r.in_pos, r.out_batch, r.out_head, r.out_pos, r.heads};
  return true;
}

}  // namespace

bool good_spec(const fa_rotary_spec& r, int d) {
  if (!r.inv_freq || (reinterpret_cast<uintptr_t>(r.inv_freq) & 3u)) return false;
  if (r.rot_dim < 16 || r.rot_dim % 16 != 0 || r.rot_dim > d) return false;
  if (r.axes < 1 || r.axes > 4 || (r.interleaved != 0 && r.interleaved != 1)) return false;
  for (int i = 0; i < r.rot_dim / 2; ++i)
    if (r.axis[i] >= r.axes) return false;
  return true;
}

void put_spec(TurnParams& p, const fa_rotary_spec& r) {
  p.inv_freq = r.inv_freq;
  p.half = r.rot_dim / 2;
  p.interleaved = r.interleaved;
  std::memcpy(p.axis, r.axis, sizeof(p.axis));
}

fa_status put_turn(TurnParams& p, const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N,
                   int d, const int* positions, long long axis_stride, long long batch_stride,
                   const fa_rotary_spec* spec, float sign) {
  if (!q || (spec && !positions) || B < 1 || N < 1) return FA_ERR_INVALID_ARGUMENT;
  if (d != 64 && d != 96 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) || axis_stride < 0 || batch_stride < 0)
    return FA_ERR_INVALID_ARGUMENT;
  if ((spec && !good_spec(*spec, d)) || !put_rows(p.q, *q, B, N) || (k && !put_rows(p.k, *k, B, N)))
    return FA_ERR_INVALID_ARGUMENT;
  p.tokens = static_cast<long long>(B) * N;
  if (p.tokens > 0x7fffffffLL || (static_cast<long long>(p.q.heads) + p.k.heads) * d > (1 << 24))
    return FA_ERR_INVALID_ARGUMENT;
  p.N = N;
  p.positions = spec ? positions : nullptr;
  p.axis_stride = axis_stride;
  p.batch_stride = batch_stride;
  p.sign = sign;
  if (spec) put_spec(p, *spec);
  return FA_OK;
}

namespace {

fa_status turn(const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N, int d,
               const int* positions, long long axis_stride, long long batch_stride,
               const fa_rotary_spec* spec, float sign, cudaStream_t stream) {
  if (!spec) return FA_ERR_INVALID_ARGUMENT;
  TurnParams p{};
  const fa_status st =
      put_turn(p, q, k, B, N, d, positions, axis_stride, batch_stride, spec, sign);
  if (st != FA_OK) return st;
  return launch_turn<kTurnOnly>(p, d, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

fa_status validate_cache(const fa_paged_cache* c, const fa_paged_batch* b, int T) {
  if (!c || !b || T < 0 || b->S < 0) return FA_ERR_INVALID_ARGUMENT;
  if (c->d != 64 && c->d != 96 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (c->H_kv < 1 || c->n_pages < 1 || b->max_pages < 0 || b->max_q_len < 0)
    return FA_ERR_INVALID_ARGUMENT;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return FA_ERR_INVALID_ARGUMENT;
  if (c->dtype != FA_CACHE_BF16 && c->dtype != FA_CACHE_E4M3) return FA_ERR_INVALID_ARGUMENT;
  for (float f : {c->k_descale, c->v_descale})
    if (!std::isfinite(f) || !(f > 0.0f) || !std::isfinite(1.0f / f) ||
        (c->dtype == FA_CACHE_BF16 && f != 1.0f))
      return FA_ERR_INVALID_ARGUMENT;
  const int elem = c->dtype == FA_CACHE_BF16 ? 2 : 1;
  // Rows, heads and pages lie apart and start on 16-byte boundaries; a tensor
  // map's strides end at 2^40 bytes.
  for (long long s : {c->row_stride, c->head_stride, c->page_stride})
    if (s < c->d || s * elem % 16 != 0 || s >= (1LL << 39)) return FA_ERR_INVALID_ARGUMENT;
  // Positions are 32-bit.
  if (static_cast<long long>(b->max_pages) * c->page_size > 0x7fffff00LL)
    return FA_ERR_INVALID_ARGUMENT;
  if (T == 0 || b->S == 0) return FA_OK;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return FA_ERR_INVALID_ARGUMENT;
  if (!b->q_start || !b->kv_len || !b->block_table || b->max_pages < 1 || b->table_stride < 0)
    return FA_ERR_INVALID_ARGUMENT;
  for (const int* q : {b->q_start, b->kv_len, b->block_table})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return FA_ERR_INVALID_ARGUMENT;
  return FA_OK;
}

fa_status put_append(TurnParams& p, const fa_paged_cache* cache, const fa_paged_batch* batch,
                     const void* k, long long k_token, long long k_head, const void* v,
                     long long v_token, long long v_head, int T, const void* q, long long q_token,
                     long long q_head, void* q_out, long long qo_token, long long qo_head, int H_q,
                     const fa_rotary_spec* spec, const int* positions, long long axis_stride,
                     bool* nothing) {
  const fa_status st = validate_cache(cache, batch, T);
  if (st != FA_OK) return st;
  if (spec && !good_spec(*spec, cache->d)) return FA_ERR_INVALID_ARGUMENT;
  if (!q != !q_out || (q && H_q < 1)) return FA_ERR_INVALID_ARGUMENT;
  *nothing = T == 0 || batch->S == 0;
  if (*nothing) return FA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out))
    return FA_ERR_INVALID_ARGUMENT;
  for (long long s : {k_token, k_head, v_token, v_head})
    if (!good_stride(s)) return FA_ERR_INVALID_ARGUMENT;
  if (q && (!good_stride(q_token) || !good_stride(q_head) || !good_out(qo_token, T) ||
            !good_out(qo_head, H_q)))
    return FA_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) || axis_stride < 0)
    return FA_ERR_INVALID_ARGUMENT;
  const int H = cache->H_kv;
  if (((q ? static_cast<long long>(H_q) : 0) + 2LL * H) * cache->d > (1 << 24))
    return FA_ERR_INVALID_ARGUMENT;
  p.err = device_error_word();
  if (!p.err) return FA_ERR_CUDA;
  if (q)
    p.q = TurnRows{static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(q_out), 0, q_head,
               q_token, 0, qo_head, qo_token, H_q};
  p.k = TurnRows{static_cast<const __nv_bfloat16*>(k), nullptr, 0, k_head, k_token, 0, 0, 0, H};
  p.v = TurnRows{static_cast<const __nv_bfloat16*>(v), nullptr, 0, v_head, v_token, 0, 0, 0, H};
  p.N = T;
  p.tokens = T;
  p.positions = positions;
  p.axis_stride = axis_stride;
  p.sign = 1.0f;
  if (spec) put_spec(p, *spec);
  p.q_start = batch->q_start;
  p.kv_len = batch->kv_len;
  p.table = batch->block_table;
  p.table_stride = batch->table_stride;
  p.S = batch->S;
  p.max_pages = batch->max_pages;
  p.page_size = cache->page_size;
  p.n_pages = cache->n_pages;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.k_pages = cache->k;
  p.v_pages = cache->v;
  p.k_scale = 1.0f / cache->k_descale;
  p.v_scale = 1.0f / cache->v_descale;
  return FA_OK;
}

}  // namespace fa

extern "C" {

fa_status fa_rotary(const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N, int d,
                    const int* positions, long long axis_stride, long long batch_stride,
                    const fa_rotary_spec* spec, cudaStream_t stream) {
  return fa::turn(q, k, B, N, d, positions, axis_stride, batch_stride, spec, 1.0f, stream);
}

fa_status fa_rotary_backward(const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N, int d,
                             const int* positions, long long axis_stride, long long batch_stride,
                             const fa_rotary_spec* spec, cudaStream_t stream) {
  return fa::turn(q, k, B, N, d, positions, axis_stride, batch_stride, spec, -1.0f, stream);
}

fa_status fa_paged_append(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* k,
                          long long k_token, long long k_head, const void* v, long long v_token,
                          long long v_head, int T, const void* q, long long q_token,
                          long long q_head, void* q_out, long long qo_token, long long qo_head,
                          int H_q, const fa_rotary_spec* spec, const int* positions,
                          long long axis_stride, cudaStream_t stream) {
  using namespace fa;
  TurnParams p{};
  bool nothing = false;
  const fa_status st =
      put_append(p, cache, batch, k, k_token, k_head, v, v_token, v_head, T, q, q_token, q_head,
                 q_out, qo_token, qo_head, H_q, spec, positions, axis_stride, &nothing);
  if (st != FA_OK || nothing) return st;
  const cudaError_t e = cache->dtype == FA_CACHE_BF16 ? launch_turn<kToBf16>(p, cache->d, stream)
                                                      : launch_turn<kToE4m3>(p, cache->d, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
