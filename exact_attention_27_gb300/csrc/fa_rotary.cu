// Rotary positions and appending to a paged cache (fa_rotary.cuh has the mathematics): the
// kernel, the entry points, and the checks that they share with the norms' (fa_norm.cu).
//
// Both are bound by memory: they read and write every row once (3 operations
// for 4 bytes of traffic).  The angles of a position are shared by all its
// heads: a block takes TOK positions, one thread makes one sine and cosine, and
// a thread then keeps those of its 8 pairs in registers and goes through the
// heads, kBatch at a time, the first of them loaded before the angles are made.
// 16384 positions of 32 + 8 heads at d = 128: 55.8 us, 6.0 TB/s.  (Four heads at a
// time at this occupancy spill: 76 us; at three blocks an SM 54.2 us, but 8192
// positions of 16 heads, d = 64, take 9.7 us instead of 8.6 and the append below
// 39.3.)  Appending 8527 tokens of 32 + 8 + 8 heads, d = 128, to e4m3 pages: 37.5 us,
// 5.1 TB/s (40.2 us with a thread's k rows before its v rows).

#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kBatch = 2;  // heads a thread loads at a time

// A unit is 16 values of a row: two 16-byte vectors that hold 8 whole pairs
// (or 16 values past rot_dim).  Thread: unit u of token tt, heads hg, hg + HG, ...
template <int D, int TOK, int TO>
__global__ void __launch_bounds__(kThreads, 4) fa_turn_kernel(const __grid_constant__ TurnParams p) {
  constexpr int UNITS = D / 16;
  constexpr int HG = kThreads / (UNITS * TOK);
  static_assert(HG >= 1, "threads");
  __shared__ __align__(16) float2 cs[TOK][kMaxPairs];
  __shared__ uint64_t fraction[kMaxPairs];
  __shared__ long long place[TOK];  // cache offset of the token's row in head 0; -1: not stored
  __shared__ int seq_pos[TOK];      // place in the sequence; INT_MIN: no sequence

  grid_launch_dependents();
  grid_dependency_wait();

  const int tid = threadIdx.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * TOK;
  const int half = p.half;
  const int u = tid % UNITS, tt = tid / UNITS % TOK, hg = tid / (UNITS * TOK);
  const long long t = t0 + tt;
  const bool here = hg < HG && t < p.tokens;
  // (fewer than 2^31 positions in all)
  const long long b = TO == kTurnOnly ? static_cast<uint32_t>(t) / static_cast<uint32_t>(p.N) : 0;
  const long long n = t - b * p.N;
  // The unit's first vector and the distance to its second, in elements.
  const bool turned = u < half / 8;
  const int first = p.interleaved ? 16 * u : turned ? 8 * u : 2 * half + 16 * (u - half / 8);
  const int gap = p.interleaved || !turned ? 8 : half;
  // First row of each tensor for this thread, and the step to its next head.
  const __nv_bfloat16* q_in = p.q.in + (b * p.q.ib + n * p.q.ip + hg * p.q.ih + first);
  const __nv_bfloat16* k_in = p.k.in + (b * p.k.ib + n * p.k.ip + hg * p.k.ih + first);
  uint4 lo[kBatch], hi[kBatch];
  auto load = [&](const __nv_bfloat16* src, long long step, int left) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i * HG < left) {
        lo[i] = *reinterpret_cast<const uint4*>(src + i * step);
        hi[i] = *reinterpret_cast<const uint4*>(src + i * step + gap);
      }
    }
  };
  const long long q_step = p.q.ih * HG, k_step = p.k.ih * HG;
  if (here) load(q_in, q_step, p.q.heads - hg);

  if constexpr (TO != kTurnOnly) find_tokens(p, t0, TOK, place, seq_pos);
  // (fp64 is slow here: once a pair, not once an angle)
  if (tid < half) fraction[tid] = turn_fraction(p.inv_freq[tid]);
  __syncthreads();
  for (int i = tid; i < TOK * half; i += kThreads) {
    const int w = i / half, pair = i - w * half;
    const long long tw = t0 + w;
    if (tw >= p.tokens) break;
    int pos = TO == kTurnOnly ? 0 : seq_pos[w];
    if (p.positions) {
      const long long bw =
          TO == kTurnOnly ? static_cast<uint32_t>(tw) / static_cast<uint32_t>(p.N) : 0;
      pos = p.positions[p.axis[pair] * p.axis_stride + bw * p.batch_stride + (tw - bw * p.N)];
    }
    cs[w][pair] = cos_sin(pos, fraction[pair], p.sign);
  }
  __syncthreads();
  if (!here || (TO != kTurnOnly && seq_pos[tt] == INT_MIN)) return;

  float2 t8[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = *reinterpret_cast<const float4*>(&cs[tt][turned ? 8 * u + 2 * e : 0]);
    t8[2 * e] = make_float2(v.x, v.y);
    t8[2 * e + 1] = make_float2(v.z, v.w);
  }
  auto turn = [&](float (&x)[8], float (&y)[8]) {
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
        x[2 * e] = x0 * t8[e].x - x1 * t8[e].y;
        x[2 * e + 1] = x0 * t8[e].y + x1 * t8[e].x;
        y[2 * e] = y0 * t8[e + 4].x - y1 * t8[e + 4].y;
        y[2 * e + 1] = y0 * t8[e + 4].y + y1 * t8[e + 4].x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = x[e], y0 = y[e];
        x[e] = x0 * t8[e].x - y0 * t8[e].y;
        y[e] = x0 * t8[e].y + y0 * t8[e].x;
      }
    }
  };
  // A loaded row to a bf16 row at dst, or to an e4m3 row times `scale`.
  auto put = [&](const uint4& lo, const uint4& hi, auto* dst, bool turns, float scale) {
    if (sizeof(*dst) == 2 && !turns) {
      *reinterpret_cast<uint4*>(dst) = lo;
      *reinterpret_cast<uint4*>(dst + gap) = hi;
      return;
    }
    float x[8], y[8];
    unpack8(lo, x);
    unpack8(hi, y);
    if (turns) turn(x, y);
    if constexpr (sizeof(*dst) == 2) {
      *reinterpret_cast<uint4*>(dst) = pack8(x);
      *reinterpret_cast<uint4*>(dst + gap) = pack8(y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= scale;
        y[e] *= scale;
      }
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
      *reinterpret_cast<uint2*>(dst + gap) =
          make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
    }
  };
  // The heads hg, hg + HG, ... of one tensor, the first kBatch in lo and hi.
  auto rows = [&](const __nv_bfloat16* src, long long step, int heads, __nv_bfloat16* dst,
                  long long dst_step) {
    for (int left = heads - hg; left > 0;) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i * HG < left) put(lo[i], hi[i], dst + i * dst_step, turned, 1.0f);
      src += kBatch * step;
      dst += kBatch * dst_step;
      left -= kBatch * HG;
      load(src, step, left);
    }
  };
  rows(q_in, q_step, p.q.heads,
       p.q.out + (b * p.q.ob + n * p.q.op + hg * p.q.oh + first), p.q.oh * HG);
  if constexpr (TO == kTurnOnly) {
    load(k_in, k_step, p.k.heads - hg);
    rows(k_in, k_step, p.k.heads,
         p.k.out + (b * p.k.ob + n * p.k.op + hg * p.k.oh + first), p.k.oh * HG);
  } else {
    if (place[tt] < 0) return;
    using Elem = std::conditional_t<TO == kToBf16, __nv_bfloat16, uint8_t>;
    const long long off = place[tt] + hg * p.head_stride + first;
    const __nv_bfloat16* v_in = p.v.in + (n * p.v.ip + hg * p.v.ih + first);
    Elem* k_out = static_cast<Elem*>(p.k_pages) + off;
    Elem* v_out = static_cast<Elem*>(p.v_pages) + off;
    for (int h = hg; h < p.k.heads; h += HG) {  // a head's k and v together
      const uint4 k0 = *reinterpret_cast<const uint4*>(k_in);
      const uint4 k1 = *reinterpret_cast<const uint4*>(k_in + gap);
      const uint4 v0 = *reinterpret_cast<const uint4*>(v_in);
      const uint4 v1 = *reinterpret_cast<const uint4*>(v_in + gap);
      put(k0, k1, k_out, turned, p.k_scale);
      put(v0, v1, v_out, false, p.v_scale);
      k_in += k_step;
      v_in += p.v.ih * HG;
      k_out += p.head_stride * HG;
      v_out += p.head_stride * HG;
    }
  }
}

template <int D, int TO>
cudaError_t launch_turn_d(const TurnParams& p, cudaStream_t stream) {
  const int heads = p.q.heads + p.k.heads + p.v.heads;
  const long long sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  // The most positions a block that leave a block for every SM and a thread at
  // most ten heads: the angles' cost is shared, and a short loop ends evenly.
  // Measured with 1 / 4 / 8 / 16: 8192 positions of 16 heads, d = 64: 38 / 14.5 /
  // 10.1 / 8.7 us; 16384 of 40, d = 128: 107 / 54.6 / 55.7 / 57.9; 1025 of 32, d =
  // 96: 6.3 / 4.5 / 4.9 / 7.2; 4 of 48, d = 128: 4.0 / 4.8 / 5.8 / 8.5.
  int tok = 1;
  for (int more : {4, 8, 16})
    if (p.tokens >= sms * more && heads * (D / 16) * more <= 10 * kThreads) tok = more;
  const long long grid = (p.tokens + tok - 1) / tok;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = tok == 1 ? fa_turn_kernel<D, 1, TO>
              : tok == 4 ? fa_turn_kernel<D, 4, TO>
              : tok == 8 ? fa_turn_kernel<D, 8, TO>
                         : fa_turn_kernel<D, 16, TO>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, p);
}

template <int TO>
cudaError_t launch_turn(const TurnParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_turn_d<64, TO>(p, stream);
    case 96: return launch_turn_d<96, TO>(p, stream);
    case 128: return launch_turn_d<128, TO>(p, stream);
    case 256: return launch_turn_d<256, TO>(p, stream);
  }
  return cudaErrorInvalidValue;
}

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
