// Rotary positions with several axes, and appending a step's keys and values
// to a paged cache with the turn applied on the way.
//
// A pair (x_i, x_j) of a head row is turned by a = position * f:
//     y_i = x_i cos a - x_j sin a,   y_j = x_i sin a + x_j cos a,
// and the gradient is the turn by -a (the turn is orthogonal).
//
// Angle.  Only a mod one turn matters.  f / 2 pi becomes a 64-bit fraction of a
// turn F, from a double product (off by 2^-52 relative), and position * F wraps
// modulo 2^64, which is exact: at position 2^20 and f = 1 it is off by 2^-34 of a
// turn, where position * f in fp32 would be off by 2^-5 radians.  The top 32 bits,
// as a signed fraction in [-1/2, 1/2), go through fp32 to sincospif: 2^-32 of a
// turn for the cut and 2^-26 for fp32, at any position, which is the larger part
// up to position 2^28 (the product's is 2^-23.6 at 2^31).
//
// The kernels are in fa_rotary.cu, and with the heads' norms in fa_norm.cu.

#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "fa_internal.h"
#include "fa_paged_host.h"
#include "fa_ptx.cuh"

namespace fa {

constexpr int kMaxPairs = 128;  // rot_dim / 2 at d = 256

struct TurnRows {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  long long ib, ih, ip, ob, oh, op;  // strides: batch, head, position
  int heads;
};

struct TurnParams {
  TurnRows q, k, v;  // v: appending only
  int N;         // positions per batch entry
  long long tokens;
  const int* positions;  // nullptr: the token's place in its sequence
  long long axis_stride, batch_stride;
  const float* inv_freq;
  int half;         // pairs turned, rot_dim / 2
  int interleaved;
  float sign;       // -1 for the gradient
  alignas(4) unsigned char axis[kMaxPairs];
  // norms of the heads' rows before they are turned
  const void* q_weight;  // [d], nullptr: ones
  const void* k_weight;
  int weight_bf16;
  float eps;
  // appending: the cache and the batch
  const int* q_start;
  const int* kv_len;
  const int* table;
  long long table_stride;
  int S, max_pages, page_size, n_pages;
  long long page_stride, row_stride, head_stride;
  void* k_pages;
  void* v_pages;
  float k_scale, v_scale;  // 1 / descale
  uint32_t* err;
};

// Checks, and what they fill in (fa_rotary.cu).
bool good_spec(const fa_rotary_spec& r, int d);
void put_spec(TurnParams& p, const fa_rotary_spec& r);
// q and k (nullptr: none) at their positions; spec nullptr: nothing is turned.
fa_status put_turn(TurnParams& p, const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N,
                   int d, const int* positions, long long axis_stride, long long batch_stride,
                   const fa_rotary_spec* spec, float sign);
// A step's rows on their way into the cache.  *nothing: there is nothing to do (FA_OK).
fa_status put_append(TurnParams& p, const fa_paged_cache* cache, const fa_paged_batch* batch,
                     const void* k, long long k_token, long long k_head, const void* v,
                     long long v_token, long long v_head, int T, const void* q, long long q_token,
                     long long q_head, void* q_out, long long qo_token, long long qo_head, int H_q,
                     const fa_rotary_spec* spec, const int* positions, long long axis_stride,
                     bool* nothing);

namespace {

constexpr int kThreads = 256;

enum { kTurnOnly = 0, kToBf16 = 1, kToE4m3 = 2 };  // where k (and v) rows go

// f / 2 pi modulo one turn, as a 64-bit fraction.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const double t = static_cast<double>(f) * 0.15915494309189535;  // 1 / (2 pi)
  return static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ float2 cos_sin(int position, uint64_t fraction, float sign) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<long long>(position)) * fraction;
  const int top = static_cast<int>(static_cast<uint32_t>(turns >> 32));
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c, sign * s);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// The tokens t0 .. t0 + tok - 1 of a step: each one's place in its sequence (INT_MIN: it has
// none), and the cache offset of its row in head 0 (-1: not stored).  The whole block calls
// this, a barrier after it.
__device__ __forceinline__ void find_tokens(const TurnParams& p, long long t0, int tok,
                                            long long* place, int* seq_pos) {
  const int tid = threadIdx.x;
  // Warp w finds token w (tok / 8 rounds): its sequence is the number of
  // starts q_start[1..S] at or below it, counted by all lanes.  Up to 32
  // sequences, each lane brings its sequence's end and length with that.
  const int lane = tid & 31;
  for (int w = tid >> 5; w < tok; w += kThreads / 32) {
    const long long tw = t0 + w;
    int s, from, to, len;  // the sequence, its first token, its end, its length
    if (p.S <= 32) {
      const int end = lane < p.S ? p.q_start[lane + 1] : 0;
      const int kv = lane < p.S ? p.kv_len[lane] : 0;
      const int start = p.q_start[0];
      s = __popc(__ballot_sync(0xffffffffu, lane < p.S && end <= tw));
      to = __shfl_sync(0xffffffffu, end, s & 31);
      len = __shfl_sync(0xffffffffu, kv, s & 31);
      from = __shfl_sync(0xffffffffu, end, (s - 1) & 31);
      if (s == 0) from = start;
    } else {
      int below = 0;
      for (int i = lane; i < p.S; i += 32) below += p.q_start[i + 1] <= tw;
      s = __reduce_add_sync(0xffffffffu, below);
      const int x = min(s, p.S - 1);
      from = p.q_start[x];
      to = p.q_start[x + 1];
      len = p.kv_len[x];
    }
    if (lane == 0) {
      int pos = INT_MIN;
      long long where = -1;
      if (tw < p.tokens && s < p.S && tw >= from) {
        pos = static_cast<int>(len - (to - tw));
        const int slot = pos < 0 ? 0 : pos / p.page_size;
        if (pos >= 0 && slot < p.max_pages) {
          const int page = p.table[s * p.table_stride + slot];
          if (page >= 0 && page < p.n_pages)
            where = page * p.page_stride + (pos - slot * p.page_size) * p.row_stride;
          else
            atomicOr(p.err, kErrBadPage);
        } else if (pos >= 0) {
          atomicOr(p.err, kErrBadPage);
        }
      }
      place[w] = where;
      seq_pos[w] = pos;
    }
  }
}

}  // namespace
}  // namespace fa
