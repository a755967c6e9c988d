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
  unsigned char axis[kMaxPairs];
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
constexpr int kBatch = 2;       // heads a thread loads at a time

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

// 8 weights of a norm from element `at`, in fp32.
__device__ __forceinline__ void load_weights(const void* w, int bf16, int at, float (&x)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.0f;
  } else if (bf16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at), x);
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// Sum over the LANES lanes (a power of two, aligned) that share a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
  const unsigned lane = lane_id();
  const unsigned mask =
      LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (lane & ~(LANES - 1u));
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) x += __shfl_xor_sync(mask, x, d);
  return x;
}

// Lanes of a row: D / 16 units, rounded up to a power of two where the row is summed (two of
// eight lanes idle at d = 96).
__host__ __device__ constexpr int row_lanes(int d, bool norm) { return norm && d == 96 ? 8 : d / 16; }

// A unit is 16 values of a row: two 16-byte vectors that hold 8 whole pairs
// (or 16 values past rot_dim).  Thread: unit u of token tt, heads hg, hg + HG, ...
//
// NORM: a row x of q or k becomes x / sqrt(mean x^2 + eps) times its weights before it is
// turned, in fp32 up to the one rounding at the end.  The lanes of a row sum its squares by
// shuffles among themselves (other rows of the warp may have ended); bound by memory as the
// turn alone is, with the weights in registers.
template <int D, int TOK, int TO, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 3 : 4)
    fa_turn_kernel(const __grid_constant__ TurnParams p) {
  constexpr int UNITS = row_lanes(D, NORM);
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
  // (lanes without values stay for their row's sum, with zeros)
  const bool lane_on = UNITS * 16 == D || u < D / 16;
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
      if (i * HG < left && lane_on) {
        lo[i] = *reinterpret_cast<const uint4*>(src + i * step);
        hi[i] = *reinterpret_cast<const uint4*>(src + i * step + gap);
      } else if (UNITS * 16 != D) {
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  const long long q_step = p.q.ih * HG, k_step = p.k.ih * HG;
  if (here) load(q_in, q_step, p.q.heads - hg);

  if (TO != kTurnOnly) {
    // Warp w finds token w (TOK / 8 rounds): its sequence is the number of
    // starts q_start[1..S] at or below it, counted by all lanes.  Up to 32
    // sequences, each lane brings its sequence's end and length with that.
    const int lane = tid & 31;
    for (int w = tid >> 5; w < TOK; w += kThreads / 32) {
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
    const float4 v = *reinterpret_cast<const float4*>(&cs[tt][turned && lane_on ? 8 * u + 2 * e : 0]);
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
  // The weights of this unit's values.
  float wx[NORM ? 8 : 1], wy[NORM ? 8 : 1];
  auto weights = [&](const void* w) {
    if constexpr (NORM) {
      load_weights(lane_on ? w : nullptr, p.weight_bf16, first, wx);
      load_weights(lane_on ? w : nullptr, p.weight_bf16, first + gap, wy);
    }
  };
  // A loaded row to a bf16 row at dst, or to an e4m3 row times `scale`.
  auto put = [&](const uint4& lo, const uint4& hi, auto* dst, bool turns, bool norms,
                 float scale) {
    if (sizeof(*dst) == 2 && !turns && !(NORM && norms)) {
      if (!lane_on) return;
      *reinterpret_cast<uint4*>(dst) = lo;
      *reinterpret_cast<uint4*>(dst + gap) = hi;
      return;
    }
    float x[8], y[8];
    unpack8(lo, x);
    unpack8(hi, y);
    if constexpr (NORM) {
      if (norms) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
        const float r = rsqrtf(row_sum<UNITS>(ss) * (1.0f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r * wx[e];
          y[e] *= r * wy[e];
        }
      }
    }
    if (!lane_on) return;
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
        if (i * HG < left) put(lo[i], hi[i], dst + i * dst_step, turned, true, 1.0f);
      src += kBatch * step;
      dst += kBatch * dst_step;
      left -= kBatch * HG;
      load(src, step, left);
    }
  };
  weights(p.q_weight);
  rows(q_in, q_step, p.q.heads,
       p.q.out + (b * p.q.ob + n * p.q.op + hg * p.q.oh + first), p.q.oh * HG);
  weights(p.k_weight);
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
      uint4 k0{}, k1{}, v0{}, v1{};
      if (lane_on) {
        k0 = *reinterpret_cast<const uint4*>(k_in);
        k1 = *reinterpret_cast<const uint4*>(k_in + gap);
        v0 = *reinterpret_cast<const uint4*>(v_in);
        v1 = *reinterpret_cast<const uint4*>(v_in + gap);
      }
      put(k0, k1, k_out, turned, true, p.k_scale);
      put(v0, v1, v_out, false, false, p.v_scale);
      k_in += k_step;
      v_in += p.v.ih * HG;
      k_out += p.head_stride * HG;
      v_out += p.head_stride * HG;
    }
  }
}

template <int D, int TO, bool NORM>
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
  auto kern = tok == 1 ? fa_turn_kernel<D, 1, TO, NORM>
              : tok == 4 ? fa_turn_kernel<D, 4, TO, NORM>
              : tok == 8 ? fa_turn_kernel<D, 8, TO, NORM>
                         : fa_turn_kernel<D, 16, TO, NORM>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, p);
}

template <int TO, bool NORM = false>
cudaError_t launch_turn(const TurnParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_turn_d<64, TO, NORM>(p, stream);
    case 96: return launch_turn_d<96, TO, NORM>(p, stream);
    case 128: return launch_turn_d<128, TO, NORM>(p, stream);
    case 256: return launch_turn_d<256, TO, NORM>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace fa
