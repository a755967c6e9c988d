// Shared by the kernels of fa_forward_scores, fa_backward_scores and
// fa_forward_paged_scores: what is done to a score between Q K^T and the softmax,
// and which keys a query row sees.
//
//   x = scale q.k;   x = softcap tanh(x / softcap);   x = x - slope_h |pos - j|
//
// and row i, at position pos = q_offset + i, sees the keys of one span
//   [max(first_i, pos - window + 1, 0), min(end_i, pos + 1 if causal, N_kv)),
// so a row's mask is two integers that its thread keeps in registers, a tile needs
// no mask at all where every row's span covers it, and tiles outside the union of the
// rows' spans are never visited.
//
// Everything after Q K^T is in the log2 domain (factors of log2(e) are folded in on
// the host).  The tanh: for |y| <= 0.4, y = x / softcap, as y P(y^2) with P of degree 3,
// fitted here for the least largest relative error, 9.8e-8; with the roundings of its argument, of
// cap2 and of the coefficients (4.6 x 2^-24 together) and of the last two steps under 5.2e-7.
// Its coefficients take in scale / softcap and softcap log2(e) (score_factors), which leaves five
// operations on the FMA pipe in place of the one that scales a score, where one ex2 and one rcp
// more for each score would take the special-function unit longer than the weights' own
// exponentials.  A warp with a score beyond goes by tanh y = 1 - 2 / (e^{2y} + 1), which holds
// everywhere, to 5.5e-7 of the cap (rcp 2^-23 and the sum's 2^-24 of a quotient up to 2, the
// exponent's 2^-22 and its argument's 2.1e-7 by what tanh makes of them, half of 1 - tanh^2 and y
// (1 - tanh^2); 2^-24 at the end and of cap2).  (16 heads of 8192, d = 64, causal: dQ takes 381 us
// if all go that way.)  Caps of many thousands, whose folded coefficients would leave fp32's range,
// choose between the two score by score: there 5.5e-7 of the cap is more than a score.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "fa_ptx.cuh"
#include "fa_scores_host.h"

namespace fa {

constexpr float kScoreLog2e = 1.4426950408889634f;
constexpr float kScoreLn2 = 0.6931471805599453f;

struct KeySpan {
  int lo, hi;  // keys [lo, hi); 0, 0 for a row that sees none
};

__device__ __forceinline__ KeySpan row_span(const ScoreParams& p, int b, int i) {
  KeySpan s{0, 0};
  if (i >= p.Nq) return s;
  const long long at = b * p.span_batch + i;
  const int pos = p.q_offset + i;
  s.hi = p.Nk;
  if (p.first) s.lo = max(p.first[at], 0);
  if (p.end) s.hi = min(p.end[at], p.Nk);
  if (p.window > 0) s.lo = max(s.lo, pos - p.window + 1);
  if (p.causal) s.hi = min(s.hi, pos + 1);
  if (s.lo >= s.hi) s.lo = s.hi = 0;
  return s;
}

// The union of the spans of the warp's rows, as [lo, hi); lo = INT_MAX, hi = 0 if all are empty.
__device__ __forceinline__ KeySpan warp_hull(const KeySpan& s) {
  KeySpan h;
  h.lo = __reduce_min_sync(0xffffffffu, s.hi > s.lo ? s.lo : INT_MAX);
  h.hi = __reduce_max_sync(0xffffffffu, s.hi);
  return h;
}

// Largest magnitude of three.
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What N columns' exponents get besides their scores, in pairs: -sub, and BIAS less
// slope2 |dist0 - t|.  ONE: dist0 - t has the sign `side` (or is 0) at all N, so that this is
// linear in t: two FMAs for eight columns and an addition a pair (the distances one by one take
// four operations a pair: 16 heads of 8192, d = 64, forward 232 us instead of 219, both passes 773
// instead of 737).
template <int N, bool BIAS, bool ONE>
struct Lowering {
  float slope2, dist0, sub, k, base;
  uint64_t step[3], at;
  __device__ __forceinline__ Lowering(float slope2_, float dist0_, float sub_, float side)
      : slope2(slope2_), dist0(dist0_), sub(sub_) {
    if constexpr (!BIAS) {
      at = f2_pack(-sub, -sub);
    } else if constexpr (ONE) {
      k = side * slope2;
      base = fmaf(-k, dist0, -sub);
#pragma unroll
      for (int i = 0; i < 3; ++i) step[i] = f2_pack((2 * i + 2) * k, (2 * i + 2) * k);
    }
  }
  // Of columns t, t + 1, in order.
  __device__ __forceinline__ uint64_t pair(int t) {
    if constexpr (!BIAS) return at;
    if constexpr (ONE) {
      if (t % 8 == 0) {
        at = f2_pack(fmaf(k, static_cast<float>(t), base), fmaf(k, static_cast<float>(t + 1), base));
        return at;
      }
      return f2_add(at, step[t % 8 / 2 - 1]);
    }
    return f2_pack(fmaf(-slope2, fabsf(dist0 - static_cast<float>(t)), -sub),
                   fmaf(-slope2, fabsf(dist0 - static_cast<float>(t + 1)), -sub));
  }
};

// Scores of keys kbase + t less slope2 |pos - key|, dist0 = pos - kbase (distances are whole
// numbers, exact in fp32 up to 2^24).  The whole warp calls this.
template <int N>
__device__ __forceinline__ void lower_scores(float (&s)[N], float slope2, float dist0) {
  const bool before = __all_sync(0xffffffffu, dist0 >= static_cast<float>(N - 1));
  const bool after = __all_sync(0xffffffffu, dist0 <= 0.0f);
  if (before || after) {
    Lowering<N, true, true> low(slope2, dist0, 0.0f, before ? 1.0f : -1.0f);
#pragma unroll
    for (int t = 0; t < N; t += 2)
      f2_unpack(f2_add(f2_pack(s[t], s[t + 1]), low.pair(t)), s[t], s[t + 1]);
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t) s[t] = fmaf(-slope2, fabsf(dist0 - static_cast<float>(t)), s[t]);
  }
}

// shape_scores where it is known whether dist0 - t has one sign (Lowering).
template <int N, bool CAP, bool BIAS, bool GRAD, bool FOLDS, bool ONE, typename Again>
__device__ __forceinline__ void shape_columns(float (&s)[N], float (&g)[GRAD ? N : 1],
                                              const ScoreFactors& f, float slope2, float dist0,
                                              float sub, float side, Again&& again) {
  Lowering<N, BIAS, ONE> low(slope2, dist0, sub, side);
  if constexpr (CAP) {
    constexpr int CHAINS = N < 16 ? 1 : 2;  // independent maxima
    float part[CHAINS];
#pragma unroll
    for (int u = 0; u < CHAINS; ++u) part[u] = 0.0f;
    const uint64_t a0 = f2_pack(f.a[0], f.a[0]), a1 = f2_pack(f.a[1], f.a[1]);
    const uint64_t a2 = f2_pack(f.a[2], f.a[2]), a3 = f2_pack(f.a[3], f.a[3]);
    const uint64_t one = f2_pack(1.0f, 1.0f), nz = f2_pack(f.neg_inv_cap_sq, f.neg_inv_cap_sq);
#pragma unroll
    for (int t = 0; t < N; t += 2) {
      part[t / 2 % CHAINS] = fmax3_abs(part[t / 2 % CHAINS], s[t], s[t + 1]);
      const uint64_t v = f2_pack(s[t], s[t + 1]);
      const uint64_t v2 = f2_mul(v, v);
      const uint64_t h = f2_fma(f2_fma(f2_fma(a3, v2, a2), v2, a1), v2, a0);
      if constexpr (GRAD) {
        const uint64_t x = f2_mul(v, h);
        f2_unpack(f2_add(x, low.pair(t)), s[t], s[t + 1]);
        f2_unpack(f2_fma(f2_mul(x, x), nz, one), g[t], g[t + 1]);
      } else {
        f2_unpack(f2_fma(v, h, low.pair(t)), s[t], s[t + 1]);
      }
    }
    float big = part[0];
#pragma unroll
    for (int u = 1; u < CHAINS; ++u) big = fmaxf(big, part[u]);
    // (a NaN takes either way to a NaN)
    if (__any_sync(0xffffffffu, big > f.range)) {
      Lowering<N, BIAS, ONE> more(slope2, dist0, sub, side);
      constexpr int P = N < 32 ? N : 32;  // columns put back at a time
#pragma unroll
      for (int c0 = 0; c0 < N; c0 += P) {
        float(&y)[P] = *reinterpret_cast<float(*)[P]>(&s[c0]);
        again(y, c0);
        if (FOLDS && f.range < 0.0f) {
          // Scores one by one: within the polynomial's reach by it (the other way is off by as
          // much of a large cap, more than the scores themselves).
#pragma unroll
          for (int t = 0; t < P; t += 2) {
            float lower[2];
            f2_unpack(more.pair(c0 + t), lower[0], lower[1]);
#pragma unroll
            for (int e = t; e < t + 2; ++e) {
              const float z = y[e] * f.k, z2 = z * z;
              const float h =
                  z * fmaf(fmaf(fmaf(kTanhC3, z2, kTanhC2), z2, kTanhC1), z2, kTanhC0);
              const float r = rcp_approx(ex2_approx(z * (2.0f * kScoreLog2e)) + 1.0f);
              const bool near = fabsf(z) <= kTanhRange;
              y[e] = (near ? f.cap2 * h : fmaf(-2.0f * f.cap2, r, f.cap2)) + lower[e - t];
              if constexpr (GRAD) g[c0 + e] = near ? fmaf(-h, h, 1.0f) : 4.0f * r * (1.0f - r);
            }
          }
        } else {
#pragma unroll
          for (int t = 0; t < P; t += 2) {
            float lower[2];
            f2_unpack(more.pair(c0 + t), lower[0], lower[1]);
#pragma unroll
            for (int e = t; e < t + 2; ++e) {
              const float r = rcp_approx(ex2_approx(y[e] * (2.0f * kScoreLog2e * f.k)) + 1.0f);
              y[e] = fmaf(-2.0f * f.cap2, r, f.cap2) + lower[e - t];
              if constexpr (GRAD) g[c0 + e] = 4.0f * r * (1.0f - r);
            }
          }
        }
      }
    }
  } else {
    const uint64_t c = f2_pack(f.k, f.k);
#pragma unroll
    for (int t = 0; t < N; t += 2)
      f2_unpack(f2_fma(f2_pack(s[t], s[t + 1]), c, low.pair(t)), s[t], s[t + 1]);
  }
}

// What turns raw products s = q.k of keys kbase + t, t = 0 .. N-1, into exponents of the
// weights, x (log2 domain), less `sub`:  CAP x = cap tanh(s k) (in f), else x = s f.k;
// BIAS then - slope2 |pos - key|, dist0 = pos - kbase.  With GRAD, g gets 1 - tanh^2.  The
// whole warp calls this (f may differ between its lanes).  `again` puts the products of columns
// from c0 on into its argument once more, for the warp that finds only after the polynomial that
// it did not hold (to look first would have all of the arithmetic wait for all of the maxima: 5 %
// of dQ).  FOLDS: the coefficients take in factors, and may not hold it at all.
template <int N, bool CAP, bool BIAS, bool GRAD, bool FOLDS = true, typename Again>
__device__ __forceinline__ void shape_scores(float (&s)[N], float (&g)[GRAD ? N : 1],
                                             const ScoreFactors& f, float slope2, float dist0,
                                             float sub, Again&& again) {
  if constexpr (BIAS) {
    const bool before = __all_sync(0xffffffffu, dist0 >= static_cast<float>(N - 1));
    const bool after = __all_sync(0xffffffffu, dist0 <= 0.0f);
    if (before || after)
      shape_columns<N, CAP, BIAS, GRAD, FOLDS, true>(s, g, f, slope2, dist0, sub,
                                                     before ? 1.0f : -1.0f, again);
    else
      shape_columns<N, CAP, BIAS, GRAD, FOLDS, false>(s, g, f, slope2, dist0, sub, 0.0f, again);
  } else {
    shape_columns<N, CAP, false, GRAD, FOLDS, false>(s, g, f, slope2, dist0, sub, 0.0f, again);
  }
}

// TMEM -> registers, 16 or 32 consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 16)
    tmem_ld16(taddr, r);
  else
    tmem_ld32(taddr, r);
}

// N products out of TMEM; the whole warp calls this.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&s)[N]) {
  uint32_t r[N];
  tmem_ld<N>(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int t = 0; t < N; ++t) s[t] = __uint_as_float(r[t]);
}

// Byte offset of 16-byte chunk `ch` of row `r` in a 128-byte-swizzled block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int r, int ch) {
  return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// First query tile whose rows' spans touch keys [k0, k0 + width), and one past the last, into
// range[0] and range[1] (INT_MAX and 0 before).  The whole block calls this, a barrier before
// and after it.
template <int THREADS>
__device__ __forceinline__ void seen_by(const int2* tiles, int n, int k0, int width, int* range) {
  int from = INT_MAX, to = 0;
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const int2 t = tiles[i];
    if (t.y > k0 && t.x < k0 + width) {
      from = min(from, i);
      to = i + 1;
    }
  }
  from = __reduce_min_sync(0xffffffffu, from);
  to = __reduce_max_sync(0xffffffffu, to);
  if ((threadIdx.x & 31) == 0 && to > 0) {
    atomicMin(&range[0], from);
    atomicMax(&range[1], to);
  }
}

}  // namespace fa
