// Forward of attention with shaped scores (fa_scores.cuh says how), one 128-row query tile
// a CTA, head dimensions 64, 96, 128 and 256.
//
// The online softmax of fa_fwd_tile1.cu: S_j = Q K_j^T goes to tensor-memory buffer j mod 3,
// the softmax warpgroup (a query row a thread) makes P_j of it over the same columns, and
// O += P_j V_j reads it there; the issuer runs two key tiles ahead.  Key tiles are those
// that the union of the rows' spans touches, counted from its first.
//
// A capped score cannot pass softcap, so with no distance term the reference that the
// online softmax subtracts is fixed, at 0, as long as weights and their sums then stay within
// fp32's (and bf16's) exponents: no running maximum and no rescaling of O.  For softcap log2(e) <=
// kFixedCap the weights lie in [2^-kFixedCap, 2^kFixedCap], in the middle of the exponents: a row
// at either end of the cap has its v whole down to 2^-46 and up to 2^47 over its keys (with half
// the cap as the reference, v of 2^-18 was cut at the lower end).  A row's 128 keys of a tile then
// go to four warps, 32 each (16 heads of 8192, cap, d = 64 / 96 / 128: 201 / 219 / 228 us with
// four, 218 / 229 / 234 with two, 231 / 243 / 249 with one; two tiles a CTA 205 / 227 / 284).  With
// a moving reference, warps that share a row have to exchange maxima each tile, and wait for one
// another: slower with two or four than with one.
//
// Bound by the softmax's instructions: 55 % of the issue slots with a cap; 33 % without, where one
// warp a scheduler waits for its own results (d = 128, uncapped: 205 us, 1.34 PFLOP/s).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;

template <int D_, bool FIXED>
struct ScoreFwdCfg {
  static constexpr int D = D_;
  static constexpr int DP = (D + 63) / 64 * 64;  // tiles are whole 128-byte swizzle atoms wide
  static constexpr int BM = 128;
  static constexpr int BN = D == 256 ? 64 : 128;
  static constexpr int KH = FIXED ? 32 : BN;     // key columns of a softmax warp
  static constexpr int GROUPS = BN / KH;         // softmax warps that share a row
  static constexpr int WARPS = 4 * GROUPS;       // softmax warps; then TMA and MMA
  static constexpr int SUB = DP / 64;
  static constexpr int Q_BLOCK = BM * 128;
  static constexpr int KV_BLOCK = BN * 128;
  static constexpr int Q_TILE = SUB * Q_BLOCK;
  static constexpr int KV_TILE = SUB * KV_BLOCK;
  static constexpr int NS = D == 64 ? 4 : 2;     // K/V ring stages
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_TILE;
  static constexpr int OFF_V = OFF_K + NS * KV_TILE;
  static constexpr int OFF_BAR = OFF_V + NS * KV_TILE;
  static constexpr int B_QFULL = 0;
  static constexpr int B_KFULL = 1;
  static constexpr int B_KEMPTY = B_KFULL + NS;
  static constexpr int B_VFULL = B_KEMPTY + NS;
  static constexpr int B_VEMPTY = B_VFULL + NS;
  static constexpr int NB = 3;                   // S/P buffers
  static constexpr int B_SFULL = B_VEMPTY + NS;  // [NB] S_j in buffer j % NB
  static constexpr int B_PFULL = B_SFULL + NB;   // [NB] P_j there (every softmax warp)
  static constexpr int B_ODONE = B_PFULL + NB;   // O += P_j V_j completed
  static constexpr int B_FINAL = B_ODONE + 1;    // every product completed (once)
  static constexpr int B_SUM = B_FINAL + 1;      // the parts of l in shared memory (once)
  static constexpr int B_DRAIN = B_SUM + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;  // tmem slot, abort word, 4 warps' hulls
  static constexpr int OFF_SUM = OFF_MISC + 8 + 32;    // [GROUPS][BM] parts of l
  static constexpr int SMEM_BYTES = OFF_SUM + (GROUPS > 1 ? GROUPS * BM * 4 : 0) + 1024;
  static constexpr int THREADS = 32 * WARPS + 64;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 512 - DP;
  static_assert(NB * BN <= 512 - DP, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct ScoreFwdParams {
  ScoreParams s;
  __nv_bfloat16* o;
  float* lse;
  int n_qtiles, n_heads, heads_per_group;
};

// The scores of a row's key tile (BN keys from kbase on) at TMEM address `s_addr` to P over
// them, with the running reference m and sum l (log2 domain); keys outside `span` get 0 where
// `mask`.  Returns the factor that O and the old l are due (1 unless `moved`).  FIXED: m is
// the reference, 0, and stays.  The whole warp calls this.
template <int BN, bool CAP, bool BIAS, bool FIXED>
__device__ __forceinline__ float score_row(const ScoreParams& p, uint32_t s_addr, bool mask,
                                           const KeySpan& span, int kbase, int pos, float slope2,
                                           float& m, float& l, bool& moved) {
  const unsigned from = static_cast<unsigned>(span.lo - kbase);
  const unsigned len = static_cast<unsigned>(span.hi - span.lo);
  uint64_t ps2[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) ps2[u] = 0ull;
  float alpha = 1.0f;
  // Products of columns from c0 on.
  auto load = [&](auto& x, int c0) {
    constexpr int N = sizeof(x) / sizeof(float);
    uint32_t r[N];
#pragma unroll
    for (int c = 0; c < N / 32; ++c)
      tmem_ld32(s_addr + c0 + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
    tmem_wait_ld();
#pragma unroll
    for (int t = 0; t < N; ++t) x[t] = __uint_as_float(r[t]);
  };
  if constexpr (FIXED) {
    float x[BN], none[1];
    load(x, 0);
    shape_scores<BN, CAP, BIAS, false>(x, none, p.f, slope2,
                                       static_cast<float>(pos - kbase), m, load);
    if (mask) {
#pragma unroll
      for (int t = 0; t < BN; ++t)
        if (static_cast<unsigned>(t) - from >= len) x[t] = -INFINITY;
    }
    uint32_t pk[BN / 2];
#pragma unroll
    for (int t = 0; t < BN / 2; ++t) {
      const float p0 = ex2_approx(x[2 * t]);
      const float p1 = ex2_approx(x[2 * t + 1]);
      ps2[t & 3] = f2_add(ps2[t & 3], f2_pack(p0, p1));
      pk[t] = pack_bf16x2(p0, p1);
    }
    static_assert(!FIXED || BN == 32, "columns of a part");
    tmem_st16(s_addr, *reinterpret_cast<uint32_t(*)[16]>(&pk[0]));
  } else {
    float s[BN];
    // Without a tanh or a distance the scale waits for the exponents' multiply-add.
    constexpr bool RAW = !CAP && !BIAS;
    if constexpr (RAW) {
      load(s, 0);
    } else {
      // All columns at once, or 64 with the tanh and distances too, where all spill (16 heads of
      // 8192, two tiles at d = 64, one at d = 128: distances 219 / 210 / 207 and 306 / 286 / 276 us
      // with 32, 64 and 128 columns; both 324 / 309 / 408 and 415 / 370 / 417).
      constexpr int PART = CAP && BN > 64 ? 64 : BN;
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += PART) {
        float(&y)[PART] = *reinterpret_cast<float(*)[PART]>(&s[c0]);
        float none[1];
        load(y, c0);
        shape_scores<PART, CAP, BIAS, false>(y, none, p.f, slope2,
                                             static_cast<float>(pos - kbase - c0), 0.0f,
                                             [&](auto& z, int c1) { load(z, c0 + c1); });
      }
    }
    if (mask) {
#pragma unroll
      for (int t = 0; t < BN; ++t)
        if (static_cast<unsigned>(t) - from >= len) s[t] = -INFINITY;
    }
    // Row max over 8 independent partial maxima, two values a three-input max.
    float pm[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) pm[u] = fmaxf(s[u], s[u + 8]);
#pragma unroll
    for (int t = 16; t < BN; t += 16)
#pragma unroll
      for (int u = 0; u < 8; ++u) pm[u] = fmax3(pm[u], s[t + u], s[t + u + 8]);
    const float mx = fmaxf(fmax3(pm[0], pm[1], pm[2]),
                           fmaxf(fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])));
    const float c = RAW ? p.f.k : 1.0f;
    const float m_new = fmaxf(m, mx * c);
    // The reference moves only when the maximum has grown by more than the threshold.
    moved = m_new > m + kRescaleThreshold;
    if (moved) {
      alpha = ex2_approx(m - m_new);
      m = m_new;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    const uint64_t nm2 = f2_pack(-ref, -ref), c2 = f2_pack(c, c);
    uint32_t pk[BN / 2];
#pragma unroll
    for (int t = 0; t < BN / 2; ++t) {
      float x0, x1;
      const uint64_t x = f2_pack(s[2 * t], s[2 * t + 1]);
      f2_unpack(RAW ? f2_fma(x, c2, nm2) : f2_add(x, nm2), x0, x1);
      const float p0 = ex2_approx(x0);
      const float p1 = ex2_approx(x1);
      ps2[t & 3] = f2_add(ps2[t & 3], f2_pack(p0, p1));
      pk[t] = pack_bf16x2(p0, p1);
    }
#pragma unroll
    for (int q4 = 0; q4 < BN / 64; ++q4)
      tmem_st32(s_addr + q4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[q4 * 32]));
  }
  float sum, sum_hi;
  f2_unpack(f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3])), sum, sum_hi);
  l = l * alpha + (sum + sum_hi);
  return alpha;
}

// A row's O out of TMEM at `col_o` (any: there is one) over `weight`, and its lse; zeros and
// -infinity for a row that sees no key.  Every GROUPS-th part of 32 columns, from the g-th on.
// The whole warp calls this.
template <int D, int GROUPS>
__device__ __forceinline__ void store_row(const ScoreFwdParams& p, int bh, int qi, uint32_t col_o,
                                          int g, bool any, bool empty, float m, float l,
                                          float weight) {
  const float inv_l = 1.0f / weight;
  const bool live = qi < p.s.Nq;
  __nv_bfloat16* orow = p.o + (static_cast<size_t>(bh) * p.s.Nq + (live ? qi : 0)) * D;
#pragma unroll 1
  for (int q4 = g; q4 < D / 32; q4 += GROUPS) {
    uint32_t r[32];
    if (any) {
      tmem_ld32(col_o + q4 * 32, r);
      tmem_wait_ld();
    }
    uint32_t pk[16];
#pragma unroll
    for (int t = 0; t < 16; ++t)
      pk[t] = empty || !any ? 0u
                            : pack_bf16x2(__uint_as_float(r[2 * t]) * inv_l,
                                          __uint_as_float(r[2 * t + 1]) * inv_l);
    if (live) {
      uint4* dst = reinterpret_cast<uint4*>(orow + q4 * 32);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        dst[t] = make_uint4(pk[4 * t], pk[4 * t + 1], pk[4 * t + 2], pk[4 * t + 3]);
    }
  }
  if (live && g == 0)
    p.lse[static_cast<size_t>(bh) * p.s.Nq + qi] =
        empty ? -INFINITY : (m + log2f(l)) * kScoreLn2;
}

// FIXED: the softmax reference is 0.
template <int D, bool CAP, bool BIAS, bool FIXED>
__global__ void __launch_bounds__((ScoreFwdCfg<D, FIXED>::THREADS), 1)
    fa_scores_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ ScoreFwdParams p) {
  using C = ScoreFwdCfg<D, FIXED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  KeySpan* hulls = reinterpret_cast<KeySpan*>(smem + C::OFF_MISC + 8);
  uint32_t* err = p.s.err;

  const int warp = threadIdx.x >> 5;
  // Groups of heads whose K/V fit in L2, the last query tiles (the most keys, where the mask
  // is causal) first.
  const int per_group = p.heads_per_group * p.n_qtiles;
  const int grp = static_cast<int>(blockIdx.x) / per_group;
  const int rem = static_cast<int>(blockIdx.x) - grp * per_group;
  const int in_grp = min(p.heads_per_group, p.n_heads - grp * p.heads_per_group);
  const int qi_ = rem / in_grp;
  const int bh = grp * p.heads_per_group + (rem - qi_ * in_grp);
  const int qt = p.n_qtiles - 1 - qi_;
  const int b = bh / p.s.Hq;
  const int hq = bh - b * p.s.Hq;
  const int kvz = b * p.s.Hkv + hq / p.s.G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i)
      mbar_init(bar(i),
                (i >= C::B_PFULL && i < C::B_PFULL + C::NB) || i == C::B_SUM ? C::WARPS : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::WARPS + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  KeySpan span{0, 0};
  if (warp < C::WARPS) {
    span = row_span(p.s, b, qt * C::BM + static_cast<int>(threadIdx.x & 127));
    if (warp < 4) {
      const KeySpan h = warp_hull(span);
      if ((threadIdx.x & 31) == 0) hulls[warp] = h;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int lo = min(min(hulls[0].lo, hulls[1].lo), min(hulls[2].lo, hulls[3].lo));
  const int hi = max(max(hulls[0].hi, hulls[1].hi), max(hulls[2].hi, hulls[3].hi));
  const int j0 = hi > 0 ? lo / C::BN : 0;  // first key tile
  const int n_kv = hi > 0 ? (hi + C::BN - 1) / C::BN - j0 : 0;

  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ TMA producer
    if (n_kv > 0 && elect_one()) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      const uint64_t keep = policy_evict_last();  // K/V are re-read by the other query tiles
      mbar_arrive_expect_tx(bar(C::B_QFULL), C::Q_TILE);
#pragma unroll
      for (int s = 0; s < C::SUB; ++s)
        tma_load_3d(sQ + s * C::Q_BLOCK, &tmQ, bar(C::B_QFULL), 64 * s, qt * C::BM, bh);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n_kv; ++j) {
        const int st = j % C::NS;
        const uint32_t ph = ((j / C::NS) - 1) & 1;
        if (j >= C::NS && !mbar_wait(bar(C::B_KEMPTY + st), ph, abort_flag, err, kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_KFULL + st), C::KV_TILE);
#pragma unroll
        for (int s = 0; s < C::SUB; ++s)
          tma_load_3d_hint(sK + st * C::KV_TILE + s * C::KV_BLOCK, &tmK, bar(C::B_KFULL + st),
                           64 * s, (j0 + j) * C::BN, kvz, keep);
        k_issued = j + 1;
        if (j >= C::NS && !mbar_wait(bar(C::B_VEMPTY + st), ph, abort_flag, err, kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_VFULL + st), C::KV_TILE);
#pragma unroll
        for (int s = 0; s < C::SUB; ++s)
          tma_load_3d_hint(sV + st * C::KV_TILE + s * C::KV_BLOCK, &tmV, bar(C::B_VFULL + st),
                           64 * s, (j0 + j) * C::BN, kvz, keep);
        v_issued = j + 1;
      }
      if (*abort_flag) {
        // The copies already issued land before the CTA's memory is released.
        mbar_wait_timed(bar(C::B_QFULL), 0);
        for (int j = max(0, k_issued - C::NS); j < k_issued; ++j)
          mbar_wait_timed(bar(C::B_KFULL + j % C::NS), (j / C::NS) & 1);
        for (int j = max(0, v_issued - C::NS); j < v_issued; ++j)
          mbar_wait_timed(bar(C::B_VFULL + j % C::NS), (j / C::NS) & 1);
      }
    }
  } else if (warp == C::WARPS + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n_kv > 0 && elect_one()) {
      constexpr uint32_t ID_S = idesc_bf16_f32(128, C::BN, false, false);
      constexpr uint32_t ID_O = idesc_bf16_f32(128, C::D, false, true);
      const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(sV, C::KV_BLOCK, 1024);  // MN-major, N = D
      bool ok = mbar_wait(bar(C::B_QFULL), 0, abort_flag, err, kErrTimeoutMma);
      auto issue_s = [&](int j) -> bool {
        const int st = j % C::NS;
        if (!mbar_wait(bar(C::B_KFULL + st), (j / C::NS) & 1, abort_flag, err, kErrTimeoutMma))
          return false;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (j % C::NB) * C::BN;
        const uint64_t kd = desc_add(k_desc, st * C::KV_TILE);
        mma_ss_k<ID_S, 0>(d_tmem, q_desc, kd);
#pragma unroll
        for (int kk = 1; kk < C::D / 16; ++kk)
          mma_ss_k<ID_S, 1>(d_tmem, desc_add(q_desc, (kk >> 2) * C::Q_BLOCK + (kk & 3) * 32),
                            desc_add(kd, (kk >> 2) * C::KV_BLOCK + (kk & 3) * 32));
        mma_commit(bar(C::B_SFULL + j % C::NB));
        mma_commit(bar(C::B_KEMPTY + st));
        return true;
      };
      for (int j = 0; ok && j < min(n_kv, 2); ++j) ok = issue_s(j);
      for (int j = 0; ok && j < n_kv; ++j) {
        const int st = j % C::NS;
        const int bf = j % C::NB;
        if (!mbar_wait(bar(C::B_VFULL + st), (j / C::NS) & 1, abort_flag, err, kErrTimeoutMma))
          break;
        if (!mbar_wait(bar(C::B_PFULL + bf), (j / C::NB) & 1, abort_flag, err, kErrTimeoutMma))
          break;
        tc_fence_after();
        // O += P_j V_j: P of keys KH g.. packed at columns KH g.. of buffer bf, 16 keys a step.
        constexpr int KPW = C::KH / 16;
        const uint64_t vd = desc_add(v_desc, st * C::KV_TILE);
        const uint32_t pa = tmem + bf * C::BN;
        if (j == 0)
          mma_ts_k<ID_O, 0>(tmem + C::COL_O, pa, vd);
        else
          mma_ts_k<ID_O, 1>(tmem + C::COL_O, pa, vd);
#pragma unroll
        for (int kk = 1; kk < C::BN / 16; ++kk)
          mma_ts_k<ID_O, 1>(tmem + C::COL_O, pa + kk / KPW * C::KH + kk % KPW * 8,
                            desc_add(vd, kk * 2048));
        mma_commit(bar(C::B_ODONE));
        mma_commit(bar(C::B_VEMPTY + st));
        // Once, after the last product: at its epilogue the softmax may be two phases behind
        // on the per-tile barrier, which parity cannot tell from "done".
        if (j == n_kv - 1) mma_commit(bar(C::B_FINAL));
        // S_{j+2} into the buffer whose P_{j-1} the previous O += P V read.
        if (j + 2 < n_kv && !issue_s(j + 2)) break;
      }
      if (*abort_flag) {
        mma_commit(bar(C::B_DRAIN));
        mbar_wait_timed(bar(C::B_DRAIN), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax (rows)
    // Warp w: rows 32 (w % 4).., key columns KH (w / 4)...
    const int row = threadIdx.x & 127, g = warp >> 2;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int qi = qt * C::BM + row;
    const float slope2 = BIAS && p.s.slopes ? p.s.slopes[hq] * kScoreLog2e : 0.0f;
    const int pos = p.s.q_offset + qi;
    float m_used = FIXED ? 0.0f : -INFINITY;  // reference, log2 domain
    float l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const int bf = j % C::NB;
      // Waits are made warp-uniform: the TMEM loads and stores below are
      // warp-collective, so either every lane goes on or every lane stops.
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_SFULL + bf), (j / C::NB) & 1, abort_flag,
                                             err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      const int kbase = (j0 + j) * C::BN + C::KH * g;
      const bool need_mask = __any_sync(0xffffffffu, span.lo > kbase || span.hi < kbase + C::KH);
      bool upd = false;
      const float alpha =
          score_row<C::KH, CAP, BIAS, FIXED>(p.s, tmem + lane_off + bf * C::BN + C::KH * g,
                                             need_mask, span, kbase, pos, slope2, m_used, l, upd);
      if (!FIXED && j > 0 && __any_sync(0xffffffffu, upd)) {
        // O must be final before it is rescaled.  S_j being ready implies O += P_{j-2}
        // V_{j-2} is done, so the per-tile barrier is at most one phase behind.
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_ODONE), (j - 1) & 1, abort_flag, err,
                                               kErrTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int q4 = 0; q4 < C::D / 32; ++q4) {
          uint32_t r[32];
          tmem_ld32(tmem + lane_off + C::COL_O + q4 * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < 32; ++t) r[t] = __float_as_uint(__uint_as_float(r[t]) * alpha);
          tmem_st32(tmem + lane_off + C::COL_O + q4 * 32, r);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_PFULL + bf));
    }
    // ------------------------------------------------------------ epilogue
    if constexpr (C::GROUPS > 1) {
      float* sums = reinterpret_cast<float*>(smem + C::OFF_SUM);
      sums[g * C::BM + row] = l;
      mbar_arrive_warp(bar(C::B_SUM));
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(C::B_SUM), 0, abort_flag, err,
                                                   kErrTimeoutEpilogue));
      l = 0.0f;
#pragma unroll
      for (int k = 0; k < C::GROUPS; ++k) l += sums[k * C::BM + row];
    }
    if (ok && n_kv > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_FINAL), 0, abort_flag, err,
                                             kErrTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      // A row of one key is its v: over the weight as P holds it (with a moving reference it is 1).
      const float weight = FIXED && span.hi - span.lo == 1
                               ? __bfloat162float(__float2bfloat16_rn(l))
                               : l;
      store_row<D, C::GROUPS>(p, bh, qi, tmem + lane_off + C::COL_O, g, n_kv > 0, span.hi == 0,
                              m_used, l, weight);
    }
  }

  // Every warp reconverges first: in the TMA and MMA warps only one lane did
  // the work, and the CTA barrier below must count whole, converged warps.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARPS + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace
}  // namespace fa
