// Forward of attention with shaped scores (fa_scores.cuh says how), two 128-row query tiles a
// CTA, head dimensions 64, 96 and 128.
//
// As in fa_fwd.cu, two consecutive query tiles A and B share each K and V tile, with a softmax
// warpgroup each (a query row a thread), so that one tile's softmax runs while the tensor core
// works on the other's products: per key tile O_A += P_A V, next S_A, O_B += P_B V, next S_B.
// Each tile visits the key tiles that the union of its own rows' spans touches; the CTA loads
// all from the first to the last of either.
//
// Warps: 0-3 softmax of tile A, 4-7 of B, 8 TMA, 9 MMA issuer and tensor-memory owner, 10 and
// 11 idle.  Registers: 384 threads at 168: 224 / 224 / 56.  Tensor memory: S of tile x at
// columns 128 x (P, packed in pairs, over its first half), O at 256 + DP x.
//
// Not for scores whose cap fixes the reference (fa_scores_fwd.cuh): there four warps share a row.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_scores_fwd.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

template <int D_>
struct ScoreFwd2Cfg {
  static constexpr int D = D_;
  static constexpr int DP = (D + 63) / 64 * 64;
  static constexpr int BM = 128, BN = 128;
  static constexpr int SUB = DP / 64;
  static constexpr int BLOCK = 128 * 128;
  static constexpr int TILE = SUB * BLOCK;
  static constexpr int NS = D == 64 ? 4 : 2;     // K/V ring stages
  static constexpr int OFF_Q = 0;                // two query tiles
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + NS * TILE;
  static constexpr int OFF_BAR = OFF_V + NS * TILE;
  static constexpr int B_QFULL = 0;
  static constexpr int B_KFULL = 1;
  static constexpr int B_KEMPTY = B_KFULL + NS;
  static constexpr int B_VFULL = B_KEMPTY + NS;
  static constexpr int B_VEMPTY = B_VFULL + NS;
  static constexpr int B_SFULL = B_VEMPTY + NS;  // [2] S of tile x
  static constexpr int B_PFULL = B_SFULL + 2;    // [2] P of tile x (4 warps)
  static constexpr int B_ODONE = B_PFULL + 2;    // [2] O_x += P_x V
  static constexpr int B_DRAIN = B_ODONE + 2;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;  // tmem slot, abort word, 8 warps' hulls
  static constexpr int SMEM_BYTES = OFF_MISC + 8 + 64 + 1024;
  static constexpr int THREADS = 384;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1)
    fa_scores_fwd2_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ ScoreFwdParams p) {
  using C = ScoreFwd2Cfg<D>;
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
  const int n_pairs = (p.n_qtiles + 1) / 2;
  const int per_group = p.heads_per_group * n_pairs;
  const int grp = static_cast<int>(blockIdx.x) / per_group;
  const int rem = static_cast<int>(blockIdx.x) - grp * per_group;
  const int in_grp = min(p.heads_per_group, p.n_heads - grp * p.heads_per_group);
  const int pi = rem / in_grp;
  const int bh = grp * p.heads_per_group + (rem - pi * in_grp);
  const int pair = n_pairs - 1 - pi;
  const int b = bh / p.s.Hq;
  const int hq = bh - b * p.s.Hq;
  const int kvz = b * p.s.Hkv + hq / p.s.G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i)
      mbar_init(bar(i), i == C::B_PFULL || i == C::B_PFULL + 1 ? 4 : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp < 8) {
    const KeySpan h =
        warp_hull(row_span(p.s, b, 2 * pair * C::BM + static_cast<int>(threadIdx.x)));
    if ((threadIdx.x & 31) == 0) hulls[warp] = h;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Key tiles of each query tile, and those loaded: from the first to the last of either.
  auto hull = [&](int x, int& from, int& to) {
    const KeySpan* h = hulls + 4 * x;
    const int lo = min(min(h[0].lo, h[1].lo), min(h[2].lo, h[3].lo));
    const int hi = max(max(h[0].hi, h[1].hi), max(h[2].hi, h[3].hi));
    from = hi > 0 ? lo / C::BN : INT_MAX;
    to = hi > 0 ? (hi + C::BN - 1) / C::BN : 0;
  };
  int a0, a1, b0, b1;
  hull(0, a0, a1);
  hull(1, b0, b1);
  const int head = min(a0, b0);
  const int n_kv = max(max(a1, b1) - head, 0);
  // Counted from `head`: tile A sees [a0, a1), B [b0, b1); 0, 0 for one that sees nothing.
  a1 = max(a1 - head, 0);
  a0 = a1 > 0 ? a0 - head : 0;
  b1 = max(b1 - head, 0);
  b0 = b1 > 0 ? b0 - head : 0;

  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;

  if (warp >= 8) {
    reg_decrease<56>();
    if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      if (n_kv > 0 && elect_one()) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        const uint64_t keep = policy_evict_last();  // K/V are re-read by the other query tiles
        mbar_arrive_expect_tx(bar(C::B_QFULL), 2 * C::TILE);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int s = 0; s < C::SUB; ++s)
            tma_load_3d(sQ + x * C::TILE + s * C::BLOCK, &tmQ, bar(C::B_QFULL), 64 * s,
                        (2 * pair + x) * C::BM, bh);
        int k_issued = 0, v_issued = 0;
        for (int n = 0; n < n_kv; ++n) {
          const int st = n % C::NS;
          const uint32_t ph = ((n / C::NS) - 1) & 1;
          const int row = (head + n) * C::BN;
          if (n >= C::NS &&
              !mbar_wait(bar(C::B_KEMPTY + st), ph, abort_flag, err, kErrTimeoutLoad))
            break;
          mbar_arrive_expect_tx(bar(C::B_KFULL + st), C::TILE);
#pragma unroll
          for (int s = 0; s < C::SUB; ++s)
            tma_load_3d_hint(sK + st * C::TILE + s * C::BLOCK, &tmK, bar(C::B_KFULL + st), 64 * s,
                             row, kvz, keep);
          k_issued = n + 1;
          if (n >= C::NS &&
              !mbar_wait(bar(C::B_VEMPTY + st), ph, abort_flag, err, kErrTimeoutLoad))
            break;
          mbar_arrive_expect_tx(bar(C::B_VFULL + st), C::TILE);
#pragma unroll
          for (int s = 0; s < C::SUB; ++s)
            tma_load_3d_hint(sV + st * C::TILE + s * C::BLOCK, &tmV, bar(C::B_VFULL + st), 64 * s,
                             row, kvz, keep);
          v_issued = n + 1;
        }
        if (*abort_flag) {
          // The copies already issued land before the CTA's memory is released.
          mbar_wait_timed(bar(C::B_QFULL), 0);
          for (int n = max(0, k_issued - C::NS); n < k_issued; ++n)
            mbar_wait_timed(bar(C::B_KFULL + n % C::NS), (n / C::NS) & 1);
          for (int n = max(0, v_issued - C::NS); n < v_issued; ++n)
            mbar_wait_timed(bar(C::B_VFULL + n % C::NS), (n / C::NS) & 1);
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      if (n_kv > 0 && elect_one()) {
        constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t ID_O = idesc_bf16_f32(128, D, false, true);
        const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(sV, C::BLOCK, 1024);  // MN-major, N = D
        bool ok = mbar_wait(bar(C::B_QFULL), 0, abort_flag, err, kErrTimeoutMma);
        // S_x of tile n (K_n is there).
        auto issue_s = [&](int x, int n) {
          const uint32_t d_tmem = tmem + x * 128;
          const uint64_t qd = desc_add(q_desc, x * C::TILE);
          const uint64_t kd = desc_add(k_desc, (n % C::NS) * C::TILE);
          mma_ss_k<ID_S, 0>(d_tmem, qd, kd);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BLOCK + (kk & 3) * 32;
            mma_ss_k<ID_S, 1>(d_tmem, desc_add(qd, off), desc_add(kd, off));
          }
          mma_commit(bar(C::B_SFULL + x));
        };
        auto k_wait = [&](int n) -> bool {
          const bool there =
              mbar_wait(bar(C::B_KFULL + n % C::NS), (n / C::NS) & 1, abort_flag, err, kErrTimeoutMma);
          tc_fence_after();
          return there;
        };
        // What a tile of the range sees begins at a0 (bit 0 of `phase`: A's next P) or b0 (bit 1).
        uint32_t phase = 0;
        if (ok && (ok = k_wait(0))) {
          if (a0 == 0 && a1 > 0) issue_s(0, 0);
          if (b0 == 0 && b1 > 0) issue_s(1, 0);
          mma_commit(bar(C::B_KEMPTY));
        }
        for (int n = 0; ok && n < n_kv; ++n) {
          const int st = n % C::NS;
          if (!mbar_wait(bar(C::B_VFULL + st), (n / C::NS) & 1, abort_flag, err, kErrTimeoutMma))
            break;
          const bool next = n + 1 < n_kv;
          bool k_ready = false;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const int from = x == 0 ? a0 : b0, to = x == 0 ? a1 : b1;
            if (n >= from && n < to) {
              if (!mbar_wait(bar(C::B_PFULL + x), (phase >> x) & 1, abort_flag, err,
                             kErrTimeoutMma)) {
                ok = false;
                break;
              }
              phase ^= 1u << x;
              tc_fence_after();
              const uint64_t vd = desc_add(v_desc, st * C::TILE);
              const uint32_t pa = tmem + x * 128;
              const uint32_t od = tmem + C::COL_O + x * C::DP;
              if (n == from)
                mma_ts_k<ID_O, 0>(od, pa, vd);
              else
                mma_ts_k<ID_O, 1>(od, pa, vd);
#pragma unroll
              for (int kk = 1; kk < 8; ++kk)
                mma_ts_k<ID_O, 1>(od, pa + kk * 8, desc_add(vd, kk * 2048));
              mma_commit(bar(C::B_ODONE + x));
            }
            if (next && n + 1 >= from && n + 1 < to) {
              if (!k_ready && !(ok = k_wait(n + 1))) break;
              k_ready = true;
              issue_s(x, n + 1);
            }
          }
          if (!ok) break;
          mma_commit(bar(C::B_VEMPTY + st));
          if (next) {
            if (!k_ready && !(ok = k_wait(n + 1))) break;  // (a tile that neither sees)
            mma_commit(bar(C::B_KEMPTY + (n + 1) % C::NS));
          }
        }
        if (*abort_flag) {
          mma_commit(bar(C::B_DRAIN));
          mbar_wait_timed(bar(C::B_DRAIN), 0);
        }
      }
    }
  } else {
    reg_increase<224>();
    // ------------------------------------------------------------ softmax (rows)
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col_s = tmem + lane_off + x * 128;
    const uint32_t col_o = tmem + lane_off + C::COL_O + x * C::DP;
    const int qi = (2 * pair + x) * C::BM + row;
    // (read again rather than held across the change of the register budget)
    const KeySpan span = row_span(p.s, b, qi);
    const int j0 = x == 0 ? a0 : b0;
    const int j1 = x == 0 ? a1 : b1;
    const float slope2 = BIAS && p.s.slopes ? p.s.slopes[hq] * kScoreLog2e : 0.0f;
    const int pos = p.s.q_offset + qi;
    float m_used = -INFINITY;  // reference, log2 domain
    float l = 0.0f;
    bool ok = true;
    for (int j = j0; j < j1; ++j) {
      // Waits are made warp-uniform: the TMEM loads and stores below are
      // warp-collective, so either every lane goes on or every lane stops.
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_SFULL + x), (j - j0) & 1, abort_flag, err,
                                             kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      const int kbase = (head + j) * C::BN;
      const bool need_mask = __any_sync(0xffffffffu, span.lo > kbase || span.hi < kbase + C::BN);
      bool moved = false;
      const float alpha =
          score_row<C::BN, CAP, BIAS, false>(p.s, col_s, need_mask, span, kbase, pos, slope2,
                                             m_used, l, moved);
      // S of this tile was issued after its last O += P V, whose completion the commit behind S
      // covers: the wait for the rescale returns at once.
      if (j > j0 && __any_sync(0xffffffffu, moved)) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_ODONE + x), (j - j0 - 1) & 1, abort_flag,
                                               err, kErrTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t r[32];
          tmem_ld32(col_o + q4 * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < 32; ++t) r[t] = __float_as_uint(__uint_as_float(r[t]) * alpha);
          tmem_st32(col_o + q4 * 32, r);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_PFULL + x));
    }
    if (ok && j1 > j0)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_ODONE + x), (j1 - j0 - 1) & 1, abort_flag,
                                             err, kErrTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      store_row<D, 1>(p, bh, qi, col_o, 0, j1 > j0, span.hi == 0, m_used, l, l);
    }
  }

  // Every warp reconverges first: in the TMA and MMA warps only one lane did
  // the work, and the CTA barrier below must count whole, converged warps.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace
}  // namespace fa
