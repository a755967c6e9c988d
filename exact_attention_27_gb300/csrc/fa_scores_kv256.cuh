// dK and dV of attention with shaped scores at head dimension 256 (fa_scores.cuh says how).
//
// The layout of fa_bwd_d256.cu: one CTA owns 64 keys of one (batch, key/value head) and walks
// the 128-row query tiles of every query head of the group; the accumulators are kept
// transposed, dV^T = dO^T P and dK^T = Q^T dS, with the head dimension on the tensor-memory
// lanes (two halves of 128) and the keys on 2 x 64 columns:
//   dP = dO V^T, S = Q K^T                      tcgen05.mma  M 128 queries, N 64 keys, K 256
//   P = exp(x - L), dS = P o (1 - tanh^2) o (dP - D)    a query row a thread and half tile
//   dV^T += dO^T P, dK^T += Q^T dS              two MMAs each (halves of d)
// Q and dO come as two halves of d with a barrier each, reloaded as soon as the product that
// reads a half is done: shared memory has room for one stage.  8 query heads of 4 groups, 4000
// positions, cap, window 1024: 121 us in two rounds of CTAs.
//
// Warps: 0-7 query rows (warp w: rows 32 (w % 4).., keys 32 (w / 4)..), 8 TMA, 9 MMA issuer
// and tensor-memory owner.  Tensor memory: dV^T [0,128), dK^T [128,256), S [256,320), dP
// [320,384).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

struct ScoreKv256Cfg {
  static constexpr int D = 256;
  static constexpr int BK = 64;                    // keys per CTA
  static constexpr int BQ = 128;                   // queries per step
  static constexpr int KSUB = 64 * 128;            // 64 rows x 64 bf16
  static constexpr int QSUB = 128 * 128;           // 128 rows x 64 bf16
  static constexpr int KTILE = 4 * KSUB;
  static constexpr int QTILE = 4 * QSUB;
  static constexpr int PBYTES = 128 * 128;         // 128 query rows x 64 keys bf16
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KTILE;
  static constexpr int OFF_Q = OFF_V + KTILE;
  static constexpr int OFF_DO = OFF_Q + QTILE;
  static constexpr int OFF_P = OFF_DO + QTILE;
  static constexpr int OFF_DS = OFF_P + PBYTES;
  static constexpr int OFF_BAR = OFF_DS + PBYTES;
  // Q and dO are handled as two halves of d (128 columns, 32 KB each), so
  // that each half is reloaded as soon as the products reading it are done.
  static constexpr int B_KV = 0;
  static constexpr int B_QFULL = 1;      // [2] Q half landed
  static constexpr int B_DOFULL = 3;     // [2]
  static constexpr int B_QEMPTY = 5;     // [2] dK^T[h] of the step done: Q half h free
  static constexpr int B_DOEMPTY = 7;    // [2] dV^T[h] of the step done: dO half h free
  static constexpr int B_S = 9;          // S in tensor memory
  static constexpr int B_DP = 10;        // dP in tensor memory
  static constexpr int B_P = 11;         // P in shared memory, S read (8 warp arrivals)
  static constexpr int B_DS = 12;        // dS in shared memory, dP read (8 warp arrivals)
  static constexpr int B_PFREE = 13;     // dV^T done: P buffer free
  static constexpr int B_DSFREE = 14;    // dK^T done: dS buffer free
  static constexpr int B_FINAL = 15;     // every product issued has completed (once)
  static constexpr int B_DRAIN = 16;
  static constexpr int NBAR = 17;
  static constexpr int QHALF = 2 * QSUB;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 320;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_DV = 0, COL_DK = 128, COL_S = 256, COL_DP = 320;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct ScoreKv256Params {
  ScoreParams s;
  const float* lse;
  const float* Dvec;
  const int2* tiles;  // [B][n_qtiles] union of the spans of a query tile's rows
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* part;  // [2][split][B Hkv][Nk][256] sums for dV and dK of `split` CTAs a key tile
  int split;
  int n_qtiles, n_ktiles;
};

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(320, 1)
    fa_scores_kv256_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ CUtensorMap tmdO,
                           const __grid_constant__ ScoreKv256Params p) {
  using C = ScoreKv256Cfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* range = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  uint32_t* err = p.s.err;

  const int warp = threadIdx.x >> 5;
  // The first key tiles (the most query tiles, where the mask is causal) of all heads first,
  // the CTAs that share a key tile (as in fa_scores_dkdv.cuh) next to each other.
  const int n_units = p.s.B * p.s.Hkv;
  const int unit = static_cast<int>(blockIdx.x) / p.split;
  const int share = static_cast<int>(blockIdx.x) - unit * p.split;
  const int jt = unit / n_units;
  const int kvz = unit - jt * n_units;  // flattened (batch, kv head)
  const int b = kvz / p.s.Hkv;
  const int hkv = kvz - b * p.s.Hkv;

  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;
  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sdO = sbase + C::OFF_DO;
  const uint32_t sP = sbase + C::OFF_P;
  const uint32_t sDS = sbase + C::OFF_DS;

  // Query tiles that see these keys: i0 .. i0 + per_head - 1 of each head.
  int i0 = 0, per_head = 0, n_steps = 0, step0 = 0;
  // step -> (flattened query head, query tile)
  auto step_coords = [&](int s, int& bhq, int& it) {
    const int g = (step0 + s) / per_head;
    it = i0 + (step0 + s - g * per_head);
    bhq = b * p.s.Hq + hkv * p.s.G + g;
  };

  if (warp == 8 && elect_one()) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmdO);
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar(i), (i == C::B_P || i == C::B_DS) ? 8 : 1);
    *abort_flag = 0;
    range[0] = INT_MAX;
    range[1] = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  seen_by<C::THREADS>(p.tiles + static_cast<long long>(b) * p.n_qtiles, p.n_qtiles, jt * C::BK,
                      C::BK, range);
  __syncthreads();
  if (range[1] > 0) {
    i0 = range[0];
    per_head = range[1] - i0;
  }
  const long long all = static_cast<long long>(p.s.G) * per_head;
  step0 = static_cast<int>(all * share / p.split);  // this CTA's steps
  n_steps = static_cast<int>(all * (share + 1) / p.split) - step0;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (n_steps > 0 && elect_one()) {
      mbar_arrive_expect_tx(bar(C::B_KV), 2 * C::KTILE);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tma_load_3d(sK + c * C::KSUB, &tmK, bar(C::B_KV), 64 * c, jt * C::BK, kvz);
        tma_load_3d(sV + c * C::KSUB, &tmV, bar(C::B_KV), 64 * c, jt * C::BK, kvz);
      }
      int bhq0, it0;
      step_coords(0, bhq0, it0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mbar_arrive_expect_tx(bar(C::B_DOFULL + h), C::QHALF);
        for (int c = 2 * h; c < 2 * h + 2; ++c)
          tma_load_3d(sdO + c * C::QSUB, &tmdO, bar(C::B_DOFULL + h), 64 * c, it0 * C::BQ, bhq0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mbar_arrive_expect_tx(bar(C::B_QFULL + h), C::QHALF);
        for (int c = 2 * h; c < 2 * h + 2; ++c)
          tma_load_3d(sQ + c * C::QSUB, &tmQ, bar(C::B_QFULL + h), 64 * c, it0 * C::BQ, bhq0);
      }
      // dO of step s once dV^T of step s - 1 has read its buffer, then Q once
      // dK^T has.
      int do_half[2], q_half[2];  // steps whose half h was issued
      do_half[0] = do_half[1] = q_half[0] = q_half[1] = 1;
      for (int s = 1; s < n_steps; ++s) {
        int bhq, it;
        step_coords(s, bhq, it);
        // Halves in the order the products free them: dO[0], dO[1] (dV^T),
        // then Q[0], Q[1] (dK^T).
        bool go = true;
#pragma unroll 1
        for (int h = 0; h < 2 && go; ++h) {
          if (!mbar_wait(bar(C::B_DOEMPTY + h), (s - 1) & 1, abort_flag, err, kErrTimeoutLoad)) {
            go = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::B_DOFULL + h), C::QHALF);
          for (int c = 2 * h; c < 2 * h + 2; ++c)
            tma_load_3d(sdO + c * C::QSUB, &tmdO, bar(C::B_DOFULL + h), 64 * c, it * C::BQ, bhq);
          do_half[h] = s + 1;
        }
#pragma unroll 1
        for (int h = 0; h < 2 && go; ++h) {
          if (!mbar_wait(bar(C::B_QEMPTY + h), (s - 1) & 1, abort_flag, err, kErrTimeoutLoad)) {
            go = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::B_QFULL + h), C::QHALF);
          for (int c = 2 * h; c < 2 * h + 2; ++c)
            tma_load_3d(sQ + c * C::QSUB, &tmQ, bar(C::B_QFULL + h), 64 * c, it * C::BQ, bhq);
          q_half[h] = s + 1;
        }
        if (!go) break;
      }
      if (*abort_flag) {
        mbar_wait_timed(bar(C::B_KV), 0);
        for (int h = 0; h < 2; ++h) {
          if (do_half[h] > 0) mbar_wait_timed(bar(C::B_DOFULL + h), (do_half[h] - 1) & 1);
          if (q_half[h] > 0) mbar_wait_timed(bar(C::B_QFULL + h), (q_half[h] - 1) & 1);
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (n_steps > 0 && elect_one()) {
      constexpr uint32_t ID_SP = idesc_bf16_f32(128, 64, false, false);  // S, dP
      constexpr uint32_t ID_T = idesc_bf16_f32(128, 64, true, true);     // dV^T, dK^T
      const uint64_t q_k = smem_desc_sw128(sQ, 16, 1024);      // Q, K-major A
      const uint64_t do_k = smem_desc_sw128(sdO, 16, 1024);
      const uint64_t k_k = smem_desc_sw128(sK, 16, 1024);      // K, K-major B
      const uint64_t v_k = smem_desc_sw128(sV, 16, 1024);
      const uint64_t q_mn = smem_desc_sw128(sQ, C::QSUB, 1024);   // Q^T, MN-major A
      const uint64_t do_mn = smem_desc_sw128(sdO, C::QSUB, 1024);
      const uint64_t p_mn = smem_desc_sw128(sP, C::PBYTES, 1024);  // P, MN-major B (N = 64)
      const uint64_t ds_mn = smem_desc_sw128(sDS, C::PBYTES, 1024);
      bool ok = mbar_wait(bar(C::B_KV), 0, abort_flag, err, kErrTimeoutMma);
      for (int s = 0; ok && s < n_steps; ++s) {
        const uint32_t ph = s & 1;
        // dP = dO V^T (the dP columns were read by the threads of step s - 1
        // before they arrived on B_DS, which the previous iteration waited for).
        if (!mbar_wait(bar(C::B_DOFULL), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
        mma_ss_k<ID_SP, 0>(tmem + C::COL_DP, do_k, v_k);
#pragma unroll
        for (int kk = 1; kk < 8; ++kk)
          mma_ss_k<ID_SP, 1>(tmem + C::COL_DP,
                             desc_add(do_k, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                             desc_add(v_k, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        if (!mbar_wait(bar(C::B_DOFULL + 1), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 8; kk < 16; ++kk)
          mma_ss_k<ID_SP, 1>(tmem + C::COL_DP,
                             desc_add(do_k, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                             desc_add(v_k, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        mma_commit(bar(C::B_DP));
        // S = Q K^T
        if (!mbar_wait(bar(C::B_QFULL), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
        mma_ss_k<ID_SP, 0>(tmem + C::COL_S, q_k, k_k);
#pragma unroll
        for (int kk = 1; kk < 8; ++kk)
          mma_ss_k<ID_SP, 1>(tmem + C::COL_S,
                             desc_add(q_k, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                             desc_add(k_k, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        if (!mbar_wait(bar(C::B_QFULL + 1), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 8; kk < 16; ++kk)
          mma_ss_k<ID_SP, 1>(tmem + C::COL_S,
                             desc_add(q_k, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                             desc_add(k_k, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        mma_commit(bar(C::B_S));
        // dV^T[h] += dO^T[h] P: 128 queries in 8 steps of 16 rows (2 KB).
        if (!mbar_wait(bar(C::B_P), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t a = desc_add(do_mn, 2 * h * C::QSUB);
          const uint32_t dst = tmem + C::COL_DV + 64 * h;
          if (s == 0)
            mma_ss_k<ID_T, 0>(dst, a, p_mn);
          else
            mma_ss_k<ID_T, 1>(dst, a, p_mn);
#pragma unroll
          for (int kq = 1; kq < 8; ++kq)
            mma_ss_k<ID_T, 1>(dst, desc_add(a, kq * 2048), desc_add(p_mn, kq * 2048));
          mma_commit(bar(C::B_DOEMPTY + h));  // dO half h is no longer read
        }
        mma_commit(bar(C::B_PFREE));
        // dK^T[h] += Q^T[h] dS
        if (!mbar_wait(bar(C::B_DS), ph, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t a = desc_add(q_mn, 2 * h * C::QSUB);
          const uint32_t dst = tmem + C::COL_DK + 64 * h;
          if (s == 0)
            mma_ss_k<ID_T, 0>(dst, a, ds_mn);
          else
            mma_ss_k<ID_T, 1>(dst, a, ds_mn);
#pragma unroll
          for (int kq = 1; kq < 8; ++kq)
            mma_ss_k<ID_T, 1>(dst, desc_add(a, kq * 2048), desc_add(ds_mn, kq * 2048));
          mma_commit(bar(C::B_QEMPTY + h));  // Q half h is no longer read
        }
        mma_commit(bar(C::B_DSFREE));
        if (s == n_steps - 1) mma_commit(bar(C::B_FINAL));
      }
      if (*abort_flag) {
        mma_commit(bar(C::B_DRAIN));
        mbar_wait_timed(bar(C::B_DRAIN), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ query rows
    const int wq = warp & 3, g = warp >> 2;
    const int row = wq * 32 + static_cast<int>(threadIdx.x & 31);
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const int kbase = jt * C::BK + 32 * g;  // first key of this warp's half of the tile
    // L, D and the span of this thread's row at step s, loaded one step ahead.
    auto load_row = [&](int s, float& l, float& dd, KeySpan& span) {
      int bhq, it;
      step_coords(s, bhq, it);
      const int q = it * C::BQ + row;
      span = row_span(p.s, b, q);
      const size_t idx = static_cast<size_t>(bhq) * p.s.Nq + min(q, p.s.Nq - 1);
      l = p.lse[idx];
      dd = p.Dvec[idx];
    };
    float l_cur = 0.0f, d_cur = 0.0f;
    KeySpan span_cur{0, 0};
    if (n_steps > 0) load_row(0, l_cur, d_cur, span_cur);
    bool ok = true;
    for (int s = 0; s < n_steps; ++s) {
      const uint32_t ph = s & 1;
      int bhq, it;
      step_coords(s, bhq, it);
      const KeySpan span = span_cur;
      const bool sees = span.hi > 0;
      const float L2 = sees ? l_cur * kScoreLog2e : INFINITY;  // no key seen: P = 0
      const float nd = sees ? -d_cur : 0.0f;
      const uint64_t nd2 = f2_pack(nd, nd);
      const float slope2 =
          BIAS && p.s.slopes ? p.s.slopes[bhq - b * p.s.Hq] * kScoreLog2e : 0.0f;
      if (s + 1 < n_steps) load_row(s + 1, l_cur, d_cur, span_cur);  // used at the next step
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_S), ph, abort_flag, err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[32];
      tmem_ld32(tmem + lane_off + C::COL_S + 32 * g, sv);
      // Masking only where a row of the warp does not see all of its half; warp-uniform.
      const bool masked = __any_sync(0xffffffffu, span.lo > kbase || span.hi < kbase + 32);
      const unsigned from = static_cast<unsigned>(span.lo - kbase);
      const unsigned len = static_cast<unsigned>(span.hi - span.lo);
      tmem_wait_ld();
      float pv[32], gr[CAP ? 32 : 1];
#pragma unroll
      for (int e = 0; e < 32; ++e) pv[e] = __uint_as_float(sv[e]);
      shape_scores<32, CAP, BIAS, CAP>(
          pv, gr, p.s.f, slope2, static_cast<float>(p.s.q_offset + it * C::BQ + row - kbase), L2,
          [&](float (&y)[32], int) { load_scores(tmem + lane_off + C::COL_S + 32 * g, y); });
#pragma unroll
      for (int e = 0; e < 32; ++e) pv[e] = ex2_approx(pv[e]);
      if (masked) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (static_cast<unsigned>(e) - from >= len) pv[e] = 0.0f;
      }
      uint32_t pk[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) pk[u] = pack_bf16x2(pv[2 * u], pv[2 * u + 1]);
      if constexpr (CAP) {
#pragma unroll
        for (int e = 0; e < 32; ++e) pv[e] *= gr[e];
      }
      // The P buffer is free once dV^T of the step before has read it.
      if (s > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PFREE), (s - 1) & 1, abort_flag, err,
                                               kErrTimeoutSoftmax));
        if (!ok) break;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(sP + sw128(row, 4 * g + c), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                     pk[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_P));
      // dS = P o (1 - tanh^2) o (dP - D), 0 where masked (0 x NaN where a row that sees nothing
      // holds anything) and in a row of one key, where dP = D.
      const unsigned len_ds = len > 1 ? len : 0u;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_DP), ph, abort_flag, err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t dpv[32];
      tmem_ld32(tmem + lane_off + C::COL_DP + 32 * g, dpv);
      tmem_wait_ld();
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        float d0, d1;
        f2_unpack(f2_mul(f2_pack(pv[2 * u], pv[2 * u + 1]),
                         f2_add(f2_pack(__uint_as_float(dpv[2 * u]),
                                        __uint_as_float(dpv[2 * u + 1])),
                                nd2)),
                  d0, d1);
        if (masked) {
          if (static_cast<unsigned>(2 * u) - from >= len_ds) d0 = 0.0f;
          if (static_cast<unsigned>(2 * u + 1) - from >= len_ds) d1 = 0.0f;
        }
        pk[u] = pack_bf16x2(d0, d1);
      }
      if (s > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DSFREE), (s - 1) & 1, abort_flag, err,
                                               kErrTimeoutSoftmax));
        if (!ok) break;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(sDS + sw128(row, 4 * g + c), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                     pk[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_DS));
    }
    // ---- epilogue, once every product has completed: warpgroup 0 writes dV,
    // warpgroup 1 dK (times scale).  Lane l of warp w holds head-dimension
    // column 128 h + 32 (w % 4) + l of a half h for the tile's 64 keys.
    if (ok && n_steps > 0)
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_FINAL), 0, abort_flag, err, kErrTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      const float mul = g == 0 ? 1.0f : p.s.scale;
      __nv_bfloat16* out = g == 0 ? p.dv : p.dk;
      float* part = p.part + static_cast<size_t>((g == 0 ? 0 : p.split) + share) * n_units *
                                 p.s.Nk * C::D;
      const uint32_t col0 = g == 0 ? C::COL_DV : C::COL_DK;
      const int lane = static_cast<int>(threadIdx.x & 31);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int dcol = 128 * h + 32 * wq + lane;
#pragma unroll 1
        for (int kc = 0; kc < 2; ++kc) {
          uint32_t r[32];
          if (n_steps > 0) {
            tmem_ld32(tmem + lane_off + col0 + 64 * h + 32 * kc, r);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;  // no query sees these keys
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = jt * C::BK + 32 * kc + e;
            if (key >= p.s.Nk) continue;
            const size_t at = (static_cast<size_t>(kvz) * p.s.Nk + key) * C::D + dcol;
            if (p.split > 1)
              part[at] = __uint_as_float(r[e]) * mul;
            else
              out[at] = __float2bfloat16_rn(__uint_as_float(r[e]) * mul);
          }
        }
      }
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

template <bool CAP, bool BIAS>
cudaError_t launch_scores_kv256_t(const ScoreMaps& m, const float* lse, const float* Dv,
                                  const int2* tiles, void* dk, void* dv, float* part, int split,
                                  const ScoreParams& s, cudaStream_t stream) {
  using C = ScoreKv256Cfg;
  auto kern = fa_scores_kv256_kernel<CAP, BIAS>;
  cudaError_t e = set_smem_limit_once<fa_scores_kv256_kernel<CAP, BIAS>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  ScoreKv256Params p;
  p.s = s;
  p.lse = lse;
  p.Dvec = Dv;
  p.tiles = tiles;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.part = part;
  p.split = split;
  p.n_qtiles = (s.Nq + C::BQ - 1) / C::BQ;
  p.n_ktiles = (s.Nk + C::BK - 1) / C::BK;
  const long long grid = static_cast<long long>(p.n_ktiles) * s.B * s.Hkv * split;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(C::THREADS),
                          C::SMEM_BYTES, stream, m.q, m.k, m.v, m.dO, p);
}

}  // namespace

template <>
cudaError_t launch_scores_dkdv<256>(const ScoreMaps& m, const float* lse, const float* Dv,
                                    const int2* tiles, void* dk, void* dv, float* part,
                                    int split, const ScoreParams& p, int mode, cudaStream_t stream) {
  switch (mode) {
    case kScorePlain:
      return launch_scores_kv256_t<false, false>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    case kScoreBias:
      return launch_scores_kv256_t<false, true>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    case kScoreCap:
      return launch_scores_kv256_t<true, false>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    default: return launch_scores_kv256_t<true, true>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
  }
}

}  // namespace fa
