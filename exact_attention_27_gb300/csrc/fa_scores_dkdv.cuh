// dK and dV of attention with shaped scores at head dimensions 64, 96 and 128 (fa_scores.cuh
// says how).
//
// One CTA owns 128 keys of one (batch, key/value head) and walks the 128-row query tiles of
// every query head of the group that see them:
//   S  = Q_i K^T, dP = dO_i V^T          tcgen05.mma, operands in shared memory
//   P = exp(x - L), dS = P o (1 - tanh^2) o (dP - D)     threads (x: the shaped score)
//   dV += P^T dO_i, dK += dS^T Q_i       tcgen05.mma, A = P or dS as bf16 [query][key] in
//                                        shared memory, read MN-major
// Queries lie on the tensor-memory lanes, so that L, D, the span and the position of a row
// are registers of its thread (with keys there, as in fa_bwd.cu, a thread would read four
// values of each query from shared memory, where the mask and the tanh leave no room for L
// and D to enter through the products).  Four threads share a row, 32 keys each.
//
// Order of the products: S(0) dP(0), then per step dV(s) S(s+1) dK(s) dP(s+1); dV and S(s+1)
// wait for P(s) (S has been read then), dK and dP(s+1) for dS(s).  The P buffer is free when
// S(s+1) is ready, and the dS buffer when dP(s+1) is: their commits cover the products that
// read them, issued before by the same thread.  The threads work on dS(s) while dV(s) and
// S(s+1) run, and on P(s+1) while dK(s) and dP(s+1) do.
//
// Few or unequal key tiles (one head's, a group's under the causal mask) are shared by `split`
// CTAs each, which take equal stretches of its steps and leave fp32 sums that a second kernel
// adds in order (fa_scores.cu says when): results repeat to the bit.
//
// Bound by shared memory and the tensor core: a step's four products read 384 KiB of
// operands where d = 128, at 128 bytes a cycle, and the rows write P and dS there.  16 heads of
// 8192, causal: d = 128 363 us (1.51 PFLOP/s), cap 453; d = 64 321, cap 398.
//
// Warps: 0-15 query rows (warp w: rows 32 (w % 4).., keys 32 (w / 4)..), 16 TMA, 17 MMA issuer and
// tensor-memory owner.  Tensor memory: S [0,128), dP [128,256), dV [256, 256+DP), dK after it.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

template <int D_>
struct ScoreDkdvCfg {
  static constexpr int D = D_;
  static constexpr int DP = (D + 63) / 64 * 64;
  static constexpr int BK = 128, BQ = 128;
  static constexpr int SUB = DP / 64;
  static constexpr int BLOCK = 128 * 128;       // 128 rows of 128 bytes
  static constexpr int TILE = SUB * BLOCK;
  // S(s+1) is issued before dK(s), so Q has two stages; dO is free once dV(s) has read it.
  static constexpr int NQ = 2;
  static constexpr int NDO = D == 64 ? 2 : 1;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + TILE;
  static constexpr int OFF_Q = OFF_V + TILE;
  static constexpr int OFF_DO = OFF_Q + NQ * TILE;
  static constexpr int OFF_P = OFF_DO + NDO * TILE;
  static constexpr int OFF_DS = OFF_P + 2 * BLOCK;
  static constexpr int OFF_BAR = OFF_DS + 2 * BLOCK;
  static constexpr int B_KV = 0;
  static constexpr int B_QFULL = 1;                 // [NQ]
  static constexpr int B_QEMPTY = B_QFULL + NQ;     // [NQ]
  static constexpr int B_DOFULL = B_QEMPTY + NQ;    // [NDO]
  static constexpr int B_DOEMPTY = B_DOFULL + NDO;  // [NDO]
  static constexpr int B_S = B_DOEMPTY + NDO;       // S in tensor memory
  static constexpr int B_DP = B_S + 1;              // dP there
  static constexpr int B_P = B_DP + 1;              // P in shared memory, S read (every row warp)
  static constexpr int B_DS = B_P + 1;              // dS in shared memory, dP read (every row warp)
  static constexpr int B_FINAL = B_DS + 1;          // every product completed (once)
  static constexpr int B_DRAIN = B_FINAL + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;  // tmem slot, abort word, range
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int WARPS = 16;                   // row warps; then TMA and MMA
  static constexpr int THREADS = 32 * WARPS + 64;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DV = 256, COL_DK = 256 + DP;
  static_assert(COL_DK + DP <= TMEM_COLS, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct ScoreDkdvParams {
  ScoreParams s;
  const float* lse;
  const float* Dvec;
  const int2* tiles;  // [B][n_qtiles] union of the spans of a query tile's rows
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* part;  // [2][split][B Hkv][Nk][D] sums for dV and dK of `split` CTAs a key tile; 1: none
  int split;
  int n_qtiles, n_ktiles;
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(ScoreDkdvCfg<D>::THREADS, 1)
    fa_scores_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmdO,
                          const __grid_constant__ ScoreDkdvParams p) {
  using C = ScoreDkdvCfg<D>;
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
  // the CTAs that share a key tile next to each other.
  const int n_units = p.s.B * p.s.Hkv;
  const int unit = static_cast<int>(blockIdx.x) / p.split;
  const int share = static_cast<int>(blockIdx.x) - unit * p.split;
  const int jt = unit / n_units;
  const int kvz = unit - jt * n_units;                          // flattened (batch, kv head)
  const int b = kvz / p.s.Hkv;
  const int bh0 = b * p.s.Hq + (kvz - b * p.s.Hkv) * p.s.G;     // first query head of the group

  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;
  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sdO = sbase + C::OFF_DO;
  const uint32_t sP = sbase + C::OFF_P;
  const uint32_t sDS = sbase + C::OFF_DS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar(i), i == C::B_P || i == C::B_DS ? C::WARPS : 1);
    *abort_flag = 0;
    range[0] = INT_MAX;
    range[1] = 0;
    fence_barrier_init();
  }
  if (warp == C::WARPS + 1) {
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
  // Query tiles that see these keys: i0 .. i0 + per_head - 1 of each head.
  const int i0 = range[1] > 0 ? range[0] : 0;
  const int per_head = range[1] > 0 ? range[1] - i0 : 0;
  // This CTA's steps of the G per_head there are.
  const long long all = static_cast<long long>(p.s.G) * per_head;
  const int step0 = static_cast<int>(all * share / p.split);
  const int n_steps = static_cast<int>(all * (share + 1) / p.split) - step0;
  auto step_coords = [&](int s, int& bhq, int& it) {
    const int g = (step0 + s) / per_head;
    it = i0 + (step0 + s - g * per_head);
    bhq = bh0 + g;
  };

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ TMA producer
    if (n_steps > 0 && elect_one()) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmdO);
      mbar_arrive_expect_tx(bar(C::B_KV), 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < C::SUB; ++c) {
        tma_load_3d(sK + c * C::BLOCK, &tmK, bar(C::B_KV), 64 * c, jt * C::BK, kvz);
        tma_load_3d(sV + c * C::BLOCK, &tmV, bar(C::B_KV), 64 * c, jt * C::BK, kvz);
      }
      int q_issued = 0, do_issued = 0;
      for (int s = 0; s < n_steps; ++s) {
        int bhq, it;
        step_coords(s, bhq, it);
        const int qs = s % C::NQ, ds = s % C::NDO;
        if (s >= C::NQ && !mbar_wait(bar(C::B_QEMPTY + qs), ((s / C::NQ) - 1) & 1, abort_flag, err,
                                     kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_QFULL + qs), C::TILE);
#pragma unroll
        for (int c = 0; c < C::SUB; ++c)
          tma_load_3d(sQ + qs * C::TILE + c * C::BLOCK, &tmQ, bar(C::B_QFULL + qs), 64 * c,
                      it * C::BQ, bhq);
        q_issued = s + 1;
        if (s >= C::NDO && !mbar_wait(bar(C::B_DOEMPTY + ds), ((s / C::NDO) - 1) & 1, abort_flag,
                                      err, kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_DOFULL + ds), C::TILE);
#pragma unroll
        for (int c = 0; c < C::SUB; ++c)
          tma_load_3d(sdO + ds * C::TILE + c * C::BLOCK, &tmdO, bar(C::B_DOFULL + ds), 64 * c,
                      it * C::BQ, bhq);
        do_issued = s + 1;
      }
      if (*abort_flag) {
        // The copies already issued land before the CTA's memory is released.
        mbar_wait_timed(bar(C::B_KV), 0);
        for (int s = max(0, q_issued - C::NQ); s < q_issued; ++s)
          mbar_wait_timed(bar(C::B_QFULL + s % C::NQ), (s / C::NQ) & 1);
        for (int s = max(0, do_issued - C::NDO); s < do_issued; ++s)
          mbar_wait_timed(bar(C::B_DOFULL + s % C::NDO), (s / C::NDO) & 1);
      }
    }
  } else if (warp == C::WARPS + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n_steps > 0 && elect_one()) {
      constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);  // S, dP
      constexpr uint32_t ID_G = idesc_bf16_f32(128, D, true, true);      // dV, dK
      const uint64_t q_k = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t do_k = smem_desc_sw128(sdO, 16, 1024);
      const uint64_t k_k = smem_desc_sw128(sK, 16, 1024);
      const uint64_t v_k = smem_desc_sw128(sV, 16, 1024);
      const uint64_t q_mn = smem_desc_sw128(sQ, C::BLOCK, 1024);
      const uint64_t do_mn = smem_desc_sw128(sdO, C::BLOCK, 1024);
      const uint64_t p_mn = smem_desc_sw128(sP, C::BLOCK, 1024);
      const uint64_t ds_mn = smem_desc_sw128(sDS, C::BLOCK, 1024);
      // A (128 x D, K-major) times B^T into 128 columns.
      auto rows_by_keys = [&](uint32_t dst, uint64_t a, uint64_t bd) {
        mma_ss_k<ID_S, 0>(dst, a, bd);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::BLOCK + (kk & 3) * 32;
          mma_ss_k<ID_S, 1>(dst, desc_add(a, off), desc_add(bd, off));
        }
      };
      // dst += A^T B over the tile's 128 queries, 16 (2 KB of each block) a step.
      auto over_rows = [&](uint32_t dst, uint64_t a, uint64_t bd, bool first) {
        if (first)
          mma_ss_k<ID_G, 0>(dst, a, bd);
        else
          mma_ss_k<ID_G, 1>(dst, a, bd);
#pragma unroll
        for (int kk = 1; kk < 8; ++kk)
          mma_ss_k<ID_G, 1>(dst, desc_add(a, kk * 2048), desc_add(bd, kk * 2048));
      };
      auto issue_s = [&](int s) -> bool {
        const int qs = s % C::NQ;
        if (!mbar_wait(bar(C::B_QFULL + qs), (s / C::NQ) & 1, abort_flag, err, kErrTimeoutMma))
          return false;
        tc_fence_after();
        rows_by_keys(tmem + C::COL_S, desc_add(q_k, qs * C::TILE), k_k);
        mma_commit(bar(C::B_S));
        return true;
      };
      auto issue_dp = [&](int s) -> bool {
        const int ds = s % C::NDO;
        if (!mbar_wait(bar(C::B_DOFULL + ds), (s / C::NDO) & 1, abort_flag, err, kErrTimeoutMma))
          return false;
        tc_fence_after();
        rows_by_keys(tmem + C::COL_DP, desc_add(do_k, ds * C::TILE), v_k);
        mma_commit(bar(C::B_DP));
        return true;
      };
      bool ok = mbar_wait(bar(C::B_KV), 0, abort_flag, err, kErrTimeoutMma);
      if (ok) ok = issue_s(0) && issue_dp(0);
      for (int s = 0; ok && s < n_steps; ++s) {
        const int qs = s % C::NQ, ds = s % C::NDO;
        if (!mbar_wait(bar(C::B_P), s & 1, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
        over_rows(tmem + C::COL_DV, p_mn, desc_add(do_mn, ds * C::TILE), s == 0);
        mma_commit(bar(C::B_DOEMPTY + ds));
        if (s + 1 < n_steps && !issue_s(s + 1)) break;
        if (!mbar_wait(bar(C::B_DS), s & 1, abort_flag, err, kErrTimeoutMma)) break;
        tc_fence_after();
        over_rows(tmem + C::COL_DK, ds_mn, desc_add(q_mn, qs * C::TILE), s == 0);
        mma_commit(bar(C::B_QEMPTY + qs));
        if (s == n_steps - 1) mma_commit(bar(C::B_FINAL));
        if (s + 1 < n_steps && !issue_dp(s + 1)) break;
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
    const int kbase = jt * C::BK + 32 * g;  // first key of this warp's part of the tile
    // L, D and the span of this thread's row, loaded one step ahead; steps go through the query
    // tiles i0 .. i1 - 1 of one head after the other.
    const int i1 = i0 + per_head;
    int bhq0 = bh0, it = i0;
    if (n_steps > 0) step_coords(0, bhq0, it);
    const float* lse = p.lse + static_cast<size_t>(bhq0) * p.s.Nq;  // of the next step's head
    const float* dvec = p.Dvec + static_cast<size_t>(bhq0) * p.s.Nq;
    auto load_row = [&](int it, float& l, float& dd, KeySpan& span) {
      const int q = it * C::BQ + row;
      span = row_span(p.s, b, q);
      const int at = min(q, p.s.Nq - 1);
      l = lse[at];
      dd = dvec[at];
    };
    float l_cur = 0.0f, d_cur = 0.0f;
    KeySpan span_cur{0, 0};
    if (n_steps > 0) load_row(it, l_cur, d_cur, span_cur);
    int head = bhq0 - b * p.s.Hq;
    float slope2 = BIAS && p.s.slopes ? p.s.slopes[head] * kScoreLog2e : 0.0f;
    bool ok = true;
    for (int s = 0; s < n_steps; ++s) {
      const KeySpan span = span_cur;
      const bool sees = span.hi > 0;
      const float L2 = sees ? l_cur * kScoreLog2e : INFINITY;  // no key seen: P = 0
      const float nd = sees ? -d_cur : 0.0f;
      const float dist0 = static_cast<float>(p.s.q_offset + it * C::BQ + row - kbase);
      const float slope_now = slope2;
      if (s + 1 < n_steps) {  // used at the next step
        if (++it == i1) {
          it = i0;
          lse += p.s.Nq;
          dvec += p.s.Nq;
          if (BIAS && p.s.slopes) slope2 = p.s.slopes[++head] * kScoreLog2e;
        }
        load_row(it, l_cur, d_cur, span_cur);
      }
      const bool masked = __any_sync(0xffffffffu, span.lo > kbase || span.hi < kbase + 32);
      const unsigned from = static_cast<unsigned>(span.lo - kbase);
      const unsigned len = static_cast<unsigned>(span.hi - span.lo);
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_S), s & 1, abort_flag, err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      float w[32];  // scores, then P, and at last what dP - D is multiplied by
      load_scores(tmem + lane_off + C::COL_S + 32 * g, w);
      // CH columns at a time: all, or half of them where the tanh's derivative takes registers
      // too (96 a thread).
      constexpr int CH = CAP ? 16 : 32;
      uint32_t pk[16];
#pragma unroll
      for (int c0 = 0; c0 < 32; c0 += CH) {
        float(&x)[CH] = *reinterpret_cast<float(*)[CH]>(&w[c0]);
        float gr[CAP ? CH : 1];
        shape_scores<CH, CAP, BIAS, CAP>(
            x, gr, p.s.f, slope_now, dist0 - c0, L2, [&](float (&y)[CH], int) {
              load_scores(tmem + lane_off + C::COL_S + 32 * g + c0, y);
            });
#pragma unroll
        for (int t = 0; t < CH; ++t) x[t] = ex2_approx(x[t]);
        if (masked) {
#pragma unroll
          for (int t = 0; t < CH; ++t)
            if (static_cast<unsigned>(c0 + t) - from >= len) x[t] = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < CH; t += 2) {
          pk[(c0 + t) / 2] = pack_bf16x2(x[t], x[t + 1]);
          if constexpr (CAP)
            f2_unpack(f2_mul(f2_pack(x[t], x[t + 1]), f2_pack(gr[t], gr[t + 1])), x[t], x[t + 1]);
        }
      }
      // P as bf16 to its row in the block of 64 keys: four of its eight 16-byte chunks.
      const uint32_t blk = (g >> 1) * C::BLOCK;
      const int ch = (g & 1) * 4;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(sP + blk + sw128(row, ch + c), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2],
                     pk[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_P));
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_DP), s & 1, abort_flag, err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      const uint64_t nd2 = f2_pack(nd, nd);
      uint32_t dpv[32];
      tmem_ld32(tmem + lane_off + C::COL_DP + 32 * g, dpv);
      tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < 32; t += 2)
        f2_unpack(f2_mul(f2_pack(w[t], w[t + 1]),
                         f2_add(f2_pack(__uint_as_float(dpv[t]), __uint_as_float(dpv[t + 1])),
                                nd2)),
                  w[t], w[t + 1]);
      if (masked) {
        // (0 x NaN where a row that sees nothing holds anything; a row of one key has dP = D)
        const unsigned len_ds = len > 1 ? len : 0u;
#pragma unroll
        for (int t = 0; t < 32; ++t)
          if (static_cast<unsigned>(t) - from >= len_ds) w[t] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(sDS + blk + sw128(row, ch + c), pack_bf16x2(w[8 * c], w[8 * c + 1]),
                     pack_bf16x2(w[8 * c + 2], w[8 * c + 3]),
                     pack_bf16x2(w[8 * c + 4], w[8 * c + 5]),
                     pack_bf16x2(w[8 * c + 6], w[8 * c + 7]));
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_DS));
    }
    // ---- epilogue, once every product has completed: column groups 0 and 1 write dV, 2 and 3
    // dK (times scale), every other 32 columns each; lane l of warp w holds key 32 (w % 4) + l.
    if (ok && n_steps > 0)
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(C::B_FINAL), 0, abort_flag, err, kErrTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      const bool is_dv = g < 2;
      const float mul = is_dv ? 1.0f : p.s.scale;
      const uint32_t col0 = is_dv ? C::COL_DV : C::COL_DK;
      const int key = jt * C::BK + row;
      const bool live = key < p.s.Nk;
      const size_t at = (static_cast<size_t>(kvz) * p.s.Nk + (live ? key : 0)) * D;
      __nv_bfloat16* out = (is_dv ? p.dv : p.dk) + at;
      float* part = p.part + at + static_cast<size_t>((is_dv ? 0 : p.split) + share) * n_units *
                                      p.s.Nk * D;
#pragma unroll 1
      for (int q4 = g & 1; q4 < D / 32; q4 += 2) {
        uint32_t r[32];
        if (n_steps > 0) {
          tmem_ld32(tmem + lane_off + col0 + q4 * 32, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) r[u] = 0u;  // no query sees these keys
        }
        if (p.split > 1) {
          if (live) {
            float4* dst = reinterpret_cast<float4*>(part + q4 * 32);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[u] = make_float4(
                  __uint_as_float(r[4 * u]) * mul, __uint_as_float(r[4 * u + 1]) * mul,
                  __uint_as_float(r[4 * u + 2]) * mul, __uint_as_float(r[4 * u + 3]) * mul);
          }
          continue;
        }
        uint32_t pk[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          pk[u] = pack_bf16x2(__uint_as_float(r[2 * u]) * mul, __uint_as_float(r[2 * u + 1]) * mul);
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(out + q4 * 32);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            dst[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        }
      }
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

template <int D, bool CAP, bool BIAS>
cudaError_t launch_scores_dkdv_t(const ScoreMaps& m, const float* lse, const float* Dv,
                                 const int2* tiles, void* dk, void* dv, float* part, int split,
                                 const ScoreParams& s, cudaStream_t stream) {
  using C = ScoreDkdvCfg<D>;
  auto kern = fa_scores_dkdv_kernel<D, CAP, BIAS>;
  cudaError_t e = set_smem_limit_once<fa_scores_dkdv_kernel<D, CAP, BIAS>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  ScoreDkdvParams p;
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

template <int D>
cudaError_t launch_scores_dkdv(const ScoreMaps& m, const float* lse, const float* Dv,
                               const int2* tiles, void* dk, void* dv, float* part, int split,
                               const ScoreParams& p, int mode, cudaStream_t stream) {
  switch (mode) {
    case kScorePlain:
      return launch_scores_dkdv_t<D, false, false>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    case kScoreBias:
      return launch_scores_dkdv_t<D, false, true>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    case kScoreCap:
      return launch_scores_dkdv_t<D, true, false>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
    default: return launch_scores_dkdv_t<D, true, true>(m, lse, Dv, tiles, dk, dv, part, split, p, stream);
  }
}

}  // namespace fa
