// dQ of attention with shaped scores (fa_scores.cuh says how); the other half of the backward,
// dK and dV, is in fa_scores_dkdv.cuh.
//
// One CTA owns 128 query rows of one (batch, query head) and walks the key tiles that the
// union of its rows' spans touches, as the forward does:
//   S_j  = Q K_j^T            tcgen05.mma, operands in shared memory
//   dP_j = dO V_j^T           tcgen05.mma
//   P = exp(x - L), dS = P o (1 - tanh^2) o (dP - D)      threads (x: the shaped score)
//   dQ  += dS K_j             tcgen05.mma, A = dS (bf16) from tensor memory
// and at the end dq = bf16(scale dQ): no atomics, so the bits repeat.
//
// D = rowsum(dO o O) is off by O's rounding to bf16, which shows in dS where the weights lie on
// few keys (|O| is then as large as |V|, and dP - D far smaller than D).  So a CTA with at most
// 1024 keys goes through them twice and sums D = sum_j P dP first, and leaves that D to the dK/dV
// kernel, which runs after this one.  (Errors relative to dq's norm, 0.0017 of which is its own
// rounding and as much dS's: three keys a row, slopes: 0.0055 -> 0.0024; packed documents of 100 to
// 2000 positions: 0.0026 -> 0.0024, for a third more of this kernel's time.  One of 8192 keys,
// causal: 1 % more.)  So does a head whose weights fall by e within 10 keys or fewer, however
// many it sees (slopes of 0.71, 0.35, 0.18, 0.09: 0.0031, 0.0028, 0.0027, 0.0025 otherwise).  A
// row that sees one key has dS = 0.
//
// Pipeline as in fa_bwd_dq.cu: S_j in one of two tensor-memory buffers, dP_j in one that the
// row warps hand back as soon as they hold its values, dS_j over the S columns they have
// read.  Sixteen row warps (eight at d = 256), a row's keys split between four (two), since L
// is known and no row reduction is needed.
//
// Warps: 0 .. WARPS - 1 query rows (warp w: rows 32 (w % 4).., key columns KH (w / 4)..), then
// TMA, and MMA issuer and tensor-memory owner.  Bound by issue and the FMA pipe with a cap
// (60 % and 35 % at 16 heads of 8192, d = 64: 320 us, uncapped 189), by the tensor core otherwise
// (70 % at d = 128: 264 us, 1.04 PFLOP/s; capped 345).

#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

constexpr float kSteep = 0.1f;  // slopes from here on: D is summed

// Head dimension D in {64, 96, 128, 256}; tiles are DP = D rounded up to a
// multiple of 64 columns wide (zero-filled past D), S and dP contract over the
// D real columns and dQ runs at N = D.
template <int D>
struct ScoreDqCfg {
  static constexpr int DP = (D + 63) / 64 * 64;  // padded head dimension
  static constexpr int BM = 128;                 // query rows per CTA
  static constexpr int BN = (D == 256) ? 64 : 128;  // keys per tile
  static constexpr int EXACT_TILES = 1024 / BN;
  static constexpr int KH = 32;                  // key columns per row warp
  static constexpr int GROUPS = BN / KH;         // row warps that share a row
  static constexpr int WARPS = 4 * GROUPS;       // row warps; then TMA and MMA
  static constexpr int SUB = DP / 64;
  static constexpr int QSUB = 128 * 128;         // 128 query rows x 64 bf16
  static constexpr int KSUB = BN * 128;          // BN key rows x 64 bf16
  static constexpr int QTILE = SUB * QSUB;
  static constexpr int KTILE = SUB * KSUB;
  // K_j is read by S_j and dQ_j, and S_{j+2} is issued right after dQ_j:
  // three K stages let K_{j+2} arrive while K_j and K_{j+1} are in use.
  // V_j is read by dP_j only.  At D = 256 (64 KB Q and dO tiles) two K
  // stages and one V stage are what fits.
  static constexpr int NSK = (D == 64) ? 4 : (D == 256 ? 2 : 3);
  static constexpr int NSV = (D == 64) ? 4 : (D == 256 ? 1 : 2);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = OFF_Q + QTILE;
  static constexpr int OFF_K = OFF_DO + QTILE;
  static constexpr int OFF_V = OFF_K + NSK * KTILE;
  static constexpr int OFF_BAR = OFF_V + NSV * KTILE;
  static constexpr int B_QD = 0;
  static constexpr int B_KFULL = 1;                // [NSK]
  static constexpr int B_KEMPTY = B_KFULL + NSK;   // [NSK]
  static constexpr int B_VFULL = B_KEMPTY + NSK;   // [NSV]
  static constexpr int B_VEMPTY = B_VFULL + NSV;   // [NSV]
  static constexpr int B_SFULL = B_VEMPTY + NSV;   // [2] S_j in S buffer j % 2
  static constexpr int B_DPFULL = B_SFULL + 2;     // dP_j in the dP buffer
  static constexpr int B_DPFREE = B_DPFULL + 1;    // dP_j read by every row warp
  static constexpr int B_DSREADY = B_DPFREE + 1;   // [2] dS_j in S buffer j % 2 (every row warp)
  static constexpr int B_DQDONE = B_DSREADY + 2;   // every dQ MMA done (completes once)
  static constexpr int B_DSUM = B_DQDONE + 1;      // the parts' sums of P dP (every row warp, twice)
  static constexpr int B_DRAIN = B_DSUM + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_SUM = OFF_MISC + 8 + 32;    // [2][BM] sums of P dP
  static constexpr int SMEM_BYTES = OFF_SUM + 2 * BM * 4 + 1024;
  static constexpr int THREADS = 32 * WARPS + 64;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S = 0, COL_DP = 2 * BN;  // S buffer b at COL_S + BN b
  static constexpr uint32_t COL_DQ = (D == 256) ? 256 : 384;
  static_assert(COL_DQ + DP <= TMEM_COLS, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct ScoreDqParams {
  ScoreParams s;
  const float* lse;
  float* Dvec;  // written where it is summed here
  __nv_bfloat16* dq;
  int n_qtiles, n_heads, heads_per_group;
  int before;  // query tiles that go before the others
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(ScoreDqCfg<D>::THREADS, 1)
    fa_scores_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmdO, const __grid_constant__ ScoreDqParams p) {
  using C = ScoreDqCfg<D>;
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
  // Same launch order as the forward: groups of heads, the last tiles first; but before them,
  // behind a long window, those that go through their few keys twice.
  const int per_group = p.heads_per_group * p.n_qtiles;
  const int grp = static_cast<int>(blockIdx.x) / per_group;
  const int rem = static_cast<int>(blockIdx.x) - grp * per_group;
  const int in_grp = min(p.heads_per_group, p.n_heads - grp * p.heads_per_group);
  const int qi_ = rem / in_grp;
  const int bh = grp * p.heads_per_group + (rem - qi_ * in_grp);
  const int qt = (qi_ < p.before ? p.before : p.n_qtiles + p.before) - 1 - qi_;
  const int b = bh / p.s.Hq;
  const int hq = bh - b * p.s.Hq;
  const int kvz = b * p.s.Hkv + hq / p.s.G;

  if (threadIdx.x == 0) {
    mbar_init(bar(C::B_QD), 1);
    for (int s = 0; s < C::NSK; ++s) {
      mbar_init(bar(C::B_KFULL + s), 1);
      mbar_init(bar(C::B_KEMPTY + s), 1);
    }
    for (int s = 0; s < C::NSV; ++s) {
      mbar_init(bar(C::B_VFULL + s), 1);
      mbar_init(bar(C::B_VEMPTY + s), 1);
    }
    for (int b2 = 0; b2 < 2; ++b2) {
      mbar_init(bar(C::B_SFULL + b2), 1);
      mbar_init(bar(C::B_DSREADY + b2), C::WARPS);
    }
    mbar_init(bar(C::B_DPFULL), 1);
    mbar_init(bar(C::B_DPFREE), C::WARPS);
    mbar_init(bar(C::B_DQDONE), 1);
    mbar_init(bar(C::B_DSUM), C::WARPS);
    mbar_init(bar(C::B_DRAIN), 1);
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
    span = row_span(p.s, b, qt * C::BM + (warp & 3) * 32 + static_cast<int>(threadIdx.x & 31));
    const KeySpan h = warp_hull(span);
    if (warp < 4 && (threadIdx.x & 31) == 0) hulls[warp] = h;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int lo = min(min(hulls[0].lo, hulls[1].lo), min(hulls[2].lo, hulls[3].lo));
  const int hi = max(max(hulls[0].hi, hulls[1].hi), max(hulls[2].hi, hulls[3].hi));
  const int j0 = hi > 0 ? lo / C::BN : 0;  // first key tile
  const int n_keys = hi > 0 ? (hi + C::BN - 1) / C::BN - j0 : 0;  // key tiles
  // Tiles gone through, v = 0 .. n_kv - 1; before n_sum D is summed.
  const bool steep = BIAS && p.s.slopes && fabsf(p.s.slopes[hq]) >= kSteep;
  const int n_sum = steep || n_keys <= C::EXACT_TILES ? n_keys : 0;
  const int n_kv = n_sum + n_keys;
  auto key_tile = [&](int v) -> int { return j0 + (v < n_sum ? v : v - n_sum); };

  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sdO = sbase + C::OFF_DO;
  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ TMA producer
    if (n_kv > 0 && elect_one()) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmdO);
      mbar_arrive_expect_tx(bar(C::B_QD), 2 * C::QTILE);
#pragma unroll
      for (int s = 0; s < C::SUB; ++s) {
        tma_load_3d(sQ + s * C::QSUB, &tmQ, bar(C::B_QD), 64 * s, qt * C::BM, bh);
        tma_load_3d(sdO + s * C::QSUB, &tmdO, bar(C::B_QD), 64 * s, qt * C::BM, bh);
      }
      // K_j then V_j, in the order the products need them (S_j comes before dP_j).
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n_kv; ++j) {
        const int sk = j % C::NSK;
        if (j >= C::NSK && !mbar_wait(bar(C::B_KEMPTY + sk), ((j / C::NSK) - 1) & 1, abort_flag,
                                      err, kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_KFULL + sk), C::KTILE);
#pragma unroll
        for (int s = 0; s < C::SUB; ++s)
          tma_load_3d(sK + sk * C::KTILE + s * C::KSUB, &tmK, bar(C::B_KFULL + sk), 64 * s,
                      key_tile(j) * C::BN, kvz);
        k_issued = j + 1;
        const int sv = j % C::NSV;
        if (j >= C::NSV && !mbar_wait(bar(C::B_VEMPTY + sv), ((j / C::NSV) - 1) & 1, abort_flag,
                                      err, kErrTimeoutLoad))
          break;
        mbar_arrive_expect_tx(bar(C::B_VFULL + sv), C::KTILE);
#pragma unroll
        for (int s = 0; s < C::SUB; ++s)
          tma_load_3d(sV + sv * C::KTILE + s * C::KSUB, &tmV, bar(C::B_VFULL + sv), 64 * s,
                      key_tile(j) * C::BN, kvz);
        v_issued = j + 1;
      }
      if (*abort_flag) {
        // Let the copies in flight land before the CTA exits.
        mbar_wait_timed(bar(C::B_QD), 0);
        for (int j = max(0, k_issued - C::NSK); j < k_issued; ++j)
          mbar_wait_timed(bar(C::B_KFULL + j % C::NSK), (j / C::NSK) & 1);
        for (int j = max(0, v_issued - C::NSV); j < v_issued; ++j)
          mbar_wait_timed(bar(C::B_VFULL + j % C::NSV), (j / C::NSV) & 1);
      }
    }
  } else if (warp == C::WARPS + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n_kv > 0 && elect_one()) {
      constexpr uint32_t ID_S = idesc_bf16_f32(128, C::BN, false, false);  // S, dP
      constexpr uint32_t ID_Q = idesc_bf16_f32(128, D, false, true);  // dQ (B = K MN-major), N = D
      const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t do_desc = smem_desc_sw128(sdO, 16, 1024);
      const uint64_t k_kmaj = smem_desc_sw128(sK, 16, 1024);
      const uint64_t v_kmaj = smem_desc_sw128(sV, 16, 1024);
      const uint64_t k_mn = smem_desc_sw128(sK, C::KSUB, 1024);
      bool ok = mbar_wait(bar(C::B_QD), 0, abort_flag, err, kErrTimeoutMma);
      // S_j = Q K_j^T into S buffer j % 2.
      auto issue_s = [&](int j) -> bool {
        const int sk = j % C::NSK;
        if (!mbar_wait(bar(C::B_KFULL + sk), (j / C::NSK) & 1, abort_flag, err, kErrTimeoutMma))
          return false;
        tc_fence_after();
        const uint32_t dst = tmem + C::COL_S + C::BN * (j & 1);
        const uint64_t kd = desc_add(k_kmaj, sk * C::KTILE);
        mma_ss_k<ID_S, 0>(dst, q_desc, kd);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk)
          mma_ss_k<ID_S, 1>(dst, desc_add(q_desc, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                            desc_add(kd, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        mma_commit(bar(C::B_SFULL + (j & 1)));
        return true;
      };
      // dP_j = dO V_j^T into the dP buffer.
      auto issue_dp = [&](int j) -> bool {
        const int sv = j % C::NSV;
        if (!mbar_wait(bar(C::B_VFULL + sv), (j / C::NSV) & 1, abort_flag, err, kErrTimeoutMma))
          return false;
        tc_fence_after();
        const uint64_t vd = desc_add(v_kmaj, sv * C::KTILE);
        mma_ss_k<ID_S, 0>(tmem + C::COL_DP, do_desc, vd);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk)
          mma_ss_k<ID_S, 1>(tmem + C::COL_DP,
                            desc_add(do_desc, (kk >> 2) * C::QSUB + (kk & 3) * 32),
                            desc_add(vd, (kk >> 2) * C::KSUB + (kk & 3) * 32));
        mma_commit(bar(C::B_DPFULL));
        mma_commit(bar(C::B_VEMPTY + sv));
        return true;
      };
      if (ok) ok = issue_s(0);
      if (ok) ok = issue_dp(0);
      if (ok && n_kv > 1) ok = issue_s(1);
      for (int j = 0; ok && j < n_kv; ++j) {
        // dP_{j+1} as soon as the row warps hold dP_j in registers.
        if (j + 1 < n_kv) {
          if (!mbar_wait(bar(C::B_DPFREE), j & 1, abort_flag, err, kErrTimeoutMma)) break;
          tc_fence_after();
          if (!issue_dp(j + 1)) break;
        }
        if (!mbar_wait(bar(C::B_DSREADY + (j & 1)), (j >> 1) & 1, abort_flag, err,
                       kErrTimeoutMma))
          break;
        tc_fence_after();
        // dQ += dS_j K_j.  dS of keys KH g.. sits packed (bf16 pairs) at
        // columns KH g.. of the S buffer, 16 keys = 8 columns per step; K_j
        // is read MN-major, 16 key rows (2 KB) per step.
        const int sk = j % C::NSK;
        const uint32_t sb = tmem + C::COL_S + C::BN * (j & 1);
        const uint64_t kmn = desc_add(k_mn, sk * C::KTILE);
        constexpr int KPW = C::KH / 16;  // 16-key steps per row warp's columns
        if (j >= n_sum) {
          if (j == n_sum)
            mma_ts_k<ID_Q, 0>(tmem + C::COL_DQ, sb, kmn);
          else
            mma_ts_k<ID_Q, 1>(tmem + C::COL_DQ, sb, kmn);
#pragma unroll
          for (int kk = 1; kk < C::BN / 16; ++kk)
            mma_ts_k<ID_Q, 1>(tmem + C::COL_DQ, sb + (kk / KPW) * C::KH + (kk % KPW) * 8,
                              desc_add(kmn, kk * 2048));
        }
        mma_commit(bar(C::B_KEMPTY + sk));
        // S_{j+2} reuses this S buffer; the products run in issue order, so it
        // overwrites dS_j only after dQ_j has read it.
        if (j + 2 < n_kv && !issue_s(j + 2)) break;
        // Once, after the last tile: a barrier that completed once per tile
        // could not tell its last phase from an earlier one by parity alone.
        if (j == n_kv - 1) mma_commit(bar(C::B_DQDONE));
      }
      if (*abort_flag) {
        mma_commit(bar(C::B_DRAIN));
        mbar_wait_timed(bar(C::B_DRAIN), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ query rows
    // Warp w reads tensor-memory lanes 32 (w % 4) .. +31 (its query rows)
    // and key columns KH (w / 4) .. of each tile.
    const int wq = warp & 3, g = warp >> 2;
    const int row = wq * 32 + static_cast<int>(threadIdx.x & 31);
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const int qi = qt * C::BM + row;
    const bool live = qi < p.s.Nq;
    const size_t ridx = static_cast<size_t>(bh) * p.s.Nq + (live ? qi : 0);
    const bool sees = span.hi > 0;
    const float L2 = sees ? p.lse[ridx] * kScoreLog2e : INFINITY;  // no key seen: P = 0
    float Drow = sees && n_sum == 0 ? p.Dvec[ridx] : 0.0f;
    const float slope2 = BIAS && p.s.slopes ? p.s.slopes[hq] * kScoreLog2e : 0.0f;
    uint64_t nd2 = f2_pack(-Drow, -Drow);
    float* sums = reinterpret_cast<float*>(smem + C::OFF_SUM);
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_SFULL + (j & 1)), (j >> 1) & 1, abort_flag,
                                             err, kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      const uint32_t scol = C::COL_S + C::BN * (j & 1) + C::KH * g;
      constexpr int KH = C::KH;
      const int kbase = key_tile(j) * C::BN + KH * g;
      const bool need_mask = __any_sync(0xffffffffu, span.lo > kbase || span.hi < kbase + KH);
      const unsigned from = static_cast<unsigned>(span.lo - kbase);
      const int n_seen = span.hi - span.lo;
      const float dist0 = static_cast<float>(p.s.q_offset + qi - kbase);
      // A row of one key has P = 1 and dP = D, so dS = 0.
      const unsigned len = n_seen > 1 || j < n_sum ? static_cast<unsigned>(n_seen) : 0u;
      // What dP - D is multiplied by (dP where D is summed), from S alone: dP is asked for last,
      // so that it is there, and its columns are handed back at once.
      float w[KH];
      load_scores(tmem + lane_off + scol, w);
      // CH columns at a time: all, or half of them where the tanh's derivative and the distances
      // both take registers (96 a thread; both passes of 16 heads of 8192, d = 64: cap 946 us in
      // halves, 932 at once, with slopes too 1098 and 1136).
      constexpr int CH = CAP && BIAS ? KH / 2 : KH;
#pragma unroll
      for (int c0 = 0; c0 < KH; c0 += CH) {
        float(&x)[CH] = *reinterpret_cast<float(*)[CH]>(&w[c0]);
        float gr[CAP ? CH : 1];
        shape_scores<CH, CAP, BIAS, CAP>(x, gr, p.s.f, slope2, dist0 - c0, L2,
                                         [&](float (&y)[CH], int) {
                                           load_scores(tmem + lane_off + scol + c0, y);
                                         });
#pragma unroll
        for (int t = 0; t < CH; t += 2) {
          uint64_t v = f2_pack(ex2_approx(x[t]), ex2_approx(x[t + 1]));
          if constexpr (CAP)
            if (j >= n_sum) v = f2_mul(v, f2_pack(gr[t], gr[t + 1]));
          f2_unpack(v, x[t], x[t + 1]);
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DPFULL), j & 1, abort_flag, err,
                                             kErrTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t dpv[KH];
      tmem_ld32(tmem + lane_off + C::COL_DP + KH * g, dpv);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_DPFREE));
      if (j < n_sum) {
        // D = sum of P dP, over all parts of the row's keys.
#pragma unroll
        for (int t = 0; t < KH; ++t)
          if (static_cast<unsigned>(t) - from < len)
            Drow = fmaf(w[t], __uint_as_float(dpv[t]), Drow);
        mbar_arrive_warp(bar(C::B_DSREADY + (j & 1)));
        if (j == n_sum - 1) {
          // The row's parts join: groups 2 and 3 hand theirs to 0 and 1, which all then add.
          if (g >= 2) sums[(g - 2) * C::BM + row] = Drow;
          mbar_arrive_warp(bar(C::B_DSUM));
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DSUM), 0, abort_flag, err,
                                                 kErrTimeoutSoftmax));
          if (!ok) break;
          if (g < 2) sums[g * C::BM + row] = Drow + (C::GROUPS > 2 ? sums[g * C::BM + row] : 0.0f);
          mbar_arrive_warp(bar(C::B_DSUM));
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DSUM), 1, abort_flag, err,
                                                 kErrTimeoutSoftmax));
          if (!ok) break;
          Drow = sums[row] + sums[C::BM + row];
          nd2 = f2_pack(-Drow, -Drow);
          if (g == 0 && sees) p.Dvec[ridx] = Drow;
        }
        continue;
      }
#pragma unroll
      for (int t = 0; t < KH; t += 2)
        f2_unpack(f2_mul(f2_pack(w[t], w[t + 1]),
                         f2_add(f2_pack(__uint_as_float(dpv[t]), __uint_as_float(dpv[t + 1])),
                                nd2)),
                  w[t], w[t + 1]);
      if (need_mask) {
#pragma unroll
        for (int t = 0; t < KH; ++t)
          if (static_cast<unsigned>(t) - from >= len) w[t] = 0.0f;
      }
      uint32_t pk[KH / 2];
#pragma unroll
      for (int u = 0; u < KH / 2; ++u) pk[u] = pack_bf16x2(w[2 * u], w[2 * u + 1]);
      // dS (bf16 pairs) over S columns this warp has already read.
      tmem_st16(tmem + lane_off + scol, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(bar(C::B_DSREADY + (j & 1)));
    }
    // ---- epilogue: dq = bf16(scale dQ), one row per thread, 32-column
    // chunks split between the warps of a row
    if (ok && n_kv > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DQDONE), 0, abort_flag, err,
                                             kErrTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* qrow = p.dq + ridx * D;
#pragma unroll 1
      for (int q4 = g; q4 < D / 32; q4 += C::GROUPS) {
        uint32_t r[32];
        if (n_kv > 0) {
          tmem_ld32(tmem + lane_off + C::COL_DQ + q4 * 32, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) r[u] = 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          pk[u] = pack_bf16x2(__uint_as_float(r[2 * u]) * p.s.scale,
                              __uint_as_float(r[2 * u + 1]) * p.s.scale);
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(qrow + q4 * 32);
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
cudaError_t launch_scores_dq_t(const ScoreMaps& m, const float* lse, float* Dv, void* dq,
                               const ScoreParams& s, cudaStream_t stream) {
  using C = ScoreDqCfg<D>;
  auto kern = fa_scores_dq_kernel<D, CAP, BIAS>;
  cudaError_t e = set_smem_limit_once<fa_scores_dq_kernel<D, CAP, BIAS>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  ScoreDqParams p;
  p.s = s;
  p.lse = lse;
  p.Dvec = Dv;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.n_qtiles = (s.Nq + C::BM - 1) / C::BM;
  p.n_heads = s.B * s.Hq;
  p.heads_per_group = static_cast<int>(heads_per_group(s.Nk, D, 2.0, s.G, p.n_heads));
  // (8 heads of 4000, d = 256, cap, window 1024: 78 us instead of 97)
  constexpr int kFew = C::EXACT_TILES * C::BN;
  p.before = 0;
  if (s.causal && s.window > kFew - C::BM)
    p.before = std::min(std::max(kFew - s.q_offset, 0) / C::BM, p.n_qtiles);
  const long long grid = static_cast<long long>(p.n_heads) * p.n_qtiles;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(C::THREADS),
                          C::SMEM_BYTES, stream, m.q, m.k, m.v, m.dO, p);
}

}  // namespace

template <int D>
cudaError_t launch_scores_dq(const ScoreMaps& m, const float* lse, float* Dv, void* dq,
                             const ScoreParams& p, int mode, cudaStream_t stream) {
  switch (mode) {
    case kScorePlain: return launch_scores_dq_t<D, false, false>(m, lse, Dv, dq, p, stream);
    case kScoreBias: return launch_scores_dq_t<D, false, true>(m, lse, Dv, dq, p, stream);
    case kScoreCap: return launch_scores_dq_t<D, true, false>(m, lse, Dv, dq, p, stream);
    default: return launch_scores_dq_t<D, true, true>(m, lse, Dv, dq, p, stream);
  }
}

}  // namespace fa
