// Attention of new tokens over a paged cache where sequences bring more than a
// few rows, at head dimension 256: tiles of 128 rows (tokens x grouped query
// heads) on the tcgen05 tensor cores.  (At d = 64, 96 and 128 two such tiles
// share the keys: fa_paged_tile2.cu.  Here a 128 x 256 Q tile is 64 KB and its
// fp32 O takes 256 of the 512 TMEM columns.)
//
// Same mathematics as fa_paged.cu (online softmax in base 2, lazy rescale of
// O), the division of work and the parts of fa_paged.cuh, with key tiles of 64.
// A CTA lives for the whole call: its items' key tiles form
// one sequence n = 0, 1, ..., and S_{n+1} and S_{n+2} are computed, across the
// end of an item too, while the softmax works on S_n.
//
// Warp roles (384 threads, three warpgroups):
//   warps 0-3   softmax: thread t owns row t of the item; epilogue.
//   warps 4-7   Q of each item into shared memory (thread t row t: a row's
//               token and head need not be a regular box), and V's rows past the
//               last key made 0: their p is 0, but the page may hold anything
//               there.  e4m3 pages: also K and V from bytes to fp16 tiles.
//   warp 8      TMA producer: one box per page and 128-byte column block.
//   warp 9      MMA issuer and TMEM owner: S_0, S_1, then per tile n:
//               O += P_n V_n, S_{n+2} into buffer (n+2) mod 3.
//   warps 10-11 idle (they complete the warpgroup).
// Registers: launched at 168 a thread; 240 / 160 / 104 (their sum is 3 x 168).
//
// Tensor memory: S buffers b = 0, 1, 2 at columns BN b (P, packed in pairs,
// over the first half of its S), O at 512 - DP.
//
// Order.  S_n lies in buffer n mod 3, which S_{n+3} overwrites; that is issued
// after O += P_{n+1} V_{n+1}, so after P_n was read.  O is first written for an
// item by its first product, which waits for a P that the softmax makes after
// the epilogue of the item before.
//
// e4m3 pages: as in fa_paged.cu, K and V as fp16 (exact), P as fp16 up to 2^15, Q as
// fp16 with a power of two taken out of each row.
//
// Every wait is bounded (about a second); on expiry the kernel sets an error
// bit, every role skips its remaining work and the CTA exits.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_paged_host.h"
#include "fa_paged_tile.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

template <int D_, bool E4M3_>
struct TileCfg {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int DP = (D + 63) / 64 * 64;    // whole 128-byte blocks of 16-bit values
  static constexpr int BM = 128;                   // rows of an item
  static constexpr int BN = 64;                    // keys of a tile
  static constexpr int SUB = DP / 64;
  static constexpr int Q_BLOCK = BM * 128;
  static constexpr int KV_BLOCK = BN * 128;
  static constexpr int Q_TILE = SUB * Q_BLOCK;
  static constexpr int KV_TILE = SUB * KV_BLOCK;
  static constexpr int NQ = 1;                     // Q tiles (shared memory has room for one)
  static constexpr int NS = 2;                     // K and V stages each
  // e4m3 bytes as they come: K and V tiles in turn.
  static constexpr int RSUB = (D + 127) / 128;
  static constexpr int RAW_TILE = E4M3 ? RSUB * KV_BLOCK : 0;
  static constexpr int NR = E4M3 ? 2 : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQ * Q_TILE;
  static constexpr int OFF_V = OFF_K + NS * KV_TILE;
  static constexpr int OFF_RAW = OFF_V + NS * KV_TILE;
  static constexpr int OFF_SCALE = OFF_RAW + NR * RAW_TILE;  // [NQ][128] scale of a row's scores
  static constexpr int OFF_SCR = OFF_SCALE + NQ * BM * 4;
  static constexpr int OFF_BAR = OFF_SCR + 40 * 8;
  static constexpr int NB = 3;                     // S buffers
  static constexpr int B_QFULL = 0;                // [NQ] 4 warps
  static constexpr int B_QEMPTY = B_QFULL + NQ;    // [NQ] the item's last S, and 4 softmax warps
  static constexpr int B_KFULL = B_QEMPTY + NQ;    // [NS] bytes (e4m3: 4 warps)
  static constexpr int B_KEMPTY = B_KFULL + NS;
  static constexpr int B_VFULL = B_KEMPTY + NS;    // [NS] bytes (e4m3: not used)
  static constexpr int B_VEMPTY = B_VFULL + NS;
  static constexpr int B_VFIX = B_VEMPTY + NS;     // [NS] 4 warps: V is whole and finite
  static constexpr int B_RFULL = B_VFIX + NS;      // [NR] bytes
  static constexpr int B_REMPTY = B_RFULL + NR;    // [NR] 4 warps
  static constexpr int B_SFULL = B_REMPTY + NR;    // [NB]
  static constexpr int B_PFULL = B_SFULL + NB;     // [NB] 4 warps
  static constexpr int B_ODONE = B_PFULL + NB;     // O += P_n V_n
  static constexpr int B_FINAL = B_ODONE + 1;      // an item's last product
  static constexpr int B_DRAIN = B_FINAL + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 384;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 512 - DP;
  static_assert(NB * BN <= 512 - DP, "tensor memory");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(384, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = TileCfg<D, E4M3>;
  constexpr int BN = C::BN;
  using Walk = PagedWalk<C::BM, BN, 2>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(bar(C::B_QFULL + i), 4);
      mbar_init(bar(C::B_QEMPTY + i), 5);
    }
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(C::B_KFULL + s), E4M3 ? 4 : 1);
      mbar_init(bar(C::B_KEMPTY + s), 1);
      mbar_init(bar(C::B_VFULL + s), 1);
      mbar_init(bar(C::B_VEMPTY + s), 1);
      mbar_init(bar(C::B_VFIX + s), 4);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(bar(C::B_RFULL + s), 1);
      mbar_init(bar(C::B_REMPTY + s), 4);
    }
    for (int x = 0; x < C::NB; ++x) {
      mbar_init(bar(C::B_SFULL + x), 1);
      mbar_init(bar(C::B_PFULL + x), 4);
    }
    mbar_init(bar(C::B_ODONE), 1);
    mbar_init(bar(C::B_FINAL), 1);
    mbar_init(bar(C::B_DRAIN), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8 && elect_one()) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_launch_dependents();
  grid_dependency_wait();
  long long* scratch = reinterpret_cast<long long*>(smem + C::OFF_SCR);
  const int cta = blockIdx.x;
  {
    // The roles take their start from shared memory: registers that live
    // across the change of the register budgets would be spilled.
    const PagedRange r = paged_range<Walk, C::THREADS>(p, scratch);
    if (threadIdx.x == 0) p.notes[cta].last = -1;
    PagedSegments<Walk> first;
    if (!first.start(p, r)) return;  // block-uniform, nothing in flight
    __syncthreads();
    if (threadIdx.x == 0) {
      *reinterpret_cast<PagedRange*>(scratch) = r;
      *reinterpret_cast<PagedSegments<Walk>*>(scratch + 10) = first;
    }
  }
  static_assert(sizeof(PagedRange) <= 80 && sizeof(PagedSegments<Walk>) <= 240, "scratch");
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sQ = sbase + C::OFF_Q;
  const uint32_t sK = sbase + C::OFF_K;
  const uint32_t sV = sbase + C::OFF_V;
  const uint32_t sR = sbase + C::OFF_RAW;
  float* q_scale = reinterpret_cast<float*>(smem + C::OFF_SCALE);

  if (warp >= 8) {
    reg_decrease<104>();
    if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      PagedSegments<Walk> seg = *reinterpret_cast<const PagedSegments<Walk>*>(scratch + 10);
      const int page = 1 << p.page_shift;
      const int box_rows = min(page, BN);
      constexpr int BLOCKS = E4M3 ? C::RSUB : C::SUB;
      const bool mine = lane < BN / box_rows * BLOCKS;
      const int row0 = lane / BLOCKS * box_rows, sub = lane % BLOCKS;
      const uint32_t dst0 = sub * C::KV_BLOCK + row0 * 128;
      // Copies the lanes' boxes of one tile; `full` counts their bytes.
      auto copy = [&](const CUtensorMap* tm, uint32_t dst, uint32_t full, bool issue, int key0,
                      int head, int id) {
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, issue));
        if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_rows * 128);
        __syncwarp();
        if (issue) tma_load_4d(dst + dst0, tm, full, sub * 128, key0 & (page - 1), head, id);
      };
      auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err, kErrTimeoutLoad)) !=
               0;
      };
      int nk = 0, nv = 0;  // K and V tiles issued
      bool ok = true;
      do {
        for (int t = seg.t0; ok && t < seg.t1; ++t) {
          const int key0 = t * BN + row0;
          bool issue = mine && key0 < seg.keys;
          int id = 0;
          if (issue) {
            id = p.table[seg.w.s * p.table_stride + (key0 >> p.page_shift)];
            if (id < 0 || id >= p.n_pages) {
              atomicOr(p.err, kErrBadPage);
              issue = false;
            }
          }
          if constexpr (E4M3) {
            const int i = 2 * nk, j = i + 1;  // raw tiles: K, then V
            if (i >= C::NR && !(ok = wait(bar(C::B_REMPTY + i % C::NR), ((i / C::NR) - 1) & 1)))
              break;
            copy(&tmK, sR + i % C::NR * C::RAW_TILE, bar(C::B_RFULL + i % C::NR), issue, key0,
                 seg.w.h, id);
            ++nk;
            if (j >= C::NR && !(ok = wait(bar(C::B_REMPTY + j % C::NR), ((j / C::NR) - 1) & 1)))
              break;
            copy(&tmV, sR + j % C::NR * C::RAW_TILE, bar(C::B_RFULL + j % C::NR), issue, key0,
                 seg.w.h, id);
            ++nv;
          } else {
            const int st = nk % C::NS;
            const uint32_t ph = ((nk / C::NS) - 1) & 1;
            if (nk >= C::NS && !(ok = wait(bar(C::B_KEMPTY + st), ph))) break;
            copy(&tmK, sK + st * C::KV_TILE, bar(C::B_KFULL + st), issue, key0, seg.w.h, id);
            ++nk;
            if (nv >= C::NS && !(ok = wait(bar(C::B_VEMPTY + st), ph))) break;
            copy(&tmV, sV + st * C::KV_TILE, bar(C::B_VFULL + st), issue, key0, seg.w.h, id);
            ++nv;
          }
        }
      } while (ok && seg.next(p));
      if (*abort_flag) {
        // Let the copies already issued land before the CTA's memory is released.
        if constexpr (E4M3) {
          for (int i = max(0, nk + nv - C::NR); i < nk + nv; ++i)
            mbar_wait_timed(bar(C::B_RFULL + i % C::NR), (i / C::NR) & 1);
        } else {
          for (int i = max(0, nk - C::NS); i < nk; ++i)
            mbar_wait_timed(bar(C::B_KFULL + i % C::NS), (i / C::NS) & 1);
          for (int i = max(0, nv - C::NS); i < nv; ++i)
            mbar_wait_timed(bar(C::B_VFULL + i % C::NS), (i / C::NS) & 1);
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        PagedSegments<Walk> seg = *reinterpret_cast<const PagedSegments<Walk>*>(scratch + 10);
        constexpr uint32_t ID_S = E4M3 ? idesc_f16_f32(128, BN, false)
                                       : idesc_bf16_f32(128, BN, false, false);
        constexpr uint32_t ID_O = E4M3 ? idesc_f16_f32(128, D, true)
                                       : idesc_bf16_f32(128, D, false, true);
        const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(sV, C::KV_BLOCK, 1024);  // MN-major, N = D
        auto wait = [&](int b, uint32_t parity) {
          return mbar_wait(bar(b), parity, abort_flag, p.err, kErrTimeoutMma);
        };
        // The S products run two tiles ahead of the P V products.
        PagedSegments<Walk> ahead = seg;
        bool more = true;  // S products are left
        int ta = ahead.t0, na = 0, ia = 0;  // its tile, running number, item
        auto issue_s = [&]() -> bool {
          const int st = na % C::NS, qs = ia % C::NQ;
          if (ta == ahead.t0 && !wait(C::B_QFULL + qs, (ia / C::NQ) & 1)) return false;
          if (!wait(C::B_KFULL + st, (na / C::NS) & 1)) return false;
          tc_fence_after();
          const uint32_t d_tmem = tmem + (na % C::NB) * BN;
          const uint64_t qd = desc_add(q_desc, qs * C::Q_TILE);
          const uint64_t kd = desc_add(k_desc, st * C::KV_TILE);
          mma_ss_k<ID_S, 0>(d_tmem, qd, kd);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk)
            mma_ss_k<ID_S, 1>(d_tmem, desc_add(qd, (kk >> 2) * C::Q_BLOCK + (kk & 3) * 32),
                              desc_add(kd, (kk >> 2) * C::KV_BLOCK + (kk & 3) * 32));
          mma_commit(bar(C::B_SFULL + na % C::NB));
          mma_commit(bar(C::B_KEMPTY + st));
          ++na;
          if (++ta == ahead.t1) {
            mma_commit(bar(C::B_QEMPTY + qs));
            more = ahead.next(p);
            ta = 0;
            ++ia;
          }
          return true;
        };
        bool ok = issue_s();
        if (ok && more) ok = issue_s();
        int n = 0;
        do {
          for (int t = seg.t0; ok && t < seg.t1; ++t, ++n) {
            const int st = n % C::NS, bf = n % C::NB;
            ok = (E4M3 || wait(C::B_VFULL + st, (n / C::NS) & 1)) &&
                 wait(C::B_VFIX + st, (n / C::NS) & 1) && wait(C::B_PFULL + bf, (n / C::NB) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd = desc_add(v_desc, st * C::KV_TILE);
            const uint32_t pa = tmem + bf * BN;
            if (t == seg.t0)
              mma_ts_k<ID_O, 0>(tmem + C::COL_O, pa, vd);
            else
              mma_ts_k<ID_O, 1>(tmem + C::COL_O, pa, vd);
#pragma unroll
            for (int kk = 1; kk < BN / 16; ++kk)
              mma_ts_k<ID_O, 1>(tmem + C::COL_O, pa + kk * 8, desc_add(vd, kk * 2048));
            mma_commit(bar(C::B_ODONE));
            mma_commit(bar(C::B_VEMPTY + st));
            if (t == seg.t1 - 1) mma_commit(bar(C::B_FINAL));
            if (more) ok = issue_s();
          }
        } while (ok && seg.next(p));
        if (*abort_flag) {
          // Let the MMAs already issued finish before tensor memory is released.
          mma_commit(bar(C::B_DRAIN));
          mbar_wait_timed(bar(C::B_DRAIN), 0);
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ Q, V's tail, conversion
    reg_decrease<160>();
    PagedSegments<Walk> seg = *reinterpret_cast<const PagedSegments<Walk>*>(scratch + 10);
    const int row = threadIdx.x & 127;
    auto wait = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu,
                        mbar_wait(bar(b), parity, abort_flag, p.err, kErrTimeoutLoad)) != 0;
    };
    // Q of item `i` (segment s): row `row`, zeros past the sequence's rows.
    auto load_q = [&](const PagedSegments<Walk>& s, int i) -> bool {
      const int qs = i % C::NQ;
      if (i >= C::NQ && !wait(C::B_QEMPTY + qs, ((i / C::NQ) - 1) & 1)) return false;
      q_scale[qs * C::BM + row] =
          paged_load_q<D, E4M3>(p, paged_row(p, s, row), sQ + qs * C::Q_TILE, row);
      fence_proxy_async_smem();
      mbar_arrive_warp(bar(C::B_QFULL + qs));
      return true;
    };
    int n = 0, i = 0;
    bool ok = load_q(seg, 0), more = true;
    do {
      for (int t = seg.t0; ok && t < seg.t1; ++t, ++n) {
        const int st = n % C::NS;
        const uint32_t ph = ((n / C::NS) - 1) & 1;
        const int keep = min(seg.keys - t * BN, BN);  // rows that are keys
        if constexpr (E4M3) {
          for (int kv = 0; kv < 2 && ok; ++kv) {
            const int x = 2 * n + kv, rs = x % C::NR;
            ok = (n < C::NS || wait((kv ? C::B_VEMPTY : C::B_KEMPTY) + st, ph)) &&
                 wait(C::B_RFULL + rs, (x / C::NR) & 1);
            if (!ok) break;
            paged_convert<D, BN>(sR + rs * C::RAW_TILE, (kv ? sV : sK) + st * C::KV_TILE, keep, row);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(C::B_REMPTY + rs));
            mbar_arrive_warp(bar((kv ? C::B_VFIX : C::B_KFULL) + st));
          }
        } else {
          if (n >= C::NS && !(ok = wait(C::B_VEMPTY + st, ph))) break;
          if (keep < BN) {
            if (!(ok = wait(C::B_VFULL + st, (n / C::NS) & 1))) break;
            paged_zero_rows<C::SUB, BN, 128>(sV + st * C::KV_TILE, max(keep, 0), row);
            fence_proxy_async_smem();
          }
          mbar_arrive_warp(bar(C::B_VFIX + st));
        }
      }
      if (!ok) break;
      ++i;
      more = seg.next(p);
      if (more) ok = load_q(seg, i);
    } while (ok && more);
  } else {
    // ------------------------------------------------------------ softmax (rows)
    reg_increase<240>();
    PagedSegments<Walk> seg = *reinterpret_cast<const PagedSegments<Walk>*>(scratch + 10);
    const int row = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    // Waits are made warp-uniform: the TMEM loads and stores are
    // warp-collective, so either every lane goes on or every lane stops.
    auto wait = [&](int b, uint32_t parity, uint32_t code) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, p.err, code)) != 0;
    };
    int n = 0, i = 0;
    bool ok = true;
    do {
      const PagedRow x = paged_row(p, seg, row);
      const int qs = i % C::NQ;
      if (!(ok = wait(C::B_QFULL + qs, (i / C::NQ) & 1, kErrTimeoutSoftmax))) break;
      const float c = q_scale[qs * C::BM + row];
      mbar_arrive_warp(bar(C::B_QEMPTY + qs));
      float m_used = -INFINITY;  // reference maximum, log2 domain
      float l = 0.0f;
      for (int t = seg.t0; t < seg.t1; ++t, ++n) {
        const int bf = n % C::NB;
        const uint32_t col_s = bf * BN;
        if (!(ok = wait(C::B_SFULL + bf, (n / C::NB) & 1, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        bool upd;
        const float alpha =
            paged_softmax<BN, E4M3>(tmem + lane_off + col_s, t * BN + BN - 1 > x.all_see,
                                    x.last - t * BN, c, m_used, l, upd);
        if (t > seg.t0 && __any_sync(0xffffffffu, upd)) {
          // O is final before it is rescaled: S_n implies O += P_{n-2} V_{n-2},
          // so the barrier is at most one phase behind.
          if (!(ok = wait(C::B_ODONE, (n - 1) & 1, kErrTimeoutSoftmax))) break;
          tc_fence_after();
          paged_rescale<D>(tmem + lane_off + C::COL_O, alpha);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(C::B_PFULL + bf));
      }
      if (!ok || !(ok = wait(C::B_FINAL, i & 1, kErrTimeoutEpilogue))) break;
      // ---------------------------------------------------------- end of the item
      tc_fence_after();
      const int slot = cta * 2 + (seg.t0 == 0 ? 1 : 0);
      paged_store_row<D, E4M3, false>(p, x, tmem + lane_off + C::COL_O, 0, 1.0f, 0.0f,
                                seg.t0 == 0 && seg.t1 == seg.tiles,
                                static_cast<long long>(slot) * C::BM + row, m_used, l);
      if (row == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
        p.notes[cta] = paged_note(p, *reinterpret_cast<const PagedRange*>(scratch), seg);
      // (The next item's first O product follows this thread's next P, after a fence.)
      ++i;
    } while (seg.next(p));
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool E4M3>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int ctas,
                     cudaStream_t stream) {
  using C = TileCfg<D, E4M3>;
  const cudaError_t e = set_smem_limit_once<fa_paged_tile_kernel<D, E4M3>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_paged_tile_kernel<D, E4M3>, dim3(ctas), dim3(C::THREADS),
                          C::SMEM_BYTES, stream, tk, tv, p);
}

}  // namespace

cudaError_t launch_paged_tile(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                              bool e4m3, int ctas, cudaStream_t stream) {
  return e4m3 ? launch_t<256, true>(tk, tv, p, ctas, stream)
              : launch_t<256, false>(tk, tv, p, ctas, stream);
}

}  // namespace fa
