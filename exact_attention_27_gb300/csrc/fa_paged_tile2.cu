// Attention of new tokens over a paged cache where sequences bring more than a
// few rows, at head dimensions 64, 96 and 128: items of 256 rows (tokens x
// grouped query heads), two tiles A and B of 128 that share each K and V tile,
// on the tcgen05 tensor cores.
//
// Same mathematics as fa_paged.cu (online softmax in base 2, lazy rescale of
// O), the division of work and the parts of fa_paged.cuh.  Bound by the tensor
// and exponential units: a 128 x 128 tile pair costs 1024 tensor cycles at d =
// 128 and 512 of the exponential unit; sharing keys between two tiles halves
// what is read from L2 (64 KB per 2 x 128 x 128 scores), and one tile's softmax
// runs while the tensor core works on the other's products.
//
// A CTA lives for the whole call: its items' key tiles form one sequence, and
// the first scores of an item are computed while the softmax warps still store
// the last one's O.
//
// Warp roles:
//   warps 0-3   softmax of tile A, warps 4-7 of tile B: thread t owns row t.
//               It also puts its row of Q into shared memory (a row's token and
//               head need not be a regular box): the next item's once its last
//               scores of this one are there, so before the epilogue.
//   warp 8      TMA producer: one box per page and 128-byte column block.
//   warp 9      MMA issuer and TMEM owner, per key tile:
//               O_A += P_A V, S_A of the next tile, O_B += P_B V, next S_B:
//               each S as soon as its tile's last one is used up.
//   the helpers (bf16 pages: warps 10 and 11; e4m3: warps 12-15, 10 and 11
//               being idle): V's rows past the last key made 0 (their p is 0,
//               but the page may hold anything there); e4m3 pages: K and V from
//               bytes to fp16 tiles, which both tiles then use.
// An item of at most 128 rows (single tokens, among chunks) has its rows in both
// tiles: A takes its even and B its odd key tiles, so that softmax and products
// still overlap, and A's warps join (O, m, l) of both, out of tensor memory.
// Registers: bf16 384 threads at 168: 224 / 224 / 56; e4m3 512 at 128: 200 /
// 200 / 56 / 56 (the sums are the launch totals 504 and 512).  The e4m3 kernels spill
// 68 to 124 bytes a thread at 128 registers, the bf16 ones 12.
//
// Tensor memory: S of tile x at columns 128 x (P, packed in pairs, over its
// first half), O at 256 + DP x.  A tile's next S follows its own O += P V.  The
// products of an item begin with tile A's, and wait for a P that A's warps make
// after the epilogue of the item before, so they overwrite no O still in use.
//
// Every wait is bounded (about a second); on expiry the kernel sets an error
// bit, every role skips its remaining work and the CTA exits.

#include <cuda.h>
#include <cuda_bf16.h>
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
struct Tile2Cfg {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int DP = (D + 63) / 64 * 64;  // whole 128-byte blocks of 16-bit values
  static constexpr int BM = 256;                 // rows of an item
  static constexpr int BN = 128;                 // keys of a tile
  static constexpr int SUB = DP / 64;
  static constexpr int BLOCK = 128 * 128;        // 128 rows x 128 bytes
  static constexpr int TILE = SUB * BLOCK;       // of Q (each of A and B), K or V
  static constexpr int NS = D == 64 ? 4 : 2;     // K and V stages each
  static constexpr int NR = !E4M3 ? 0 : D == 64 ? 4 : 2;  // e4m3 tiles as they come, K and V in turn
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + NS * TILE;
  static constexpr int OFF_RAW = OFF_V + NS * TILE;
  static constexpr int OFF_SCR = OFF_RAW + NR * BLOCK;
  static constexpr int OFF_ML = OFF_SCR + 40 * 8;  // [128] (m, l) of B's half of a split item
  static constexpr int OFF_BAR = OFF_ML + 128 * 8;
  static constexpr int HELPERS = E4M3 ? 4 : 2;   // warps
  static constexpr int B_QFULL = 0;              // [2] 4 warps
  static constexpr int B_KFULL = B_QFULL + 2;    // [NS] bytes (e4m3: the helpers)
  static constexpr int B_KEMPTY = B_KFULL + NS;
  static constexpr int B_VFULL = B_KEMPTY + NS;  // [NS] bytes (e4m3: not used)
  static constexpr int B_VEMPTY = B_VFULL + NS;
  static constexpr int B_VFIX = B_VEMPTY + NS;   // [NS] the helpers: V is whole and finite
  static constexpr int B_RFULL = B_VFIX + NS;    // [NR] bytes
  static constexpr int B_REMPTY = B_RFULL + NR;  // [NR] the helpers
  static constexpr int B_SFULL = B_REMPTY + NR;  // [2] S of tile x
  static constexpr int B_PFULL = B_SFULL + 2;    // [2] 4 warps
  static constexpr int B_ODONE = B_PFULL + 2;    // [2] O_x += P_x V
  static constexpr int B_SPLIT = B_ODONE + 2;    // 4 warps: B's half of a split item is final
  static constexpr int B_DRAIN = B_SPLIT + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(Tile2Cfg<D, E4M3>::THREADS, 1)
    fa_paged_tile2_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = Tile2Cfg<D, E4M3>;
  constexpr int BN = C::BN;
  // A key tile of an item of at most 128 rows (one product pair of half the size)
  // takes two thirds of another's time: half to nine tenths, by how much of it is
  // copies and conversion.  24 sequences, 3 chunks among single tokens, 16 / 4
  // heads, with 1:1, 3:2, 2:1: d = 64 46.4 / 41.0 / 40.0 us, d = 128 57.9 / 53.2 /
  // 57.6, e4m3 70.1 / 63.5 / 66.0; five e4m3 chunks 166 / 166 to 172 / 184.
  using Walk = PagedWalk<C::BM, BN, 2, 3, 2>;
  using Seg = PagedSegments<Walk>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::B_QFULL + x), 4);
      mbar_init(bar(C::B_SFULL + x), 1);
      mbar_init(bar(C::B_PFULL + x), 4);
      mbar_init(bar(C::B_ODONE + x), 1);
    }
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(C::B_KFULL + s), E4M3 ? C::HELPERS : 1);
      mbar_init(bar(C::B_KEMPTY + s), 1);
      mbar_init(bar(C::B_VFULL + s), 1);
      mbar_init(bar(C::B_VEMPTY + s), 1);
      mbar_init(bar(C::B_VFIX + s), C::HELPERS);
    }
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(bar(C::B_RFULL + s), 1);
      mbar_init(bar(C::B_REMPTY + s), C::HELPERS);
    }
    mbar_init(bar(C::B_SPLIT), 4);
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
    Seg first;
    if (!first.start(p, r)) return;  // block-uniform, nothing in flight
    __syncthreads();
    if (threadIdx.x == 0) {
      *reinterpret_cast<PagedRange*>(scratch) = r;
      *reinterpret_cast<Seg*>(scratch + 10) = first;
    }
  }
  static_assert(sizeof(PagedRange) <= 80 && sizeof(Seg) <= 240, "scratch");
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

  // Whether the item's rows fill one tile only, and its key tiles go in turn to A and B.
  auto split = [&](const Seg& s) -> bool { return Walk::half(p, s.w.g, s.w.rt); };

  if (warp >= 8) {
    reg_decrease<56>();
    if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      Seg seg = *reinterpret_cast<const Seg*>(scratch + 10);
      const int page = 1 << p.page_shift;
      const int box_rows = min(page, BN);
      constexpr int BLOCKS = E4M3 ? 1 : C::SUB;
      const bool mine = lane < BN / box_rows * BLOCKS;
      const int row0 = lane / BLOCKS * box_rows, sub = lane % BLOCKS;
      const uint32_t dst0 = sub * C::BLOCK + row0 * 128;
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
            const int i = 2 * nk, j = i + 1;  // as they come: K, then V
            if (i >= C::NR && !(ok = wait(bar(C::B_REMPTY + i % C::NR), ((i / C::NR) - 1) & 1)))
              break;
            copy(&tmK, sR + i % C::NR * C::BLOCK, bar(C::B_RFULL + i % C::NR), issue, key0,
                 seg.w.h, id);
            ++nk;
            if (j >= C::NR && !(ok = wait(bar(C::B_REMPTY + j % C::NR), ((j / C::NR) - 1) & 1)))
              break;
            copy(&tmV, sR + j % C::NR * C::BLOCK, bar(C::B_RFULL + j % C::NR), issue, key0,
                 seg.w.h, id);
            ++nv;
          } else {
            const int st = nk % C::NS;
            const uint32_t ph = ((nk / C::NS) - 1) & 1;
            if (nk >= C::NS && !(ok = wait(bar(C::B_KEMPTY + st), ph))) break;
            copy(&tmK, sK + st * C::TILE, bar(C::B_KFULL + st), issue, key0, seg.w.h, id);
            ++nk;
            if (nv >= C::NS && !(ok = wait(bar(C::B_VEMPTY + st), ph))) break;
            copy(&tmV, sV + st * C::TILE, bar(C::B_VFULL + st), issue, key0, seg.w.h, id);
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
        Seg seg = *reinterpret_cast<const Seg*>(scratch + 10);
        constexpr uint32_t ID_S = E4M3 ? idesc_f16_f32(128, BN, false)
                                       : idesc_bf16_f32(128, BN, false, false);
        constexpr uint32_t ID_O = E4M3 ? idesc_f16_f32(128, D, true)
                                       : idesc_bf16_f32(128, D, false, true);
        const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(sV, C::BLOCK, 1024);  // MN-major, N = D
        auto wait = [&](int b, uint32_t parity) {
          return mbar_wait(bar(b), parity, abort_flag, p.err, kErrTimeoutMma);
        };
        // Parities of the next Q (bits 0, 1) and P (bits 2, 3) of each tile; in
        // registers, as the issuer's own latency lies between P and O += P V.
        uint32_t phase = 0;
        // Products S, in order of the key tiles (A before B), run ahead of the
        // products P V, which follow in the same order: at most one S a tile is
        // waiting for its P.  job0 and job1 are those: bit 0 tile, bit 1 the item's
        // first of the tile, bit 2 the key tile's last use, key tile above.
        uint32_t job0 = 0, job1 = 0;
        int waiting = 0, v_tile = -1;
        bool have = true, sp = split(seg);
        int t = seg.t0, x = 0, n = 0;
        bool k_ready = false;
        auto issue_s = [&]() -> bool {
          const bool first = sp ? t - seg.t0 < 2 : t == seg.t0;
          const int st = n % C::NS;
          if (first) {
            if (!wait(C::B_QFULL + x, (phase >> x) & 1)) return false;
            phase ^= 1u << x;
          }
          if (!k_ready && !wait(C::B_KFULL + st, (n / C::NS) & 1)) return false;
          k_ready = true;
          tc_fence_after();
          const uint32_t d_tmem = tmem + x * 128;
          const uint64_t qd = desc_add(q_desc, x * C::TILE);
          const uint64_t kd = desc_add(k_desc, st * C::TILE);
          mma_ss_k<ID_S, 0>(d_tmem, qd, kd);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BLOCK + (kk & 3) * 32;
            mma_ss_k<ID_S, 1>(d_tmem, desc_add(qd, off), desc_add(kd, off));
          }
          mma_commit(bar(C::B_SFULL + x));
          const bool last = sp || x == 1;
          if (last) mma_commit(bar(C::B_KEMPTY + st));
          const uint32_t job = (static_cast<uint32_t>(n) << 3) | (last ? 4u : 0u) |
                               (first ? 2u : 0u) | static_cast<uint32_t>(x);
          if (waiting == 0)
            job0 = job;
          else
            job1 = job;
          ++waiting;
          // The next S: tile B of the same keys, or the next key tile.
          x ^= 1;
          if (last) {
            ++n;
            k_ready = false;
            if (++t == seg.t1) {
              have = seg.next(p);
              t = x = 0;
              sp = have && split(seg);
            }
          }
          return true;
        };
        bool ok = true;
        while (true) {
          while (ok && have && (waiting == 0 || (waiting == 1 && (job0 & 1) != static_cast<uint32_t>(x))))
            ok = issue_s();
          if (!ok || waiting == 0) break;
          const uint32_t job = job0;
          job0 = job1;
          --waiting;
          const int y = job & 1, tile = job >> 3, st = tile % C::NS;
          if (tile != v_tile) {
            ok = (E4M3 || wait(C::B_VFULL + st, (tile / C::NS) & 1)) &&
                 wait(C::B_VFIX + st, (tile / C::NS) & 1);
            v_tile = tile;
          }
          if (!ok || !(ok = wait(C::B_PFULL + y, (phase >> (2 + y)) & 1))) break;
          phase ^= 4u << y;
          tc_fence_after();
          const uint64_t vd = desc_add(v_desc, st * C::TILE);
          const uint32_t pa = tmem + y * 128;
          const uint32_t od = tmem + C::COL_O + y * C::DP;
          if (job & 2)
            mma_ts_k<ID_O, 0>(od, pa, vd);
          else
            mma_ts_k<ID_O, 1>(od, pa, vd);
#pragma unroll
          for (int kk = 1; kk < BN / 16; ++kk)
            mma_ts_k<ID_O, 1>(od, pa + kk * 8, desc_add(vd, kk * 2048));
          mma_commit(bar(C::B_ODONE + y));
          if (job & 4) mma_commit(bar(C::B_VEMPTY + st));
        }
        if (*abort_flag) {
          // Let the MMAs already issued finish before tensor memory is released.
          mma_commit(bar(C::B_DRAIN));
          mbar_wait_timed(bar(C::B_DRAIN), 0);
        }
      }
    } else if (warp >= (E4M3 ? 12 : 10)) {
      // ---------------------------------------------------------- helpers
      Seg seg = *reinterpret_cast<const Seg*>(scratch + 10);
      const int tid = threadIdx.x - 32 * (E4M3 ? 12 : 10);
      auto wait = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu,
                          mbar_wait(bar(b), parity, abort_flag, p.err, kErrTimeoutLoad)) != 0;
      };
      int n = 0;
      bool ok = true;
      do {
        for (int t = seg.t0; ok && t < seg.t1; ++t, ++n) {
          const int st = n % C::NS;
          const uint32_t ph = ((n / C::NS) - 1) & 1;
          const int keep = min(seg.keys - t * BN, BN);  // rows that are keys
          if constexpr (E4M3) {
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const int i = 2 * n + kv, rs = i % C::NR;
              ok = (n < C::NS || wait((kv ? C::B_VEMPTY : C::B_KEMPTY) + st, ph)) &&
                   wait(C::B_RFULL + rs, (i / C::NR) & 1);
              if (!ok) break;
              paged_convert<D, BN>(sR + rs * C::BLOCK, (kv ? sV : sK) + st * C::TILE, keep, tid);
              fence_proxy_async_smem();
              mbar_arrive_warp(bar(C::B_REMPTY + rs));
              mbar_arrive_warp(bar((kv ? C::B_VFIX : C::B_KFULL) + st));
            }
          } else {
            if (n >= C::NS && !(ok = wait(C::B_VEMPTY + st, ph))) break;
            if (keep < BN) {
              if (!(ok = wait(C::B_VFULL + st, (n / C::NS) & 1))) break;
              paged_zero_rows<C::SUB, BN, 64>(sV + st * C::TILE, max(keep, 0), tid);
              fence_proxy_async_smem();
            }
            mbar_arrive_warp(bar(C::B_VFIX + st));
          }
        }
      } while (ok && seg.next(p));
    }
  } else {
    // ------------------------------------------------------------ softmax (rows)
    if constexpr (E4M3)
      reg_increase<200>();
    else
      reg_increase<224>();
    Seg seg = *reinterpret_cast<const Seg*>(scratch + 10);
    const int x = warp >> 2;            // tile of this warpgroup
    const int row = threadIdx.x & 127;  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + x * 128;
    const uint32_t o_addr = tmem + lane_off + C::COL_O + x * C::DP;
    // Waits are made warp-uniform: the TMEM loads and stores are
    // warp-collective, so either every lane goes on or every lane stops.
    auto wait = [&](int b, uint32_t parity, uint32_t code) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, p.err, code)) != 0;
    };
    // The next item with work for this tile (the one at hand if it has): a
    // split item of one key tile has none for B.
    auto settle = [&](bool have) {
      while (have && x == 1 && split(seg) && seg.t1 - seg.t0 == 1) have = seg.next(p);
      return have;
    };
    auto load_q = [&](PagedRow& r) -> float {
      r = paged_row(p, seg, (split(seg) ? 0 : x * 128) + row);
      const float c = paged_load_q<D, E4M3>(p, r, sQ + x * C::TILE, row);
      fence_proxy_async_smem();
      mbar_arrive_warp(bar(C::B_QFULL + x));
      return c;
    };
    float2* half_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    bool have = settle(true), ok = true;
    PagedRow r{};
    float c = 0.0f;
    if (have) c = load_q(r);
    uint32_t n = 0;       // key tiles of this warpgroup
    uint32_t joins = 0;   // split items of both warpgroups
    while (have) {
      float m = -INFINITY;  // reference maximum, log2 domain
      float l = 0.0f;
      const bool sp = split(seg);
      const int t_first = sp ? seg.t0 + x : seg.t0;
      for (int t = t_first; t < seg.t1; t += sp ? 2 : 1, ++n) {
        if (!(ok = wait(C::B_SFULL + x, n & 1, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        bool moved;
        const float alpha = paged_softmax<BN, E4M3>(s_addr, t * BN + BN - 1 > r.all_see,
                                                    r.last - t * BN, c, m, l, moved);
        if (t > t_first && __any_sync(0xffffffffu, moved)) {
          // O is final before it is rescaled (S of this tile was issued after
          // O += P V of the one before, so this does not wait long).
          if (!(ok = wait(C::B_ODONE + x, (n - 1) & 1, kErrTimeoutSoftmax))) break;
          tc_fence_after();
          paged_rescale<D>(o_addr, alpha);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(C::B_PFULL + x));
      }
      if (!ok) break;
      // ---------------------------------------------------------- end of the item
      // Its last scores have been read, so Q's tile is free.
      const PagedRow now = r;
      const bool whole = seg.t0 == 0 && seg.t1 == seg.tiles;
      const bool both = sp && seg.t1 - seg.t0 > 1;
      const long long part =
          static_cast<long long>(cta * 2 + (seg.t0 == 0 ? 1 : 0)) * C::BM + (sp ? 0 : x * 128) + row;
      if (threadIdx.x == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
        p.notes[cta] = paged_note(p, *reinterpret_cast<const PagedRange*>(scratch), seg);
      have = settle(seg.next(p));
      if (have) c = load_q(r);
      if (!(ok = wait(C::B_ODONE + x, (n - 1) & 1, kErrTimeoutEpilogue))) break;
      tc_fence_after();
      if (!both) {
        paged_store_row<D, E4M3, false>(p, now, o_addr, 0, 1.0f, 0.0f, whole, part, m, l);
      } else if (x == 1) {
        half_ml[row] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive_warp(bar(C::B_SPLIT));
        ++joins;
      } else {
        if (!(ok = wait(C::B_SPLIT, joins++ & 1, kErrTimeoutEpilogue))) break;
        tc_fence_after();
        const float2 b = half_ml[row];
        const float m2 = fmaxf(m, b.x);
        const float ref = m2 == -INFINITY ? 0.0f : m2;
        const float fa = ex2_approx(m - ref), fb = ex2_approx(b.x - ref);
        paged_store_row<D, E4M3, true>(p, now, o_addr, o_addr + C::DP, fa, fb, whole, part, m2,
                                 l * fa + b.y * fb);
      }
      tc_fence_before();
      // The next item's first O products wait for P of tile A, which its warps
      // make after this: until then neither O, and no (m, l), is overwritten.
    }
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
  using C = Tile2Cfg<D, E4M3>;
  const cudaError_t e = set_smem_limit_once<fa_paged_tile2_kernel<D, E4M3>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_paged_tile2_kernel<D, E4M3>, dim3(ctas), dim3(C::THREADS),
                          C::SMEM_BYTES, stream, tk, tv, p);
}

template <bool E4M3>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int d,
                     int ctas, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_t<64, E4M3>(tk, tv, p, ctas, stream);
    case 96: return launch_t<96, E4M3>(tk, tv, p, ctas, stream);
    case 128: return launch_t<128, E4M3>(tk, tv, p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_tile2(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                               int d, bool e4m3, int ctas, cudaStream_t stream) {
  return e4m3 ? launch_d<true>(tk, tv, p, d, ctas, stream)
              : launch_d<false>(tk, tv, p, d, ctas, stream);
}

}  // namespace fa
