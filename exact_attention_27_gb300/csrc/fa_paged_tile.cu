// Attention of new tokens over a paged cache where sequences bring more than a
// few rows: tiles of 128 rows (tokens x grouped query heads) on the tcgen05
// tensor cores.
//
// Same mathematics as fa_paged.cu (online softmax in base 2, lazy rescale of
// O), the division of work and the parts of fa_paged.cuh, with key tiles of 128
// (64 at d = 256).  A CTA lives for the whole call: its items' key tiles form
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
// e4m3 pages: as in fa_paged.cu, K and V as fp16 (exact), P as fp16, Q as fp16
// with a power of two taken out of each row.
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
#include "fa_paged_launch.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kRescaleThreshold = 8.0f;

template <int D_, bool E4M3_>
struct TileCfg {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int DP = (D + 63) / 64 * 64;    // whole 128-byte blocks of 16-bit values
  static constexpr int BM = 128;                   // rows of an item
  static constexpr int BN = D == 256 ? 64 : 128;   // keys of a tile
  static constexpr int SUB = DP / 64;
  static constexpr int Q_BLOCK = BM * 128;
  static constexpr int KV_BLOCK = BN * 128;
  static constexpr int Q_TILE = SUB * Q_BLOCK;
  static constexpr int KV_TILE = SUB * KV_BLOCK;
  static constexpr int NQ = D == 256 || (E4M3 && D != 64) ? 1 : 2;  // Q tiles
  static constexpr int NS = D == 64 ? 4 : 2;                        // K and V stages each
  // e4m3 bytes as they come: K and V tiles in turn.
  static constexpr int RSUB = (D + 127) / 128;
  static constexpr int RAW_TILE = E4M3 ? RSUB * KV_BLOCK : 0;
  static constexpr int NR = !E4M3 ? 0 : D == 256 ? 2 : D == 64 ? 3 : 4;
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

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(v)));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Instruction descriptor for kind::f16 with fp16 A and B (format code 0) and
// an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(N) >> 3) << 17) |
         ((static_cast<uint32_t>(M) >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A CTA's segments: the items of its range one after the other, each with the
// key tiles [t0, t1) that lie in the range.  Every role walks them on its own.
template <int BN>
struct Segments {
  PagedWalk<128, BN> w;
  long long unit, end;
  int t0, t1, tiles, keys;
  __device__ __forceinline__ void load(const PagedParams& p, int t) {
    tiles = w.my_tiles(p);
    keys = w.my_keys(p);
    t0 = t;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), t + (end - unit)));
  }
  __device__ __forceinline__ void start(const PagedParams& p, const PagedRange& r) {
    unit = r.first;
    end = r.end;
    load(p, w.start(p, r.seq, r.rem));
  }
  // False when the range is done.
  __device__ __forceinline__ bool next(const PagedParams& p) {
    unit += t1 - t0;
    if (unit >= end) return false;
    w.next(p);
    load(p, 0);
    return true;
  }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(384, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using C = TileCfg<D, E4M3>;
  constexpr int BN = C::BN;
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
  grid_dependency_wait();
  grid_launch_dependents();
  const PagedRange range =
      paged_range<C::BM, BN, C::THREADS>(p, reinterpret_cast<long long*>(smem + C::OFF_SCR));
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) p.notes[cta].last = -1;
  if (range.end <= range.first) return;  // block-uniform, nothing in flight

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

  Segments<BN> seg;

  if (warp >= 8) {
    reg_decrease<104>();
    if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
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
      seg.start(p, range);
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
        Segments<BN> ahead;
        ahead.start(p, range);
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
        seg.start(p, range);
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
    const int row = threadIdx.x & 127;
    auto wait = [&](int b, uint32_t parity) {
      return __all_sync(0xffffffffu,
                        mbar_wait(bar(b), parity, abort_flag, p.err, kErrTimeoutLoad)) != 0;
    };
    // Q of item `i` (segment s): row `row`, zeros past the sequence's rows.
    auto load_q = [&](const Segments<BN>& s, int i) -> bool {
      const int qs = i % C::NQ;
      if (i >= C::NQ && !wait(C::B_QEMPTY + qs, ((i / C::NQ) - 1) & 1)) return false;
      const int r = s.w.rt * C::BM + row;
      const bool live = r < s.w.g.qlen * p.G;
      const int tok = live ? r / p.G : 0;
      const __nv_bfloat16* src = p.q + (s.w.g.q0 + tok) * p.q_token +
                                 (s.w.h * p.G + (live ? r - tok * p.G : 0)) * p.q_head;
      const uint32_t dst = sQ + qs * C::Q_TILE + row * 128;
      auto at = [&](int c) -> uint32_t {  // 16-byte chunk c of the row
        return dst + (c >> 3) * C::Q_BLOCK + (((c & 7) ^ (row & 7)) << 4);
      };
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if constexpr (E4M3) {
        // Scaled by 2^e to a largest element in [2^7, 2^8), as fp16.
        float mx = 0.0f;
        if (live) {
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = reinterpret_cast<const uint4*>(src)[c];
            for (uint32_t x : {v.x, v.y, v.z, v.w})
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x << 16)),
                                   fabsf(__uint_as_float(x & 0xffff0000u))));
          }
        }
        int e = 134 - static_cast<int>(__float_as_uint(mx) >> 23);
        if (mx == 0.0f || !(mx < INFINITY)) e = 0;
        e = min(max(e, -120), 120);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        q_scale[qs * C::BM + row] =
            p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        auto half = [&](uint32_t x) {
          return pack_half2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
        };
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? reinterpret_cast<const uint4*>(src)[c] : zero;
          sts128(at(c), make_uint4(half(v.x), half(v.y), half(v.z), half(v.w)));
        }
      } else {
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c)
          sts128(at(c), live ? reinterpret_cast<const uint4*>(src)[c] : zero);
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(bar(C::B_QFULL + qs));
      return true;
    };
    // e4m3 tile in raw slot `raw` to the fp16 tile at `dst`, rows from `keep` on as zeros.
    auto convert = [&](uint32_t raw, uint32_t dst, int keep) {
      constexpr int PER = 128 / BN;  // threads a row
      const int r = row % BN;
#pragma unroll 4
      for (int c = row / BN; c < D / 16; c += PER) {
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (r < keep) {
          const uint4 v = lds128(raw + (c >> 3) * C::KV_BLOCK + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          lo = make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y),
                          e4m3x2_to_f16x2(v.y >> 16));
          hi = make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w),
                          e4m3x2_to_f16x2(v.w >> 16));
        }
        const uint32_t blk = dst + (c >> 2) * C::KV_BLOCK + r * 128;
        sts128(blk + ((((c & 3) * 2) ^ (r & 7)) << 4), lo);
        sts128(blk + ((((c & 3) * 2 + 1) ^ (r & 7)) << 4), hi);
      }
    };
    seg.start(p, range);
    Segments<BN> ahead = seg;  // the next item's Q (two Q tiles: one item ahead)
    int n = 0, i = 0;
    bool ok = load_q(ahead, 0), more = true;
    do {
      if (C::NQ == 2 && ok) {
        more = ahead.next(p);
        if (more) ok = load_q(ahead, i + 1);
      }
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
            convert(sR + rs * C::RAW_TILE, (kv ? sV : sK) + st * C::KV_TILE, keep);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(C::B_REMPTY + rs));
            mbar_arrive_warp(bar((kv ? C::B_VFIX : C::B_KFULL) + st));
          }
        } else {
          if (n >= C::NS && !(ok = wait(C::B_VEMPTY + st, ph))) break;
          if (keep < BN) {
            if (!(ok = wait(C::B_VFULL + st, (n / C::NS) & 1))) break;
            constexpr int CHUNKS = C::SUB * 8;  // 16-byte chunks of a row
            const int first = max(keep, 0);
            for (int x = first * CHUNKS + row; x < BN * CHUNKS; x += 128) {
              const int r = x / CHUNKS, c = x % CHUNKS;
              sts128(sV + st * C::KV_TILE + (c >> 3) * C::KV_BLOCK + r * 128 + ((c & 7) << 4),
                     make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
          }
          mbar_arrive_warp(bar(C::B_VFIX + st));
        }
      }
      if (!ok) break;
      ++i;
      more = seg.next(p);
      if (C::NQ == 1 && more) ok = load_q(seg, i);
    } while (ok && more);
  } else {
    // ------------------------------------------------------------ softmax (rows)
    reg_increase<240>();
    const int row = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    // Waits are made warp-uniform: the TMEM loads and stores are
    // warp-collective, so either every lane goes on or every lane stops.
    auto wait = [&](int b, uint32_t parity, uint32_t code) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, p.err, code)) != 0;
    };
    int n = 0, i = 0;
    bool ok = true;
    seg.start(p, range);
    do {
      const int rows = seg.w.g.qlen * p.G;
      const int r = seg.w.rt * C::BM + row;
      const bool live = r < rows;
      const int tok = live ? r / p.G : 0;
      const int head = seg.w.h * p.G + (live ? r - tok * p.G : 0);
      const int base = seg.w.g.klen - seg.w.g.qlen;
      const int last = p.causal ? base + tok : seg.w.g.klen - 1;  // last key this row sees
      const int all_see = p.causal ? base + seg.w.rt * C::BM / p.G : seg.w.g.klen - 1;
      const int qs = i % C::NQ;
      if (!(ok = wait(C::B_QFULL + qs, (i / C::NQ) & 1, kErrTimeoutSoftmax))) break;
      const float c = E4M3 ? q_scale[qs * C::BM + row] : p.scale_log2;
      mbar_arrive_warp(bar(C::B_QEMPTY + qs));
      float m_used = -INFINITY;  // reference maximum, log2 domain
      float l = 0.0f;
      for (int t = seg.t0; t < seg.t1; ++t, ++n) {
        const int bf = n % C::NB;
        const uint32_t col_s = bf * BN;
        if (!(ok = wait(C::B_SFULL + bf, (n / C::NB) & 1, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        float s[BN];
        {
          uint32_t x[BN];
#pragma unroll
          for (int q4 = 0; q4 < BN / 32; ++q4)
            tmem_ld32(tmem + lane_off + col_s + q4 * 32,
                      *reinterpret_cast<uint32_t(*)[32]>(&x[q4 * 32]));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < BN; ++k) s[k] = __uint_as_float(x[k]);
        }
        if (t * BN + BN - 1 > all_see) {
          const int see = last - t * BN;
#pragma unroll
          for (int k = 0; k < BN; ++k)
            if (k > see) s[k] = -INFINITY;
        }
        // Row maximum over 8 partial maxima, two new values each time.
        float pm[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) pm[u] = fmaxf(s[u], s[u + 8]);
#pragma unroll
        for (int k = 16; k < BN; k += 16)
#pragma unroll
          for (int u = 0; u < 8; ++u) pm[u] = fmax3(pm[u], s[k + u], s[k + u + 8]);
        const float mx = fmaxf(fmax3(pm[0], pm[1], pm[2]),
                               fmaxf(fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])));
        const float m_new = fmaxf(m_used, mx * c);
        float alpha = 1.0f;
        const bool upd = m_new > m_used + kRescaleThreshold;
        if (upd) {
          alpha = ex2_approx(m_used - m_new);
          m_used = m_new;
        }
        const float m_ref = (m_used == -INFINITY) ? 0.0f : m_used;
        const uint64_t c2 = f2_pack(c, c);
        const uint64_t nm2 = f2_pack(-m_ref, -m_ref);
        uint64_t ps2[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) ps2[u] = 0ull;
        {
          uint32_t pk[BN / 2];
#pragma unroll
          for (int k = 0; k < BN / 2; ++k) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(s[2 * k], s[2 * k + 1]), c2, nm2), x0, x1);
            const float p0 = ex2_approx(x0);
            const float p1 = ex2_approx(x1);
            ps2[k & 3] = f2_add(ps2[k & 3], f2_pack(p0, p1));
            pk[k] = E4M3 ? pack_half2(p0, p1) : pack_bf16x2(p0, p1);
          }
#pragma unroll
          for (int q4 = 0; q4 < BN / 64; ++q4)
            tmem_st32(tmem + lane_off + col_s + q4 * 32,
                      *reinterpret_cast<uint32_t(*)[32]>(&pk[q4 * 32]));
        }
        float sum, sum_hi;
        f2_unpack(f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3])), sum, sum_hi);
        l = l * alpha + (sum + sum_hi);
        if (t > seg.t0 && __any_sync(0xffffffffu, upd)) {
          // O is final before it is rescaled: S_n implies O += P_{n-2} V_{n-2},
          // so the barrier is at most one phase behind.
          if (!(ok = wait(C::B_ODONE, (n - 1) & 1, kErrTimeoutSoftmax))) break;
          tc_fence_after();
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t x[32];
            tmem_ld32(tmem + lane_off + C::COL_O + q4 * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
            tmem_st32(tmem + lane_off + C::COL_O + q4 * 32, x);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(bar(C::B_PFULL + bf));
      }
      if (!ok || !(ok = wait(C::B_FINAL, i & 1, kErrTimeoutEpilogue))) break;
      // ---------------------------------------------------------- end of the item
      tc_fence_after();
      const bool whole = seg.t0 == 0 && seg.t1 == seg.tiles;
      const int slot = cta * 2 + (seg.t0 == 0 ? 1 : 0);
      const float inv = l > 0.0f ? p.v_scale / l : 0.0f;
      const long long token = seg.w.g.q0 + tok;
      __nv_bfloat16* dst = p.o + token * p.o_token + head * p.o_head;
      float* part = p.part_o + (static_cast<long long>(slot) * C::BM + row) * D;
#pragma unroll 1
      for (int q4 = 0; q4 < D / 32; ++q4) {
        uint32_t x[32];
        tmem_ld32(tmem + lane_off + C::COL_O + q4 * 32, x);
        tmem_wait_ld();
        if (!live) continue;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              y[u] = pack_bf16x2(__uint_as_float(x[8 * k + 2 * u]) * inv,
                                 __uint_as_float(x[8 * k + 2 * u + 1]) * inv);
            reinterpret_cast<uint4*>(dst + q4 * 32)[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            reinterpret_cast<uint4*>(part + q4 * 32)[k] =
                make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      }
      if (live) {
        if (!whole)
          p.part_ml[static_cast<long long>(slot) * C::BM + row] = make_float2(m_used, l);
        else if (p.lse)
          p.lse[token * p.Hq + head] = l > 0.0f ? (m_used + log2f(l)) * kPagedLn2 : -INFINITY;
      }
      if (row == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
        p.notes[cta] = paged_note<C::BM, BN>(p, range, seg.w, seg.unit);
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

template <bool E4M3>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int d,
                     int ctas, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_t<64, E4M3>(tk, tv, p, ctas, stream);
    case 96: return launch_t<96, E4M3>(tk, tv, p, ctas, stream);
    case 128: return launch_t<128, E4M3>(tk, tv, p, ctas, stream);
    case 256: return launch_t<256, E4M3>(tk, tv, p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_tile(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                              int d, bool e4m3, int ctas, cudaStream_t stream) {
  return e4m3 ? launch_d<true>(tk, tv, p, d, ctas, stream)
              : launch_d<false>(tk, tv, p, d, ctas, stream);
}

}  // namespace fa
