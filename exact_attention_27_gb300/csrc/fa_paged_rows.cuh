// Attention of new tokens over a paged cache for few rows a sequence (single
// tokens, short drafts): bound by the bytes of K and V.
//
// An item is 16 rows (tokens x grouped query heads) of one sequence and
// key/value head; fa_paged.cuh says how the key tiles of all items are divided
// among the CTAs.  Per key tile of 64 keys a producer warp copies K and V into
// a ring of shared memory, one box per page and 128-byte column block, and
// four warps take 16 keys each, with their own running maximum, sum
// and O in registers, so that they meet only at the end of an item:
//     S = Q K^T;  m' = max(m, max S);  p = 2^(S - m');
//     l = l 2^(m - m') + sum p;  O = O 2^(m - m') + p V.
// m moves only when the maximum has grown by more than 8 (log2), which bounds p by
// 2^8 and leaves O / l as it is.  At the end the four key groups join (O, m, l)
// through shared memory.
//
// Why mma.sync here: 16 rows fill an eighth of a tcgen05 tile, and at 7 TB/s an
// SM gets 23 bytes a cycle, 12 bf16 values, which the 16-row products use up at
// under a quarter of the rate of the warp-level instruction.  What counts is
// bytes in flight: two CTAs an SM with about 96 KB of ring each.  64 sequences of
// 100 to 8000 keys, 8 heads, d = 128: 172 us, 6.5 TB/s; one of 120,000 e4m3
// keys: 49.0 us, 5.0 TB/s (each tile's conversions and products take as long as
// its bytes there, and hide behind other warps' in part).
//
// bf16 cache: P is rounded to bf16 (2^-8 relative at most) for P V, as in
// fa_forward; l sums the unrounded fp32 values.  e4m3 cache: K and V convert to
// fp16 exactly, P is rounded to fp16 with m held 7 (log2) lower, so that p is at most
// 2^15 (2^-11 of each p, and 2^-32 of the largest where that is more), and each row of
// Q is scaled by a power of two to a largest element in [2^7, 2^8), so that its bf16
// values fit fp16 (what falls below fp16's range is 2^-33 of the row's largest); the
// power is taken out of the scale of the row's scores.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_paged_host.h"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"

namespace fa {
namespace {

constexpr int kTK = 64;  // keys per tile

// CTAs an SM.  A CTA's four warps each wait for loads, conversions and products
// in turn, so more of them hide more, as registers and shared memory allow; with
// bytes half as many, e4m3 pages want three (120,000 keys of 8 heads, d = 128: 59
// us with two, though d = 128 then spills 60 bytes a thread).
constexpr int rows_occupancy(int d, bool e4m3) { return d == 256 ? 1 : e4m3 ? 3 : 2; }

template <int D_, bool E4M3_>
struct RowsCfg {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int ROWS = 16;
  static constexpr int WARPS = 4;        // consumers
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int SUB = (D * (E4M3 ? 1 : 2) + 127) / 128;  // 128-byte column blocks
  static constexpr int BLOCK = kTK * 128;
  static constexpr int STAGE = 2 * SUB * BLOCK;                 // K and V
  static constexpr int MERGE = 2 * ROWS * D * 4;                // two of the four key groups' O
  static constexpr int OCC = rows_occupancy(D, E4M3);           // CTAs an SM
  static constexpr int BUDGET = (OCC == 3 ? 74 : OCC == 2 ? 112 : 224) * 1024;
  // At d = 256 and with three CTAs the fragments of Q (64 or 32 registers) lie
  // in shared memory.
  static constexpr bool QS = D == 256 || OCC == 3;
  static constexpr int QBYTES = QS ? ROWS * D * 2 : 0;
  static constexpr int FIT = (BUDGET - MERGE - QBYTES - 3 * 1024) / STAGE;
  static constexpr int NS = FIT > 8 ? 8 : FIT;
  static constexpr int OFF_MERGE = NS * STAGE;
  static constexpr int OFF_Q = OFF_MERGE + MERGE;               // [D / 16][32 lanes] fragments
  static constexpr int OFF_ML = OFF_Q + QBYTES;                 // [4][16] (m, l)
  static constexpr int OFF_SCR = OFF_ML + 4 * 16 * 8;
  static constexpr int OFF_BAR = OFF_SCR + 40 * 8;
  static constexpr int OFF_MISC = OFF_BAR + 2 * NS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(NS >= 2 && SMEM_BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Scores of two 8-key tiles (keys key + 8 i + (x & 1); rows by x >> 1) to exponents: products
// times `by` (capped: scale / softcap, see paged_softmax), capped and lowered (fa_scores.cuh; the
// tanh as there).  The whole warp calls this.
__device__ __forceinline__ void shape_rows(const PagedParams& p, float (&s)[2][4],
                                           const ScoreFactors& f, const float (&by)[2],
                                           const float (&slope2)[2], const float (&pos)[2],
                                           int key) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[4], none[1];
    auto load = [&](float (&y)[4], int) {
      y[0] = s[0][2 * h] * by[h], y[1] = s[0][2 * h + 1] * by[h];
      y[2] = s[1][2 * h] * by[h], y[3] = s[1][2 * h + 1] * by[h];
    };
    load(v, 0);
    if (p.cap2 > 0.0f) shape_scores<4, true, false, false, false>(v, none, f, 0.0f, 0.0f, 0.0f, load);
    if (p.slopes) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float at = static_cast<float>(key + 8 * (x >> 1) + (x & 1));
        v[x] = fmaf(-slope2[h], fabsf(pos[h] - at), v[x]);
      }
    }
    s[0][2 * h] = v[0];
    s[0][2 * h + 1] = v[1];
    s[1][2 * h] = v[2];
    s[1][2 * h + 1] = v[3];
  }
}

// Barrier among the consumer warps.
__device__ __forceinline__ void group_sync() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

template <int D, bool E4M3, bool SHAPED>
__global__ void __launch_bounds__(RowsCfg<D, E4M3>::THREADS, RowsCfg<D, E4M3>::OCC)
    fa_paged_rows_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedParams p) {
  using C = RowsCfg<D, E4M3>;
  using Walk = PagedWalk<C::ROWS, kTK, 1, SHAPED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int st) -> uint32_t { return sbase + C::OFF_BAR + 8 * st; };
  auto empty = [&](int st) -> uint32_t { return sbase + C::OFF_BAR + 8 * (C::NS + st); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int st = 0; st < C::NS; ++st) {
      mbar_init(full(st), 1);
      mbar_init(empty(st), C::WARPS);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::WARPS && elect_one()) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_launch_dependents();
  grid_dependency_wait();
  const PagedRange range =
      paged_range<Walk, C::THREADS>(p, reinterpret_cast<long long*>(smem + C::OFF_SCR));
  __syncthreads();
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) p.notes[cta].last = -1;
  PagedSegments<Walk> seg;
  if (!seg.start(p, range)) return;  // block-uniform, no copies in flight
  bool more = true;

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ producer
    const int page = 1 << p.page_shift;
    const int box_rows = min(page, kTK);
    const int boxes_k = kTK / box_rows * C::SUB;
    // This lane's box: K or V, which rows of the tile, which column block.
    const bool mine = lane < 2 * boxes_k;
    const int is_v = lane >= boxes_k;
    const int in_k = lane - is_v * boxes_k;
    const int row0 = in_k / C::SUB * box_rows, sub = in_k % C::SUB;
    const uint32_t dst0 = sbase + (is_v * C::SUB + sub) * C::BLOCK + row0 * 128;
    int n = 0;  // tiles issued
    bool ok = true;
    for (; ok && more; more = seg.next(p)) {
      for (int t = seg.t0; t < seg.t1; ++t, ++n) {
        const int st = n % C::NS;
        const int key0 = (seg.tile0() + t) * kTK + row0;
        // (pages before the window are not read)
        bool issue = mine && key0 < seg.keys && (!SHAPED || key0 + box_rows > seg.first);
        int id = 0;
        if (issue) {
          id = p.table[seg.w.s * p.table_stride + (key0 >> p.page_shift)];
          if (id < 0 || id >= p.n_pages) {
            atomicOr(p.err, kErrBadPage);
            issue = false;
          }
        }
        if (n >= C::NS)
          ok = __all_sync(0xffffffffu, mbar_wait(empty(st), ((n / C::NS) - 1) & 1, abort_flag,
                                                 p.err, kErrTimeoutLoad));
        if (!ok) break;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, issue));
        if (lane == 0) mbar_arrive_expect_tx(full(st), boxes * box_rows * 128);
        __syncwarp();
        if (issue)
          tma_load_4d(dst0 + st * C::STAGE, is_v ? &tmV : &tmK, full(st), sub * 128,
                      key0 & (page - 1), seg.w.h, id);
      }
    }
    // On the abort path the copies already issued land before the CTA's memory is released.
    if (*abort_flag)
      for (int i = max(0, n - C::NS); i < n; ++i)
        mbar_wait_timed(full(i % C::NS), (i / C::NS) & 1);
  } else {
    // ------------------------------------------------------------ consumers
    const int kg = warp;                    // which 16 keys of a tile
    const int g = lane >> 2, c = lane & 3;  // row (and row + 8), column quad of the fragments
    constexpr int NT = D / 8;               // 8-column tiles of O
    float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    uint4* qs = reinterpret_cast<uint4*>(smem + C::OFF_Q);
    int n = 0;
    bool ok = true;
    for (; more; more = seg.next(p)) {
      const Walk& w = seg.w;
      const int keys = seg.keys;
      const int rows = w.g.qlen * p.G;
      const int r0 = w.rt * C::ROWS;  // first row
      // Rows r0 + g and r0 + g + 8: token, query head, last key seen.
      int tok[2], head[2], last[2], first[2];
      float slope2[2], pos[2];
      bool live[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + g + 8 * i;
        live[i] = r < rows;
        tok[i] = live[i] ? r / p.G : 0;
        head[i] = w.h * p.G + (live[i] ? r - tok[i] * p.G : 0);
        last[i] = p.causal ? w.g.klen - w.g.qlen + tok[i] : w.g.klen - 1;
        if constexpr (SHAPED) {
          const int at = w.g.base + tok[i];
          first[i] = paged_from(p, at);
          slope2[i] = p.slopes ? p.slopes[head[i]] * kPagedLog2e : 0.0f;
          pos[i] = static_cast<float>(at);
        }
      }
      // Keys up to here are seen by every row of the tile.
      const int all_see = p.causal ? w.g.klen - w.g.qlen + w.rt * C::ROWS / p.G : w.g.klen - 1;
      // ... and keys from here on, as far as windows go.
      const int from_all =
          SHAPED ? paged_from(p, w.g.base + (min(r0 + C::ROWS, rows) - 1) / p.G) : 0;
      // Q fragments, from global memory (rows past the sequence: zeros).  For
      // e4m3, K is read 8 bytes a lane, which fixes the order of the columns.
      uint32_t qf[D / 16][4];
      float cs[2] = {p.scale_log2, p.scale_log2};
      {
        const __nv_bfloat16* src[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          src[i] = p.q + (w.g.q0 + tok[i]) * p.q_token + head[i] * p.q_head;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = x & 1;
            const int col = E4M3 ? kk / 2 * 32 + 8 * c + (kk & 1) * 4 + (x >> 1) * 2
                                 : kk * 16 + 2 * c + (x >> 1) * 8;
            qf[kk][x] = live[i] ? *reinterpret_cast<const uint32_t*>(src[i] + col) : 0u;
          }
        if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = 0.0f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
              for (int x = i; x < 4; x += 2)
                mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(qf[kk][x] << 16)),
                                     fabsf(__uint_as_float(qf[kk][x] & 0xffff0000u))));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^e with e = 7 - exponent of the largest, within fp32's range.
            int e = 134 - static_cast<int>(__float_as_uint(mx) >> 23);
            if (mx == 0.0f || !(mx < INFINITY)) e = 0;
            e = min(max(e, -120), 120);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            cs[i] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
              for (int x = i; x < 4; x += 2)
                qf[kk][x] = pack_f16x2(__uint_as_float(qf[kk][x] << 16) * up,
                                       __uint_as_float(qf[kk][x] & 0xffff0000u) * up);
          }
        }
      }
      ScoreFactors factors;
      float by[2];
      if constexpr (SHAPED) {
        factors = score_factors(1.0f, p.cap2);
#pragma unroll
        for (int i = 0; i < 2; ++i) by[i] = p.cap2 > 0.0f ? cs[i] / p.cap2 : cs[i];
      }
      if constexpr (C::QS) {
        if (kg == 0) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            qs[kk * 32 + lane] = make_uint4(qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
        }
        group_sync();
      }
      auto q_frag = [&](int kk, uint32_t (&a)[4]) {
        if constexpr (C::QS) {
          const uint4 v = qs[kk * 32 + lane];
          a[0] = v.x;
          a[1] = v.y;
          a[2] = v.z;
          a[3] = v.w;
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) a[x] = qf[kk][x];
        }
      };
      float o[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.0f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

      for (int t = seg.t0; t < seg.t1; ++t, ++n) {
        const int st = n % C::NS;
        // Warp-uniform.  After a timeout the warp still goes through every
        // item's barriers, without work.
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait(full(st), (n / C::NS) & 1, abort_flag, p.err,
                                                 kErrTimeoutSoftmax));
        if (!ok) continue;
        const int key0 = (seg.tile0() + t) * kTK + kg * 16;  // this warp's first key
        if (key0 < keys) {
          const uint32_t sk = sbase + st * C::STAGE, sv = sk + C::SUB * C::BLOCK;
          // S: two 8-key tiles.
          float s[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[i][x] = 0.0f;
          if constexpr (E4M3) {
#pragma unroll
            for (int k2 = 0; k2 < D / 32; ++k2) {
              const int byte = k2 * 32 + 8 * c;
              uint32_t a0[4], a1[4];
              q_frag(2 * k2, a0);
              q_frag(2 * k2 + 1, a1);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int row = kg * 16 + 8 * i + g;
                const uint2 v = lds64(sk + (byte >> 7) * C::BLOCK + row * 128 +
                                      ((((byte >> 4) & 7) ^ (row & 7)) << 4) + (byte & 8));
                mma16816<true>(s[i], a0, e4m3x2_f16x2(v.x), e4m3x2_f16x2(v.x >> 16));
                mma16816<true>(s[i], a1, e4m3x2_f16x2(v.y), e4m3x2_f16x2(v.y >> 16));
              }
            }
          } else {
            const int row = kg * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int chunk = kk * 2 + ((lane >> 3) & 1);
              uint32_t a[4], b[4];
              q_frag(kk, a);
              ldsm4(sk + (chunk >> 3) * C::BLOCK + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), b);
              mma16816<false>(s[0], a, b[0], b[1]);
              mma16816<false>(s[1], a, b[2], b[3]);
            }
          }
          if constexpr (SHAPED) shape_rows(p, s, factors, by, slope2, pos, key0 + 2 * c);
          if (key0 + 15 > all_see || (SHAPED && key0 < from_all)) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int key = key0 + 8 * i + 2 * c + (x & 1);
                if (key > last[x >> 1] || (SHAPED && key < first[x >> 1])) s[i][x] = -INFINITY;
              }
          }
          // Running maximum and sum of rows g (x = 0, 1) and g + 8 (x = 2, 3).
          float alpha[2];
          bool upd = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]),
                             fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[i] = 1.0f;
            const float unit = SHAPED ? 1.0f : cs[i];  // (shaped scores are exponents)
            if (paged_moves<E4M3>(mx, unit, m[i])) {
              const float m_new = paged_reference<E4M3>(mx, unit);
              alpha[i] = ex2_approx(m[i] - m_new);
              m[i] = m_new;
              upd = true;
            }
            const float ref = m[i] == -INFINITY ? 0.0f : m[i];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int x = 2 * i; x < 2 * i + 2; ++x)
                s[j][x] = ex2_approx(SHAPED ? s[j][x] - ref : fmaf(s[j][x], cs[i], -ref));
            l[i] = l[i] * alpha[i] + ((s[0][2 * i] + s[0][2 * i + 1]) +
                                      (s[1][2 * i] + s[1][2 * i + 1]));
          }
          if (__any_sync(0xffffffffu, upd)) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              o[i][0] *= alpha[0];
              o[i][1] *= alpha[0];
              o[i][2] *= alpha[1];
              o[i][3] *= alpha[1];
            }
          }
          uint32_t pf[4];
          if constexpr (E4M3) {
            pf[0] = pack_f16x2(s[0][0], s[0][1]);
            pf[1] = pack_f16x2(s[0][2], s[0][3]);
            pf[2] = pack_f16x2(s[1][0], s[1][1]);
            pf[3] = pack_f16x2(s[1][2], s[1][3]);
          } else {
            pf[0] = pack_bf16x2(s[0][0], s[0][1]);
            pf[1] = pack_bf16x2(s[0][2], s[0][3]);
            pf[2] = pack_bf16x2(s[1][0], s[1][1]);
            pf[3] = pack_bf16x2(s[1][2], s[1][3]);
          }
          // O += P V.  Rows of V at and past `keys` (stale or never copied)
          // have p = 0 but may hold anything, so they are made 0.
          // (Likewise rows before the item's first key, whose pages may not have been copied.)
          const bool tail = key0 + 16 > keys || (SHAPED && key0 < seg.first);
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
          if (tail) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k = key0 + 8 * i + 2 * c;
              keep[i] = (k < keys ? 0xffffu : 0u) | (k + 1 < keys ? 0xffff0000u : 0u);
              if constexpr (SHAPED)
                keep[i] &= (k >= seg.first ? 0xffffu : 0u) | (k + 1 >= seg.first ? 0xffff0000u : 0u);
            }
          }
          if constexpr (E4M3) {
            // A transposed fragment element is a pair of neighbouring columns
            // of one key; the even and the odd columns form a tile each.
            const int row = kg * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int d2 = 0; d2 < D / 32; ++d2) {
              const int chunk = d2 * 2 + (lane >> 4);
              uint32_t v[4];
              ldsm4_trans(sv + (chunk >> 3) * C::BLOCK + row * 128 +
                              (((chunk & 7) ^ (row & 7)) << 4), v);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t ev = __byte_perm(v[2 * i], v[2 * i + 1], 0x6420);
                const uint32_t od = __byte_perm(v[2 * i], v[2 * i + 1], 0x7531);
                uint32_t e0 = e4m3x2_f16x2(ev), e1 = e4m3x2_f16x2(ev >> 16);
                uint32_t d0 = e4m3x2_f16x2(od), d1 = e4m3x2_f16x2(od >> 16);
                if (tail) {
                  e0 &= keep[0];
                  e1 &= keep[1];
                  d0 &= keep[0];
                  d1 &= keep[1];
                }
                mma16816<true>(o[4 * d2 + 2 * i], pf, e0, e1);
                mma16816<true>(o[4 * d2 + 2 * i + 1], pf, d0, d1);
              }
            }
          } else {
            const int row = kg * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int d2 = 0; d2 < D / 16; ++d2) {
              const int chunk = d2 * 2 + (lane >> 4);
              uint32_t v[4];
              ldsm4_trans(sv + (chunk >> 3) * C::BLOCK + row * 128 +
                              (((chunk & 7) ^ (row & 7)) << 4), v);
              if (tail) {
                v[0] &= keep[0];
                v[1] &= keep[1];
                v[2] &= keep[0];
                v[3] &= keep[1];
              }
              mma16816<false>(o[2 * d2], pf, v[0], v[1]);
              mma16816<false>(o[2 * d2 + 1], pf, v[2], v[3]);
            }
          }
        }
        mbar_arrive_warp(empty(st));
      }

      // ---------------------------------------------------------- end of the item
      // The four key groups join: common maximum, then O of groups 2 and 3
      // onto 0 and 1, then of 1 onto 0, in registers' order (lane-contiguous).
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (c == 0) ml[kg * 16 + g + 8 * i] = make_float2(m[i], l[i]);
      }
      group_sync();
      float M[2], L[2], f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = ml[k * 16 + g + 8 * i];
        M[i] = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
        const float ref = M[i] == -INFINITY ? 0.0f : M[i];
        L[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) L[i] += x[k].y * ex2_approx(x[k].x - ref);
        f[i] = ex2_approx(m[i] - ref);
      }
      auto halves = [&](auto&& go) {  // rows g, and g + 8 if there are any
#pragma unroll
        for (int i = 0; i < NT * 2; ++i) go(i >> 1, i & 1, i * 32 + lane, f[0]);
        if (rows - r0 > 8) {
#pragma unroll
          for (int i = 0; i < NT * 2; ++i)
            go(i >> 1, 2 + (i & 1), (NT * 2 + i) * 32 + lane, f[1]);
        }
      };
      if (kg >= 2)
        halves([&](int nt, int x, int at, float s) { merge[(kg - 2) * 16 * D + at] = o[nt][x] * s; });
      group_sync();
      if (kg < 2)
        halves([&](int nt, int x, int at, float s) {
          o[nt][x] = o[nt][x] * s + merge[kg * 16 * D + at];
          if (kg == 1) merge[16 * D + at] = o[nt][x];
        });
      group_sync();
      const bool whole = seg.t0 == 0 && seg.t1 == seg.tiles;
      if (kg == 0 && ok) {
        const int slot = cta * 2 + (seg.t0 == 0 ? 1 : 0);
        float* po = p.part_o + static_cast<long long>(slot) * C::ROWS * D;
        float2* pml = p.part_ml + static_cast<long long>(slot) * C::ROWS;
        halves([&](int nt, int x, int at, float) { o[nt][x] += merge[16 * D + at]; });
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!live[i]) continue;
          const long long token = w.g.q0 + tok[i];
          // (v_scale / L could fall below fp32's range where o does not)
          const float inv = L[i] > 0.0f ? 1.0f / L[i] : 0.0f;
          __nv_bfloat16* dst = p.o + token * p.o_token + head[i] * p.o_head;
          float* pd = po + (g + 8 * i) * D;
#pragma unroll
          for (int nt = 0; nt < NT; nt += E4M3 ? 2 : 1) {
            // The lane's columns: two, or for e4m3 four of an even and odd tile.
            const float x0 = o[nt][2 * i], x1 = o[nt][2 * i + 1];
            if constexpr (E4M3) {
              const float y0 = o[nt + 1][2 * i], y1 = o[nt + 1][2 * i + 1];
              const int col = nt / 2 * 16 + 4 * c;
              if (whole)
                *reinterpret_cast<uint2*>(dst + col) = make_uint2(
                    pack_bf16x2(x0 * inv * p.v_scale, y0 * inv * p.v_scale),
                    pack_bf16x2(x1 * inv * p.v_scale, y1 * inv * p.v_scale));
              else
                *reinterpret_cast<float4*>(pd + col) = make_float4(x0, y0, x1, y1);
            } else {
              const int col = nt * 8 + 2 * c;
              if (whole)
                *reinterpret_cast<uint32_t*>(dst + col) = pack_bf16x2(x0 * inv, x1 * inv);
              else
                *reinterpret_cast<float2*>(pd + col) = make_float2(x0, x1);
            }
          }
          if (c == 0) {
            if (!whole)
              pml[g + 8 * i] = make_float2(M[i], L[i]);
            else if (p.lse)
              p.lse[token * p.Hq + head[i]] =
                  L[i] == 0.0f ? -INFINITY : (M[i] + log2f(L[i])) * kPagedLn2;
          }
        }
        if (lane == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
          p.notes[cta] = paged_note(p, range, seg);
      }
    }
  }
  __syncthreads();
}

template <int D, bool E4M3, bool SHAPED>
cudaError_t launch_rows_t(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                          int ctas, cudaStream_t stream) {
  using C = RowsCfg<D, E4M3>;
  const cudaError_t e = set_smem_limit_once<fa_paged_rows_kernel<D, E4M3, SHAPED>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_paged_rows_kernel<D, E4M3, SHAPED>, dim3(ctas), dim3(C::THREADS),
                          C::SMEM_BYTES, stream, tk, tv, p);
}

template <bool E4M3, bool SHAPED>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int d,
                        int ctas, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_rows_t<64, E4M3, SHAPED>(tk, tv, p, ctas, stream);
    case 96: return launch_rows_t<96, E4M3, SHAPED>(tk, tv, p, ctas, stream);
    case 128: return launch_rows_t<128, E4M3, SHAPED>(tk, tv, p, ctas, stream);
    case 256: return launch_rows_t<256, E4M3, SHAPED>(tk, tv, p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace fa
