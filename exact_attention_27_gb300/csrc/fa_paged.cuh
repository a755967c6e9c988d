// Shared by the kernels of fa_forward_paged: the step's geometry, the division
// of its key tiles among the CTAs, and the partial results of what is divided.
//
// Work is counted in units, one or a few a key tile of an item; an item is a tile of
// ROWS query rows of one (sequence, key/value head), its rows being the
// head's tokens x the G query heads that share it (row r: token r / G, head
// r % G), so that grouped heads read K and V once.  Items stand in order of
// sequence, head and row tile, and CTA c of C takes the units
// [c U / C, (c + 1) U / C): every CTA about the same work, however
// ragged the lengths, and a long sequence of few rows is spread over many.
// Lengths live on the device, so every CTA works its own range out at its
// start (one pass over q_start and kv_len by the whole block).
//
// An item inside one CTA is finished there.  The part of an item that a CTA
// shares with others goes to the workspace as (O, m, l), unnormalised fp32:
// slot 1 of the CTA where the item starts, slot 0 of each CTA that goes on
// with it (a range has at most one of each), and a second kernel joins them in
// CTA order, so results do not depend on timing.  The starting CTA leaves a
// note of the item and of the last CTA that has a part.  (Joining in the CTA that
// brings an item's last part, found by counting, measured 11.8 us against 10.8 us
// for two sequences of a thousand keys.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_paged_host.h"
#include "fa_ptx.cuh"

namespace fa {

// 4-D tiled copy global -> shared of a page's rows: x in bytes (a multiple of
// 128 here), row in the page, head, page.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x,
                                            int row, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(row), "r"(head), "r"(page)
      : "memory");
}

// Two e4m3 values (the low half of `v`) as packed fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(v)));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kPagedLog2e = 1.4426950408889634f;
constexpr float kPagedLn2 = 0.6931471805599453f;

// P = 2^(S - m).  The reference m moves only when the maximum has grown by more
// than kPagedRescale (log2) past what it was set for.  For fp16 P (e4m3 pages) it
// lies kPagedP16 below that maximum, so that the largest p is 2^7 to 2^15 and uses
// the range that fp16 (up to 65504) has above 1: fp16 ends at half steps of 2^-25,
// 2^-32 of the largest p, instead of 2^-25 of it, where many small weights would be
// lost from O and still count in l.  l, the parts and lse follow, as all are taken
// relative to m.  bf16 P has fp32's range and needs no such shift.
constexpr float kPagedRescale = 8.0f;
constexpr float kPagedP16 = 7.0f;

// Whether the reference m has to move for scores up to mx (times c).  For fp16 P the
// largest exponent is worked out as the exponents themselves are, in one rounding, so
// that none passes 15 unmoved however far the scores are from 0: fp16 has one bit more,
// where fp32's steps at 2^24 are 2.  (A moved reference is rounded to such a step too:
// by 8 at most below 2^28, so up to there p stays within 2^15.)
template <bool F16>
__device__ __forceinline__ bool paged_moves(float mx, float c, float m) {
  if constexpr (F16) return fmaf(mx, c, -m) > kPagedRescale + kPagedP16;
  return mx * c > m + kPagedRescale;
}

// The reference that scores up to mx (times c) want.
template <bool F16>
__device__ __forceinline__ float paged_reference(float mx, float c) {
  return F16 ? fmaf(mx, c, -kPagedP16) : mx * c;
}

struct PagedNote {
  int last;   // last CTA with a part of the item that starts here; -1: none
  int q0;     // first token of the sequence
  int rows;   // rows of the sequence (tokens x G)
  int tile0;  // the item's first row
  int head;   // key/value head
  int pad[3];
};

struct PagedParams {
  const __nv_bfloat16* q;
  long long q_token, q_head;
  __nv_bfloat16* o;
  long long o_token, o_head;
  float* lse;
  const int* table;
  long long table_stride;
  const int* q_start;
  const int* kv_len;
  int S, T, Hq, Hkv, G;
  int page_shift, max_pages, n_pages;
  int causal;
  int min_units;           // units that are worth a CTA
  float scale_log2;        // scale * log2(e) * k_descale
  float v_scale;
  float* part_o;           // [CTA][2][ROWS][D]
  float2* part_ml;         // [CTA][2][ROWS]
  PagedNote* notes;        // [CTA]
  uint32_t* err;
};

// a / b for a >= 0, b > 0; in 32 bits where they fit (a 64-bit division takes
// some hundred cycles, and several lie in the way of a short call).
__device__ __forceinline__ long long paged_div(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A sequence: its first row, its rows and its keys.  Its starts may go on past row T;
// those tokens have no rows here, and under the causal mask no key of theirs is seen,
// so the sequence then ends before them: its other tokens keep their places, as they
// do for the append.
struct PagedSeq {
  int q0, qlen, klen;
};

__device__ __forceinline__ int paged_room(const PagedParams& p) {
  return p.max_pages << p.page_shift;
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int s) {
  PagedSeq g;
  g.q0 = min(max(p.q_start[s], 0), p.T);
  const int end = max(p.q_start[s + 1], g.q0);
  g.qlen = min(end, p.T) - g.q0;
  g.klen = min(max(p.kv_len[s], 0), paged_room(p)) - (p.causal ? max(end - p.T, 0) : 0);
  return g;
}

// Items of ROWS rows and key tiles of TK keys.  An item counts for its key
// tiles and OVER more, about what starting and ending one costs, at FULL units each,
// or HALF where its rows fill at most half of ROWS.
template <int ROWS_, int TK_, int OVER_, int FULL_ = 1, int HALF_ = 1>
struct PagedWalk {
  static constexpr int ROWS = ROWS_, TK = TK_, OVER = OVER_, FULL = FULL_, HALF = HALF_;
  int s, h, rt, n_rt;
  PagedSeq g;

  static __device__ __forceinline__ int row_tiles(const PagedParams& p, const PagedSeq& g) {
    return (g.qlen * p.G + ROWS - 1) / ROWS;
  }
  // Keys that the last row of row tile rt sees.
  static __device__ __forceinline__ int keys(const PagedParams& p, const PagedSeq& g, int rt) {
    if (!p.causal) return g.klen;
    const int tokens =
        min(g.qlen, static_cast<int>(static_cast<uint32_t>(rt * ROWS + ROWS - 1) /
                                     static_cast<uint32_t>(p.G)) + 1);
    return max(g.klen - g.qlen + tokens, 0);
  }
  // Its key tiles: one at least, so that rows without keys are written too.
  static __device__ __forceinline__ int tiles(const PagedParams& p, const PagedSeq& g, int rt) {
    return max((keys(p, g, rt) + TK - 1) / TK, 1);
  }
  // Whether row tile rt has at most half an item's rows.
  static __device__ __forceinline__ bool half(const PagedParams& p, const PagedSeq& g, int rt) {
    return g.qlen * p.G - rt * ROWS <= ROWS / 2;
  }
  // Units of one of its key tiles.
  static __device__ __forceinline__ int weight(const PagedParams& p, const PagedSeq& g, int rt) {
    return FULL == HALF ? FULL : half(p, g, rt) ? HALF : FULL;
  }
  static __device__ __forceinline__ int units(const PagedParams& p, const PagedSeq& g, int rt) {
    return (tiles(p, g, rt) + OVER) * weight(p, g, rt);
  }
  // Units of one head of the sequence of each lane; the whole warp calls this.
  static __device__ __forceinline__ long long head_units(const PagedParams& p, const PagedSeq& g) {
    constexpr int SHORT = 4;
    const int n = row_tiles(p, g);
    if (!p.causal)  // (all but the last are alike)
      return n == 0 ? 0 : static_cast<long long>(n - 1) * units(p, g, 0) + units(p, g, n - 1);
    long long u = 0;
    if (n <= SHORT) {
      for (int rt = 0; rt < n; ++rt) u += units(p, g, rt);
    }
    // Long chunks: all lanes, one sequence after the other.
    const int lane = lane_id();
    for (unsigned todo = __ballot_sync(0xffffffffu, n > SHORT); todo != 0; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      PagedSeq x;
      x.q0 = 0;
      x.qlen = __shfl_sync(0xffffffffu, g.qlen, src);
      x.klen = __shfl_sync(0xffffffffu, g.klen, src);
      const int m = __shfl_sync(0xffffffffu, n, src);
      long long sum = 0;
      for (int rt = lane; rt < m; rt += 32) sum += units(p, x, rt);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == src) u = sum;
    }
    return u;
  }

  // Goes to unit `rem` of sequence s0, whose heads have per_head units; the
  // whole warp calls this.  Returns the unit within the item.
  __device__ __forceinline__ int start(const PagedParams& p, int s0, long long rem,
                                       long long per_head) {
    s = s0;
    g = paged_seq(p, s);
    n_rt = row_tiles(p, g);
    h = static_cast<int>(paged_div(rem, per_head));
    rem -= h * per_head;
    const int lane = lane_id();
    for (int base = 0;; base += 32) {
      const int mine = base + lane < n_rt ? units(p, g, base + lane) : 0;
      int x = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, rem < x);
      if (past != 0 || base + 32 >= n_rt) {
        const int at = past != 0 ? __ffs(past) - 1 : 0;
        rt = min(base + at, n_rt - 1);
        return static_cast<int>(rem) - __shfl_sync(0xffffffffu, x - mine, at);
      }
      rem -= __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (++rt < n_rt) return;
    rt = 0;
    if (++h < p.Hkv) return;
    h = 0;
    do {
      if (++s >= p.S) return;  // (not reached while units are left)
      g = paged_seq(p, s);
      n_rt = row_tiles(p, g);
    } while (n_rt == 0);
  }
};

struct PagedRange {
  long long units, first, end;  // all units; this CTA's
  int ctas;                     // CTAs with units
  int seq;                      // where `first` lies
  long long rem, per_head;      // its unit in that sequence; units of a head there
  // CTA whose range holds unit u.
  __device__ __forceinline__ int owner(long long u) const {
    return static_cast<int>(paged_div((u + 1) * ctas - 1, units));
  }
};

// Every thread of the block calls this; `scratch`: 40 long longs of shared
// memory, free again after the block's next barrier.
template <typename Walk, int THREADS>
__device__ __forceinline__ PagedRange paged_range(const PagedParams& p, long long* scratch) {
  constexpr int WARPS = THREADS / 32;
  static_assert(WARPS <= 32, "scratch");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Exclusive prefix of `mine` over the block; `all` gets the sum.
  auto scan = [&](long long mine, long long& all) -> long long {
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long before = 0;
    all = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    __syncthreads();
    return before + x - mine;
  };
  auto units_of = [&](int s) -> long long {
    PagedSeq g{0, 0, 0};
    if (s < p.S) {
      g = paged_seq(p, s);
      if (blockIdx.x == 0 && p.kv_len[s] > paged_room(p)) atomicOr(p.err, kErrBadPage);
    }
    return Walk::head_units(p, g) * p.Hkv;
  };
  PagedRange r;
  r.seq = 0;
  r.rem = 0;
  r.per_head = 1;
  r.first = r.end = 0;
  auto divide = [&]() -> bool {  // false: no units for this CTA
    if (r.units == 0) return false;
    r.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x),
                                  paged_div(r.units + p.min_units - 1, p.min_units)));
    if (static_cast<int>(blockIdx.x) >= r.ctas) return false;
    r.first = paged_div(blockIdx.x * r.units, r.ctas);
    r.end = paged_div((blockIdx.x + 1) * r.units, r.ctas);
    return true;
  };
  if (p.S <= 32) {
    // Every warp for itself, without barriers.
    const long long mine = units_of(lane);
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    r.units = __shfl_sync(0xffffffffu, x, 31);
    if (!divide()) return r;
    r.seq = __ffs(__ballot_sync(0xffffffffu, r.first < x)) - 1;
    r.rem = r.first - __shfl_sync(0xffffffffu, x - mine, r.seq);
    r.per_head = paged_div(__shfl_sync(0xffffffffu, mine, r.seq), p.Hkv);
    return r;
  }
  long long mine = units_of(tid), all;
  long long pre = scan(mine, all);
  r.units = all;
  for (int base = THREADS; base < p.S; base += THREADS) {
    scan(units_of(base + tid), all);
    r.units += all;
  }
  if (!divide()) return r;  // block-uniform
  if (tid == 0) {
    scratch[32] = scratch[33] = 0;
    scratch[34] = 1;
  }
  __syncthreads();
  long long done = 0;
  for (int base = 0; base < p.S; base += THREADS) {
    if (base > 0) {
      mine = units_of(base + tid);
      pre = scan(mine, all);
    } else if (p.S > THREADS) {
      pre = scan(mine, all);
    } else {
      all = r.units;
    }
    if (r.first >= done + pre && r.first < done + pre + mine) {
      scratch[32] = base + tid;
      scratch[33] = r.first - done - pre;
      scratch[34] = paged_div(mine, p.Hkv);
    }
    __syncthreads();
    if (r.first < done + all) break;
    done += all;
  }
  r.seq = static_cast<int>(scratch[32]);
  r.rem = scratch[33];
  r.per_head = scratch[34];
  return r;
}

// A CTA's segments: the items of its range one after the other, each with the
// key tiles [t0, t1) that lie in the range.  Every role walks them on its own,
// from a common start.
template <typename Walk>
struct PagedSegments {
  Walk w;
  long long unit, end;  // where the item's part of the range begins; the range's end
  int t0, t1, tiles, keys, used;
  __device__ __forceinline__ int weight(const PagedParams& p) const {
    return Walk::weight(p, w.g, w.rt);
  }
  __device__ __forceinline__ void load(const PagedParams& p, int at) {
    tiles = Walk::tiles(p, w.g, w.rt);
    keys = Walk::keys(p, w.g, w.rt);
    const int wt = weight(p);
    used = static_cast<int>(
        min(static_cast<long long>((tiles + Walk::OVER) * wt - at), end - unit));
    // A tile belongs to the range that holds its first unit.
    auto tile = [&](int u) {
      if constexpr (Walk::FULL == 1) return u;
      return wt == Walk::HALF ? (u + Walk::HALF - 1) / Walk::HALF
                              : (u + Walk::FULL - 1) / Walk::FULL;
    };
    t0 = min(tile(at), tiles);
    t1 = min(tile(at + used), tiles);
  }
  // False if the range holds no key tile.  The whole warp calls this.
  __device__ __forceinline__ bool start(const PagedParams& p, const PagedRange& r) {
    unit = r.first;
    end = r.end;
    if (unit >= end) return false;
    load(p, w.start(p, r.seq, r.rem, r.per_head));
    return t0 < t1 || next(p);
  }
  // False when the range is done.
  __device__ __forceinline__ bool next(const PagedParams& p) {
    unit += used;
    if (unit >= end) return false;
    w.next(p);
    load(p, 0);
    return true;
  }
};

// What a CTA notes about the item that starts in its range and goes on past it.
template <typename Walk>
__device__ __forceinline__ PagedNote paged_note(const PagedParams& p, const PagedRange& r,
                                                const PagedSegments<Walk>& seg) {
  const Walk& w = seg.w;
  PagedNote n{};
  n.last = r.owner(seg.unit + static_cast<long long>(seg.tiles - 1) * seg.weight(p));
  n.q0 = w.g.q0;
  n.rows = w.g.qlen * p.G;
  n.tile0 = w.rt * Walk::ROWS;
  n.head = w.h;
  return n;
}

}  // namespace fa
