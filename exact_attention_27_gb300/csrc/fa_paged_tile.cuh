// Pieces of the two tcgen05 kernels of fa_forward_paged (fa_paged_tile.cu,
// fa_paged_tile2.cu): a CTA's walk over its items, the rows of Q into shared
// memory, e4m3 tiles to fp16, the softmax of a row and what becomes of its O.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_paged.cuh"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"

namespace fa {

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

// One row of an item, as its thread sees it.
struct PagedRow {
  bool live;       // a row of the sequence
  int head;        // query head
  int last;        // last key it sees
  int all_see;     // last key that every row of the item sees
  int first;       // first key it sees, and the last of the item's rows' first ones (0 unless
  int all_from;    // a window says otherwise)
  int pos;         // its token's position (shaped scores)
  float slope2;    // slope log2(e) of its head (shaped scores)
  long long token;
};

template <typename Walk>
__device__ __forceinline__ PagedRow paged_row(const PagedParams& p, const PagedSegments<Walk>& s,
                                              int row) {
  PagedRow x;
  const int r = s.w.rt * Walk::ROWS + row;
  x.live = r < s.w.g.qlen * p.G;
  const int tok = x.live ? r / p.G : 0;
  x.head = s.w.h * p.G + (x.live ? r - tok * p.G : 0);
  const int base = s.w.g.klen - s.w.g.qlen;
  x.last = p.causal ? base + tok : s.w.g.klen - 1;
  x.all_see = p.causal ? base + s.w.rt * Walk::ROWS / p.G : s.w.g.klen - 1;
  x.token = s.w.g.q0 + tok;
  x.first = x.all_from = x.pos = 0;
  x.slope2 = 0.0f;
  if constexpr (Walk::SHAPED) {
    x.pos = s.w.g.base + tok;
    if (p.slopes) x.slope2 = p.slopes[x.head] * kPagedLog2e;
    if (p.window > 0) {
      x.first = paged_from(p, x.pos);
      const int last_row = min(s.w.rt * Walk::ROWS + Walk::ROWS, s.w.g.qlen * p.G) - 1;
      x.all_from = paged_from(p, s.w.g.base + last_row / p.G);
    }
  }
  return x;
}

// 16 bytes global -> shared without registers or an L1 line (the shared memory
// of these kernels leaves L1 some 20 KB, which the rows of two Q tiles in
// flight would overrun); zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A warp's 32 rows of a Q tile at `q` (128-byte swizzle, blocks of 128 rows x 64
// values) from global memory, zeros for rows that are none; `row`: this lane's
// row in the tile, x what it is.  A row's vectors lie with neighbouring lanes,
// several rows an instruction.  Returns the scale of the lane's row's scores:
// e4m3 pages want Q as fp16, scaled by 2^e to a largest element in [2^7, 2^8).
template <int D, bool E4M3>
__device__ __forceinline__ float paged_load_q(const PagedParams& p, const PagedRow& x, uint32_t q,
                                              int row) {
  constexpr int LPR = D == 64 ? 8 : D == 256 ? 32 : 16;  // lanes a row
  constexpr int RPI = 32 / LPR;                          // rows an instruction
  const int lane = lane_id();
  const int chunk = lane % LPR, grp = lane / LPR;
  const bool has = chunk < D / 8;
  const unsigned long long mine = reinterpret_cast<unsigned long long>(
      p.q + x.token * p.q_token + x.head * p.q_head);  // (of a row that is none: its item's first)
  const unsigned alive = __ballot_sync(0xffffffffu, x.live);
  auto at = [&](int i) -> uint32_t {  // where this lane's vector of instruction i goes
    const int r = (row & ~31) + i * RPI + grp;
    return q + (chunk >> 3) * (128 * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
  };
#pragma unroll 8
  for (int i = 0; i < LPR; ++i) {
    const int r = i * RPI + grp;
    const unsigned long long src = __shfl_sync(0xffffffffu, mine, r);
    if (has)
      cp_async16(at(i), reinterpret_cast<const uint4*>(src) + chunk, (alive >> r) & 1 ? 16 : 0);
  }
  cp_async_wait_all();
  float c = p.scale_log2;
  if constexpr (E4M3) {
#pragma unroll 4
    for (int i = 0; i < LPR; ++i) {
      uint4 v = has ? lds128(at(i)) : make_uint4(0, 0, 0, 0);
      float mx = 0.0f;
      for (uint32_t y : {v.x, v.y, v.z, v.w})
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(y << 16)),
                             fabsf(__uint_as_float(y & 0xffff0000u))));
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      int e = 134 - static_cast<int>(__float_as_uint(mx) >> 23);
      if (mx == 0.0f || !(mx < INFINITY)) e = 0;
      e = min(max(e, -120), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      auto half = [&](uint32_t y) {
        return pack_f16x2(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xffff0000u) * up);
      };
      if (has) sts128(at(i), make_uint4(half(v.x), half(v.y), half(v.z), half(v.w)));
      // The scale to the row's own lane.
      const float down = __shfl_sync(
          0xffffffffu, __uint_as_float(static_cast<uint32_t>(127 - e) << 23), (lane % RPI) * LPR);
      if (lane / RPI == i) c = p.scale_log2 * down;
    }
  }
  return c;
}

// A tile of BN keys from e4m3 bytes (at `raw`, as the copies leave them) to the
// fp16 tile at `dst`, rows before `from` and from `keep` on as zeros; 128 threads.
template <int D, int BN>
__device__ __forceinline__ void paged_convert(uint32_t raw, uint32_t dst, int from, int keep,
                                              int tid) {
  constexpr int PER = 128 / BN;  // threads a row
  constexpr int N = 4;           // chunks of 16 values in flight
  const int r = tid % BN;
  const bool key = r >= from && r < keep;
#pragma unroll
  for (int c0 = 0; c0 < D / 16; c0 += N * PER) {
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * PER + (PER == 1 ? 0 : tid / BN);
      if (c < D / 16)
        v[i] = lds128(raw + (c >> 3) * (BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * PER + (PER == 1 ? 0 : tid / BN);
      if (c >= D / 16) continue;
      if (!key) v[i] = make_uint4(0, 0, 0, 0);  // (+0 in both formats)
      const uint32_t blk = dst + (c >> 2) * (BN * 128) + r * 128;
      sts128(blk + ((((c & 3) * 2) ^ (r & 7)) << 4),
             make_uint4(e4m3x2_f16x2(v[i].x), e4m3x2_f16x2(v[i].x >> 16), e4m3x2_f16x2(v[i].y),
                        e4m3x2_f16x2(v[i].y >> 16)));
      sts128(blk + ((((c & 3) * 2 + 1) ^ (r & 7)) << 4),
             make_uint4(e4m3x2_f16x2(v[i].z), e4m3x2_f16x2(v[i].z >> 16), e4m3x2_f16x2(v[i].w),
                        e4m3x2_f16x2(v[i].w >> 16)));
    }
  }
}

// Rows first .. end - 1 of the bf16 tile at `v` (of BN keys) as zeros; THREADS threads.
template <int SUB, int BN, int THREADS>
__device__ __forceinline__ void paged_zero_rows(uint32_t v, int first, int end, int tid) {
  constexpr int CHUNKS = SUB * 8;  // 16-byte chunks of a row
  for (int x = first * CHUNKS + tid; x < end * CHUNKS; x += THREADS) {
    const int r = x / CHUNKS, c = x % CHUNKS;
    sts128(v + (c >> 3) * (BN * 128) + r * 128 + ((c & 7) << 4), make_uint4(0, 0, 0, 0));
  }
}

// The scores of a row's key tile at TMEM address `s` to P over them, with the
// running reference m and sum l (base 2, scores times c).  `see`: the last key of
// the tile that the row sees, if `mask`.  m is the reference that P is relative to
// (fa_paged.cuh); returns the factor that O and the old l are due (1 while it stays).
// SHAPED: the scores are capped and lowered first (kbase: the tile's first key), and keys
// before x.first are not seen either.
template <int BN, bool F16, bool SHAPED>
__device__ __forceinline__ float paged_softmax(const PagedParams& p, const PagedRow& x,
                                               uint32_t s_addr, bool mask, int kbase, float c,
                                               float& m, float& l, bool& moved) {
  const int see = x.last - kbase;
  float s[BN];
  if constexpr (SHAPED) {
    // All columns at once (a chunk of 1024 tokens behind 15,000, 32 / 8 heads, d = 128, cap, e4m3
    // and bf16: 377 and 338 us with 32 columns, 334 and 312 with 64, 323 and 286 with 128).
    // Over e4m3 pages a row's c takes in a power of two of q, far from 1: its products are
    // brought to the tanh's argument first, so that the coefficients keep within fp32 (with 2^(3e)
    // folded into a row's own coefficients, and out of its c, instead: 347 us for 329).
    const bool cap = p.cap2 > 0.0f;
    const float by = cap ? c / p.cap2 : c;
    float none[1];
    auto load = [&](auto& z, int c0) {
      constexpr int N = sizeof(z) / sizeof(float);
      uint32_t r[N];
#pragma unroll
      for (int q = 0; q < N / 32; ++q)
        tmem_ld32(s_addr + c0 + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * q]));
      tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < N; ++t) z[t] = __uint_as_float(r[t]);
      if (F16 || !cap) {
        const uint64_t by2 = f2_pack(by, by);
#pragma unroll
        for (int t = 0; t < N; t += 2)
          f2_unpack(f2_mul(f2_pack(z[t], z[t + 1]), by2), z[t], z[t + 1]);
      }
    };
    load(s, 0);
    if (cap) shape_scores<BN, true, false, false, !F16>(s, none, p.f, 0.0f, 0.0f, 0.0f, load);
    if (p.slopes) lower_scores<BN>(s, x.slope2, static_cast<float>(x.pos - kbase));
    c = 1.0f;
  } else {
    uint32_t raw[BN];
#pragma unroll
    for (int q4 = 0; q4 < BN / 32; ++q4)
      tmem_ld32(s_addr + q4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&raw[q4 * 32]));
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < BN; ++k) s[k] = __uint_as_float(raw[k]);
  }
  if (mask) {
#pragma unroll
    for (int k = 0; k < BN; ++k)
      if (k > see || (SHAPED && k < x.first - kbase)) s[k] = -INFINITY;
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
  float alpha = 1.0f;
  moved = paged_moves<F16>(mx, c, m);
  if (moved) {
    const float m_new = paged_reference<F16>(mx, c);
    alpha = ex2_approx(m - m_new);
    m = m_new;
  }
  const float m_ref = m == -INFINITY ? 0.0f : m;
  const uint64_t c2 = f2_pack(c, c);
  const uint64_t nm2 = f2_pack(-m_ref, -m_ref);
  uint64_t ps2[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) ps2[u] = 0ull;
  uint32_t pk[BN / 2];
#pragma unroll
  for (int k = 0; k < BN / 2; ++k) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(s[2 * k], s[2 * k + 1]), c2, nm2), x0, x1);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    ps2[k & 3] = f2_add(ps2[k & 3], f2_pack(p0, p1));
    pk[k] = F16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
  }
#pragma unroll
  for (int q4 = 0; q4 < BN / 64; ++q4)
    tmem_st32(s_addr + q4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[q4 * 32]));
  float sum, sum_hi;
  f2_unpack(f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3])), sum, sum_hi);
  l = l * alpha + (sum + sum_hi);
  return alpha;
}

// O of a row (D fp32 columns at TMEM address `o`) times alpha.
template <int D>
__device__ __forceinline__ void paged_rescale(uint32_t o_addr, float alpha) {
#pragma unroll 1
  for (int q4 = 0; q4 < D / 32; ++q4) {
    uint32_t x[32];
    tmem_ld32(o_addr + q4 * 32, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
    tmem_st32(o_addr + q4 * 32, x);
  }
}

// 32 bytes to a 32-byte boundary: a whole sector a lane.
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A row's O out of TMEM (TWO: fa times the one at o_addr plus fb times the one
// at o_addr2): the result if its item lies whole in this CTA, else its part, at
// row `part_row` of the parts.
template <int D, bool E4M3, bool TWO>
__device__ __forceinline__ void paged_store_row(const PagedParams& p, const PagedRow& x,
                                                uint32_t o_addr, uint32_t o_addr2, float fa,
                                                float fb, bool whole, long long part_row, float m,
                                                float l) {
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const float vs = E4M3 ? p.v_scale : 1.0f;  // (vs / l could fall below fp32's range)
  __nv_bfloat16* dst = p.o + x.token * p.o_token + x.head * p.o_head;
  float* part = p.part_o + part_row * D;
  const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
  for (int q4 = 0; q4 < D / 32; ++q4) {
    uint32_t v[32];
    tmem_ld32(o_addr + q4 * 32, v);
    if constexpr (TWO) {
      uint32_t w[32];
      tmem_ld32(o_addr2 + q4 * 32, w);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k)
        v[k] = __float_as_uint(__uint_as_float(v[k]) * fa + __uint_as_float(w[k]) * fb);
    } else {
      tmem_wait_ld();
    }
    if (!x.live) continue;
    if (whole) {
      uint32_t y[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        y[u] = pack_bf16x2(__uint_as_float(v[2 * u]) * inv * vs,
                           __uint_as_float(v[2 * u + 1]) * inv * vs);
      if (wide) {
        stg256(dst + q4 * 32, y);
        stg256(dst + q4 * 32 + 16, y + 8);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<uint4*>(dst + q4 * 32)[k] =
              make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) stg256(part + q4 * 32 + 8 * k, v + 8 * k);
    }
  }
  if (x.live) {
    if (!whole)
      p.part_ml[part_row] = make_float2(m, l);
    else if (p.lse)
      p.lse[x.token * p.Hq + x.head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kPagedLn2;
  }
}

}  // namespace fa
