// Norms of each head's rows of q and k with the position rotation in the same pass, their
// gradients, and the same on the way into a paged cache.
//
//     u = x / sqrt(mean x^2 + eps),   y = R(a) (u o w)
// and from g = R(-a) dy:
//     dw = sum over rows of g o u,    dx = r (g o w - u mean(g o w o u)),  r = u / x.
// All in fp32 up to the one rounding at the end.  Bound by memory: the forward kernel reads and
// writes each row once, the gradient's reads x and dy (it recomputes r and u) and writes dx.
//
// Both take a row by D / 16 lanes (rounded up to a power of two: two of eight idle at d = 96)
// with 16 values each, which add their sums by shuffles among themselves, all lanes of a warp
// together: the loops run to the same count in every lane.  A thread's rows come through shared
// memory by asynchronous copies, several on their way (no other thread reads them: no barrier).
// Appending 8527 tokens of 32 + 8 + 8 heads, d = 128, to e4m3 pages: 36.9 us, 5.2 TB/s (with
// 2 / 3 / 5 / 6 / 8 slots instead of 4: 43.3 / 37.2 / 38.6 / 40.6 / 44.8; two rows at a time in
// registers spilled: 47.3; without the norms 37.4).  The gradient of 8192 positions of 32 + 8
// heads, d = 128: 52.1 us, 4.8 TB/s, with the weights' sums (2 / 4 / 6 slots 57.7 / 52.8 / 54.1;
// one row ahead in registers 77.3).  Half of the issue slots are taken: widening, the two sums
// and the turn are some 200 instructions for a lane's 16 values.
//
// The gradient's thread keeps the sum for dw of its 16 values of a row over all rows that it
// goes through, in fp32; the threads of a block are added in a fixed order through shared
// memory, and the blocks' sums in a fixed order by a second kernel, so that results repeat to
// the bit.  Blocks are shared out between q and k by their rows, so that a block has one
// tensor's weights and sums.

#include <algorithm>

#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kTurnSlots = 4, kGradSlots = 3;  // rows of a thread in shared memory

__host__ __device__ constexpr int row_lanes(int d) { return d == 96 ? 8 : d / 16; }

// Eight values as four packed pairs.
__device__ __forceinline__ void widen8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 narrow8(const uint64_t (&x)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(x[i], f[2 * i], f[2 * i + 1]);
  return pack8(f);
}

__device__ __forceinline__ float f2_sum(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}

// Sum over the LANES lanes (a power of two, aligned) of a row; the whole warp calls this.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// 1 / sqrt(mean of the row's squares + eps) from this lane's 16 values, if it is `on`.
template <int D>
__device__ __forceinline__ float row_factor(const uint64_t (&x)[4], const uint64_t (&y)[4],
                                            float eps, bool on) {
  uint64_t a = f2_mul(x[0], x[0]), b = f2_mul(y[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = f2_fma(x[i], x[i], a);
    b = f2_fma(y[i], y[i], b);
  }
  return rsqrtf(row_sum<row_lanes(D)>(on ? f2_sum(f2_add(a, b)) : 0.0f) * (1.0f / D) + eps);
}

// Eight fp32 values out of shared memory, each time (kept over a thread's rows they spill).
__device__ __forceinline__ void shared8(const float* at, uint64_t (&x)[4]) {
  const uint32_t a = smem_u32(at);
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x[0]), "=l"(x[1]) : "r"(a) : "memory");
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
               : "=l"(x[2]), "=l"(x[3])
               : "r"(a + 16)
               : "memory");
}

// A weight of a norm in fp32.
__device__ __forceinline__ float norm_weight(const void* w, int bf16, int at) {
  if (w == nullptr) return 1.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at])
              : static_cast<const float*>(w)[at];
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The cosines and sines of a position's pairs, as a lane holds those of its eight.
struct Turn {
  uint64_t c[4], s[4], ns[4];
  __device__ __forceinline__ void load(const float* cos, const float* sin) {
    shared8(cos, c);
    shared8(sin, s);
    const uint64_t minus = f2_pack(-1.0f, -1.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) ns[i] = f2_mul(s[i], minus);
  }
  __device__ __forceinline__ void apply(uint64_t (&x)[4], uint64_t (&y)[4],
                                        bool interleaved) const {
    if (interleaved) {  // pairs within x, then within y
      float cf[8], sf[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2_unpack(c[i], cf[2 * i], cf[2 * i + 1]);
        f2_unpack(s[i], sf[2 * i], sf[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(x[i], a, b);
        x[i] = f2_pack(a * cf[i] - b * sf[i], a * sf[i] + b * cf[i]);
        f2_unpack(y[i], a, b);
        y[i] = f2_pack(a * cf[4 + i] - b * sf[4 + i], a * sf[4 + i] + b * cf[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t a = x[i], b = y[i];
        x[i] = f2_fma(a, c[i], f2_mul(b, ns[i]));
        y[i] = f2_fma(a, s[i], f2_mul(b, c[i]));
      }
    }
  }
};

// Where a lane's 16 values lie in a row: two vectors of 8, `gap` apart.
struct Lane {
  bool on, turned;
  int first, gap;
  __device__ __forceinline__ Lane(int u, int d, int half, int interleaved) {
    on = u < d / 16;
    turned = on && u < half / 8;
    first = interleaved ? 16 * u : u < half / 8 ? 8 * u : 2 * half + 16 * (u - half / 8);
    gap = interleaved || u >= half / 8 ? 8 : half;
    if (!on) first = gap = 0;
  }
};

// The angles of `tok` positions from t0: a thread makes those of N of the pairs, from positions
// that it loads well before.
template <int N>
struct Angles {
  int place[N];  // position among the tok; -1: none
  const int* from[N];
  int pos[N];

  __device__ __forceinline__ Angles(const TurnParams& p, int tok) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int i = threadIdx.x + e * kThreads;
      const int w = p.half > 0 ? i / p.half : tok;
      place[e] = w < tok ? w : -1;
      from[e] = nullptr;
      if (p.positions && w < tok) {
        // (four axes a word: the constant cache serves one address of a warp at a time)
        const int pair = i - w * p.half;
        const uint32_t four = reinterpret_cast<const uint32_t*>(p.axis)[pair >> 2];
        from[e] = p.positions + (four >> (8 * (pair & 3)) & 0xffu) * p.axis_stride;
      }
      pos[e] = 0;
    }
  }
  __device__ __forceinline__ void load(const TurnParams& p, long long t0) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const long long t = t0 + place[e];
      if (from[e] && t < p.tokens) {
        const uint32_t b = p.N > 0 ? static_cast<uint32_t>(t) / static_cast<uint32_t>(p.N) : 0;
        pos[e] = from[e][b * p.batch_stride + (t - b * static_cast<long long>(p.N))];
      }
    }
  }
  // Cosines and sines, [position][pair].  seq_pos: the positions where none are given.
  __device__ __forceinline__ void make(const TurnParams& p, const uint64_t* fraction,
                                       const int* seq_pos, float sign, float* cos,
                                       float* sin) const {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (place[e] < 0) continue;
      const int i = threadIdx.x + e * kThreads;
      const float2 a = cos_sin(from[e] ? pos[e] : seq_pos[place[e]],
                               fraction[i - place[e] * p.half], sign);
      cos[i] = a.x;
      sin[i] = a.y;
    }
  }
};

template <int D, int TOK>
struct NormTurnCfg {
  static constexpr int LANES = row_lanes(D);
  static constexpr int HG = kThreads / (LANES * TOK);
  static constexpr int ANGLES = (TOK * D / 2 + kThreads - 1) / kThreads;  // a thread's
  struct Smem {
    uint4 rows[kTurnSlots][2][kThreads];
    float cos[ANGLES * kThreads], sin[ANGLES * kThreads];
    float weight[2][D];  // of q, of k
    uint64_t fraction[D / 2];
    long long place[TOK];  // as find_tokens
    int seq_pos[TOK];
  };
};

// Thread: 16 values of token tt, heads hg, hg + HG, ... of q, then of k (and v).
template <int D, int TOK, int TO>
__global__ void __launch_bounds__(kThreads, TO == kTurnOnly ? 4 : 3)
    fa_norm_turn_kernel(const __grid_constant__ TurnParams p) {
  using C = NormTurnCfg<D, TOK>;
  constexpr int LANES = C::LANES, HG = C::HG;
  constexpr bool APPEND = TO != kTurnOnly;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  typename C::Smem& sm = *reinterpret_cast<typename C::Smem*>(smem_raw);

  grid_launch_dependents();
  grid_dependency_wait();

  const int tid = threadIdx.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * TOK;
  const int tt = tid / LANES % TOK, hg = tid / (LANES * TOK);
  const long long t = t0 + tt;
  const Lane lane(tid % LANES, D, p.half, p.interleaved);
  const int first = lane.first, gap = lane.gap;
  const bool here = t < p.tokens && lane.on;
  // (fewer than 2^31 positions in all)
  const long long b = APPEND ? 0 : static_cast<uint32_t>(t) / static_cast<uint32_t>(p.N);
  const long long n = t - b * p.N;
  const int q_rounds = (p.q.heads + HG - 1) / HG, k_rounds = (p.k.heads + HG - 1) / HG;
  const int rounds = q_rounds + (APPEND ? 2 : 1) * k_rounds;

  // The copies: round `at` takes a head of q, or of k (appending: of k and of v in turn).
  const uint32_t ring = smem_u32(&sm.rows[0][0][tid]);
  const __nv_bfloat16* q_in = p.q.in + (b * p.q.ib + n * p.q.ip + hg * p.q.ih + first);
  const __nv_bfloat16* k_in = p.k.in + (b * p.k.ib + n * p.k.ip + hg * p.k.ih + first);
  const __nv_bfloat16* v_in = APPEND ? p.v.in + (n * p.v.ip + hg * p.v.ih + first) : nullptr;
  int at = 0, at_slot = 0;
  auto copy_row = [&](const __nv_bfloat16*& src, long long step, int head, int heads) {
    if (here && head < heads) {
      const uint32_t dst = ring + at_slot * static_cast<uint32_t>(sizeof(sm.rows[0]));
      copy16_async(dst, src);
      copy16_async(dst + 16 * kThreads, src + gap);
    }
    src += step;
  };
  auto copy = [&]() {
    const int j = at - q_rounds;
    if (j < 0)
      copy_row(q_in, p.q.ih * HG, hg + at * HG, p.q.heads);
    else if (at >= rounds)
      ;
    else if (!APPEND)
      copy_row(k_in, p.k.ih * HG, hg + j * HG, p.k.heads);
    else if (!(j & 1))
      copy_row(k_in, p.k.ih * HG, hg + (j >> 1) * HG, p.k.heads);
    else
      copy_row(v_in, p.v.ih * HG, hg + (j >> 1) * HG, p.k.heads);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++at;
    at_slot = at_slot + 1 == kTurnSlots ? 0 : at_slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kTurnSlots - 1; ++i) copy();

  {
    Angles<C::ANGLES> angles(p, TOK);
    angles.load(p, t0);
    if constexpr (APPEND) find_tokens(p, t0, TOK, sm.place, sm.seq_pos);
    // (fp64 is slow here: once a pair, not once an angle)
    if (tid < p.half) sm.fraction[tid] = turn_fraction(p.inv_freq[tid]);
    for (int i = tid; i < 2 * D; i += kThreads) {
      const int of_k = i >= D, e = of_k ? i - D : i;
      sm.weight[of_k][e] = norm_weight(of_k ? p.k_weight : p.q_weight, p.weight_bf16, e);
    }
    __syncthreads();
    angles.make(p, sm.fraction, sm.seq_pos, p.sign, sm.cos, sm.sin);
  }
  __syncthreads();
  const bool known = here && (!APPEND || sm.seq_pos[tt] != INT_MIN);
  Turn turn;
  const int pairs = lane.turned ? tt * p.half + tid % LANES * 8 : 0;
  turn.load(&sm.cos[pairs], &sm.sin[pairs]);

  int slot = 0;
  auto take = [&](uint4& lo, uint4& hi) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kTurnSlots - 2) : "memory");
    lo = sm.rows[slot][0][tid];  // (of a row that is not there: whatever is, and goes nowhere)
    hi = sm.rows[slot][1][tid];
    slot = slot + 1 == kTurnSlots ? 0 : slot + 1;
    copy();  // (into the slot that the last round has read)
  };
  auto norm = [&](const uint4& lo, const uint4& hi, uint64_t (&x)[4], uint64_t (&y)[4], int of_k) {
    widen8(lo, x);
    widen8(hi, y);
    const float r = row_factor<D>(x, y, p.eps, lane.on);
    const uint64_t r2 = f2_pack(r, r);
    uint64_t wx[4], wy[4];
    shared8(&sm.weight[of_k][first], wx);
    shared8(&sm.weight[of_k][first + gap], wy);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = f2_mul(x[i], f2_mul(r2, wx[i]));
      y[i] = f2_mul(y[i], f2_mul(r2, wy[i]));
    }
    if (lane.turned) turn.apply(x, y, p.interleaved);
  };
  auto rows = [&](int n_rounds, const TurnRows& r, int of_k) {
    __nv_bfloat16* dst = r.out + (b * r.ob + n * r.op + hg * r.oh + first);
    for (int i = 0; i < n_rounds; ++i, dst += r.oh * HG) {
      const bool on = known && hg + i * HG < r.heads;
      uint4 lo, hi;
      take(lo, hi);
      uint64_t x[4], y[4];
      norm(lo, hi, x, y, of_k);
      if (on) {
        *reinterpret_cast<uint4*>(dst) = narrow8(x);
        *reinterpret_cast<uint4*>(dst + gap) = narrow8(y);
      }
    }
  };
  rows(q_rounds, p.q, 0);
  if constexpr (!APPEND) {
    rows(k_rounds, p.k, 1);
  } else {
    using Elem = std::conditional_t<TO == kToBf16, __nv_bfloat16, uint8_t>;
    const long long row0 = sm.place[tt];
    const bool stored = known && row0 >= 0;
    auto put = [&](const uint64_t (&x)[4], const uint64_t (&y)[4], Elem* dst, float scale) {
      if constexpr (TO == kToBf16) {
        *reinterpret_cast<uint4*>(dst) = narrow8(x);
        *reinterpret_cast<uint4*>(dst + gap) = narrow8(y);
      } else {
        float f[8], g[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f2_unpack(x[i], f[2 * i], f[2 * i + 1]);
          f2_unpack(y[i], g[2 * i], g[2 * i + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] *= scale;
          g[e] *= scale;
        }
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
        *reinterpret_cast<uint2*>(dst + gap) =
            make_uint2(pack_e4m3x4(g[0], g[1], g[2], g[3]), pack_e4m3x4(g[4], g[5], g[6], g[7]));
      }
    };
    for (int i = 0; i < k_rounds; ++i) {
      const bool on = stored && hg + i * HG < p.k.heads;
      const long long row = row0 + (hg + i * HG) * p.head_stride + first;
      uint4 lo, hi;
      uint64_t x[4], y[4];
      take(lo, hi);
      norm(lo, hi, x, y, 1);
      if (on) put(x, y, static_cast<Elem*>(p.k_pages) + row, p.k_scale);
      take(lo, hi);
      if (!on) continue;
      Elem* dst = static_cast<Elem*>(p.v_pages) + row;
      if constexpr (TO == kToBf16) {
        *reinterpret_cast<uint4*>(dst) = lo;
        *reinterpret_cast<uint4*>(dst + gap) = hi;
      } else {
        widen8(lo, x);
        widen8(hi, y);
        put(x, y, dst, p.v_scale);
      }
    }
  }
}

template <int D, int TOK, int TO>
cudaError_t launch_norm_tok(const TurnParams& p, cudaStream_t stream) {
  constexpr int kBytes = sizeof(typename NormTurnCfg<D, TOK>::Smem);
  const long long grid = (p.tokens + TOK - 1) / TOK;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = set_smem_limit_once<fa_norm_turn_kernel<D, TOK, TO>>(kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_norm_turn_kernel<D, TOK, TO>, dim3(static_cast<unsigned>(grid)),
                          dim3(kThreads), kBytes, stream, p);
}

template <int D, int TO>
cudaError_t launch_norm_d(const TurnParams& p, cudaStream_t stream) {
  const long long sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  // The most positions a block that give a thread at most ten heads and leave two blocks for every
  // SM, or one where a thread has four heads or fewer (2000 positions of 40 heads, d = 64 / 128 /
  // 256, with 1 / 4 / 8 positions: 13.7 / 6.4 / 8.4 us, 15.7 / 9.2 / 14.3, 21.0 / 16.1 / -; 1025 of
  // 32 with 1 / 4: 7.8 / 5.3, 8.7 / 7.7, 10.0 / 12.9).
  const int heads = p.q.heads + p.k.heads + p.v.heads;
  int tok = 1;
  for (int more : {4, 8, 16}) {
    const int rows = heads * (D / 16) * more;  // of 16 values
    if (rows <= 10 * kThreads && p.tokens >= (rows <= 4 * kThreads ? 1 : 2) * sms * more)
      tok = more;
  }
  switch (tok) {
    case 1: return launch_norm_tok<D, 1, TO>(p, stream);
    case 4: return launch_norm_tok<D, 4, TO>(p, stream);
    case 8: return launch_norm_tok<D, 8, TO>(p, stream);
    default: return launch_norm_tok<D, 16, TO>(p, stream);
  }
}

template <int TO>
cudaError_t launch_norm(const TurnParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_norm_d<64, TO>(p, stream);
    case 96: return launch_norm_d<96, TO>(p, stream);
    case 128: return launch_norm_d<128, TO>(p, stream);
    case 256: return launch_norm_d<256, TO>(p, stream);
  }
  return cudaErrorInvalidValue;
}

constexpr int kGradTok = 16;    // positions a block takes at a time, at most
constexpr int kGradAngles = 2;  // angles a thread makes for them, at most

struct NormGradParams {
  TurnParams t;  // rows: in = dy, out = dx
  TurnRows qx, kx;  // in = x
  int q_blocks;     // blocks of q; the others are k's
  int q_tok, k_tok; // log2 of the positions that a block takes at a time
  float* part;      // [block][D]
};

struct NormGradSmem {
  uint4 rows[kGradSlots][4][kThreads];  // a thread's own: dy, dy + gap, x, x + gap
  float cos[2][kGradAngles * kThreads], sin[2][kGradAngles * kThreads];
  float weight[2 * kMaxPairs];
  uint64_t fraction[kMaxPairs];
};

// A block goes through its positions, a few (1 << tok_log) at a time, and a thread through
// heads hg, hg + HG, ... of its position.  The copies run ahead across steps, as do the angles: one
// barrier a step.
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    fa_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int LANES = row_lanes(D);
  constexpr int SLOTS = kThreads / LANES;  // rows at a time
  extern __shared__ __align__(16) unsigned char smem_raw[];
  NormGradSmem& sm = *reinterpret_cast<NormGradSmem*>(smem_raw);
  static_assert(sizeof(sm.rows) >= sizeof(float) * SLOTS * D, "the sums take the rows' place");

  grid_launch_dependents();
  grid_dependency_wait();

  const TurnParams& t = p.t;
  const int tid = threadIdx.x;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const TurnRows& dy = is_k ? t.k : t.q;
  const TurnRows& xr = is_k ? p.kx : p.qx;
  const int tok_log = is_k ? p.k_tok : p.q_tok;
  const int tok = 1 << tok_log;
  const int block = static_cast<int>(blockIdx.x) - (is_k ? p.q_blocks : 0);
  const int blocks = is_k ? static_cast<int>(gridDim.x) - p.q_blocks : p.q_blocks;
  const int half = t.half;
  const int slot_row = tid / LANES;
  const int tt = slot_row & (tok - 1), hg = slot_row >> tok_log, HG = SLOTS >> tok_log;
  const Lane lane(tid % LANES, D, half, t.interleaved);
  const int first = lane.first, gap = lane.gap;
  const int heads = dy.heads, rounds = (heads + HG - 1) / HG;
  const long long start = static_cast<long long>(block) << tok_log;
  const long long step = static_cast<long long>(blocks) << tok_log;

  // Position tn + tt of a step as batch entry and place, the next step's from this one's.
  struct Place {
    long long t;
    uint32_t b, n;
  };
  auto at_start = [&]() {
    Place x{start + tt, 0, 0};
    x.b = static_cast<uint32_t>(x.t) / static_cast<uint32_t>(t.N);
    x.n = static_cast<uint32_t>(x.t) - x.b * t.N;
    return x;
  };
  auto advance = [&](Place& x) {
    x.t += step;
    x.n += static_cast<uint32_t>(step);
    if (x.n >= static_cast<uint32_t>(t.N)) {
      const uint32_t more = x.n / static_cast<uint32_t>(t.N);
      x.b += more;
      x.n -= more * t.N;
    }
  };

  // The copies: of position c, round `at` of its heads.
  const uint32_t ring = smem_u32(&sm.rows[0][0][tid]);
  Place c = at_start();
  int at = 0, at_slot = 0;
  const __nv_bfloat16* g_in = nullptr;
  const __nv_bfloat16* x_in = nullptr;
  const __nv_bfloat16* const g0 = dy.in + (hg * dy.ih + first);
  const __nv_bfloat16* const x0 = xr.in + (hg * xr.ih + first);
  const long long g_step = dy.ih * HG, x_step = xr.ih * HG, o_step = dy.oh * HG;
  auto place = [&]() {
    g_in = g0 + (c.b * dy.ib + c.n * dy.ip);
    x_in = x0 + (c.b * xr.ib + c.n * xr.ip);
  };
  auto copy = [&]() {
    if (lane.on && c.t < t.tokens && hg + at * HG < heads) {
      const uint32_t dst = ring + at_slot * static_cast<uint32_t>(sizeof(sm.rows[0]));
      copy16_async(dst, g_in);
      copy16_async(dst + 16 * kThreads, g_in + gap);
      copy16_async(dst + 32 * kThreads, x_in);
      copy16_async(dst + 48 * kThreads, x_in + gap);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    at_slot = at_slot + 1 == kGradSlots ? 0 : at_slot + 1;
    g_in += g_step;
    x_in += x_step;
    if (++at == rounds) {
      at = 0;
      advance(c);
      place();
    }
  };
  place();
#pragma unroll 1
  for (int i = 0; i < kGradSlots - 1; ++i) copy();

  const void* w = is_k ? t.k_weight : t.q_weight;
  for (int i = tid; i < D; i += kThreads) sm.weight[i] = norm_weight(w, t.weight_bf16, i);
  uint64_t ax[4], ay[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ax[i] = ay[i] = 0ull;
  Angles<kGradAngles> angles(t, tok);
  angles.load(t, start);
  if (tid < half) sm.fraction[tid] = turn_fraction(t.inv_freq[tid]);
  __syncthreads();
  angles.make(t, sm.fraction, nullptr, -1.0f, sm.cos[0], sm.sin[0]);
  angles.load(t, start + step);

  Place row = at_start();
  __nv_bfloat16* const out0 = dy.out + (hg * dy.oh + first);
  int slot = 0, buf = 0;
  for (long long t0 = start; t0 < t.tokens; t0 += step, buf ^= 1) {
    __syncthreads();  // (what is written from here on was read before this)
    if (t0 + step < t.tokens) {
      angles.make(t, sm.fraction, nullptr, -1.0f, sm.cos[buf ^ 1],
                  sm.sin[buf ^ 1]);
      angles.load(t, t0 + 2 * step);
    }
    Turn turn;
    const int pairs = lane.turned ? tt * half + tid % LANES * 8 : 0;
    turn.load(&sm.cos[buf][pairs], &sm.sin[buf][pairs]);
    __nv_bfloat16* out = out0 + (row.b * dy.ob + row.n * dy.op);
    const bool known = lane.on && row.t < t.tokens;
    advance(row);
    for (int i = 0; i < rounds; ++i, out += o_step) {
      const bool on = known && hg + i * HG < heads;
      asm volatile("cp.async.wait_group %0;" ::"n"(kGradSlots - 2) : "memory");
      uint64_t gx[4], gy[4], x[4], y[4];
      {
        uint4 v[4];  // (of a row that is not there: whatever is, and goes nowhere)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = sm.rows[slot][e][tid];
        widen8(v[0], gx);
        widen8(v[1], gy);
        widen8(v[2], x);
        widen8(v[3], y);
      }
      slot = slot + 1 == kGradSlots ? 0 : slot + 1;
      copy();  // (into the slot that the last round has read)
      const float r = row_factor<D>(x, y, t.eps, lane.on);
      const uint64_t r2 = f2_pack(r, r);
      if (lane.turned) turn.apply(gx, gy, t.interleaved);
      uint64_t wx[4], wy[4];
      shared8(&sm.weight[first], wx);
      shared8(&sm.weight[first + gap], wy);
      uint64_t dot = 0ull;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = f2_mul(x[e], r2);  // u
        y[e] = f2_mul(y[e], r2);
        if (on) {
          ax[e] = f2_fma(gx[e], x[e], ax[e]);
          ay[e] = f2_fma(gy[e], y[e], ay[e]);
        }
        gx[e] = f2_mul(gx[e], wx[e]);
        gy[e] = f2_mul(gy[e], wy[e]);
        dot = f2_fma(gx[e], x[e], f2_fma(gy[e], y[e], dot));
      }
      const float mean = row_sum<LANES>(lane.on ? f2_sum(dot) : 0.0f) * (1.0f / D);
      const uint64_t nm = f2_pack(-mean, -mean);
      if (on) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gx[e] = f2_mul(r2, f2_fma(nm, x[e], gx[e]));
          gy[e] = f2_mul(r2, f2_fma(nm, y[e], gy[e]));
        }
        *reinterpret_cast<uint4*>(out) = narrow8(gx);
        *reinterpret_cast<uint4*>(out + gap) = narrow8(gy);
      }
    }
  }
  // The block's sums, its rows in order.
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float* sums = reinterpret_cast<float*>(sm.rows);
  if (lane.on) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f2_unpack(ax[e], sums[slot_row * D + first + 2 * e], sums[slot_row * D + first + 2 * e + 1]);
      f2_unpack(ay[e], sums[slot_row * D + first + gap + 2 * e],
                sums[slot_row * D + first + gap + 2 * e + 1]);
    }
  }
  __syncthreads();
  for (int i = tid; i < D; i += kThreads) {
    float s = 0.0f;
    for (int k = 0; k < SLOTS; ++k) s += sums[k * D + i];
    p.part[static_cast<long long>(blockIdx.x) * D + i] = s;
  }
}

// dw of q (blockIdx.y = 0) and of k (1), 32 values a block: the sums of their blocks, by 32
// threads a value, each in order, then those in order.
__global__ void __launch_bounds__(1024)
    fa_norm_weight_kernel(const float* part, int d, int q_blocks, int blocks, float* dqw,
                          float* dkw) {
  __shared__ float sums[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  float* out = blockIdx.y == 0 ? dqw : dkw;
  if (out == nullptr) return;  // (the whole block)
  const int b0 = blockIdx.y == 0 ? 0 : q_blocks, b1 = blockIdx.y == 0 ? q_blocks : blocks;
  const int i = threadIdx.x % 32, g = threadIdx.x / 32;
  const float* column = part + blockIdx.x * 32 + i;
  float s = 0.0f;
#pragma unroll 8
  for (int b = b0 + g; b < b1; b += 32) s += column[static_cast<long long>(b) * d];
  sums[g][i] = s;
  __syncthreads();
  if (g == 0) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sums[k][i];
    out[blockIdx.x * 32 + i] = s;
  }
}

// Blocks of the gradient's kernel, and so of its workspace.
int grad_blocks() { return 2 * sm_count(); }

template <int D>
cudaError_t launch_grad_d(NormGradParams& p, float* dqw, float* dkw, cudaStream_t stream) {
  const int most = grad_blocks();
  if (most < 2) return cudaErrorInvalidDevice;
  // Positions at a time, of which a block's threads make kGradAngles angles each at most: enough
  // that all threads have a row, and then the most that leave a thread eight rows and the blocks
  // four steps each.  The blocks are
  // shared out by the work, a step's beside its rows counted as one row (by rows alone, with k's
  // steps of one row each: 64.2 us instead of 53.8; four rows or more instead of eight: 52.8
  // instead of 52.2).
  constexpr int SLOTS = kThreads / row_lanes(D);
  const int all = p.t.q.heads + p.t.k.heads;
  auto tok_for = [&](int heads) {
    int log = 0;
    while ((2 << log) <= kGradTok && (2 << log) <= SLOTS &&
           (p.t.half << log) * 2 <= kGradAngles * kThreads &&
           ((SLOTS >> log) > heads ||
            ((SLOTS >> log) * 8 > heads &&
             p.t.tokens * all >= static_cast<long long>(most) * heads * (8 << log))))
      ++log;
    return log;
  };
  auto steps = [&](int log) { return (p.t.tokens + (1 << log) - 1) >> log; };
  auto work = [&](int heads, int log) {
    const int at_once = SLOTS >> log;
    return steps(log) * ((heads + at_once - 1) / at_once + 1);
  };
  p.q_tok = tok_for(p.t.q.heads);
  int kb = 0;
  if (p.t.k.heads > 0) {
    p.k_tok = tok_for(p.t.k.heads);
    const long long of_q = work(p.t.q.heads, p.q_tok), of_k = work(p.t.k.heads, p.k_tok);
    kb = static_cast<int>((most * of_k + (of_q + of_k) / 2) / (of_q + of_k));
    kb = static_cast<int>(std::min<long long>(std::min(std::max(kb, 1), most - 1),
                                              steps(p.k_tok)));
  }
  const int qb = static_cast<int>(std::min<long long>(most - kb, steps(p.q_tok)));
  p.q_blocks = qb;
  cudaError_t e = set_smem_limit_once<fa_norm_grad_kernel<D>>(sizeof(NormGradSmem));
  if (e != cudaSuccess) return e;
  e = launch_dependent(fa_norm_grad_kernel<D>, dim3(qb + kb), dim3(kThreads),
                       sizeof(NormGradSmem), stream, p);
  if (e != cudaSuccess || (!dqw && !dkw)) return e;
  return launch_dependent(fa_norm_weight_kernel, dim3(D / 32, 2), dim3(1024), 0, stream,
                          static_cast<const float*>(p.part), D, qb, qb + kb, dqw, dkw);
}

bool put_norm(TurnParams& p, const fa_head_norm* n) {
  if (!n || !std::isfinite(n->eps) || !(n->eps > 0.0f)) return false;
  if (n->weight_dtype != FA_NORM_F32 && n->weight_dtype != FA_NORM_BF16) return false;
  for (const void* w : {n->q_weight, n->k_weight})
    if (reinterpret_cast<uintptr_t>(w) & 15u) return false;
  p.q_weight = n->q_weight;
  p.k_weight = n->k_weight;
  p.weight_bf16 = n->weight_dtype == FA_NORM_BF16;
  p.eps = n->eps;
  return true;
}

bool put_inputs(TurnRows& R, const fa_rotary_rows& r, int heads) {
  if (!r.in || (reinterpret_cast<uintptr_t>(r.in) & 15u) || r.heads != heads) return false;
  for (long long s : {r.in_batch, r.in_head, r.in_pos})
    if (s < 0 || s % 8 != 0) return false;
  R = TurnRows{static_cast<const __nv_bfloat16*>(r.in), nullptr, r.in_batch, r.in_head, r.in_pos,
               0, 0, 0, r.heads};
  return true;
}

size_t workspace_bytes(int d) { return static_cast<size_t>(grad_blocks()) * d * sizeof(float); }

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_norm_rotary(const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N, int d,
                         const fa_head_norm* norm, const int* positions, long long axis_stride,
                         long long batch_stride, const fa_rotary_spec* spec, cudaStream_t stream) {
  using namespace fa;
  TurnParams p{};
  const fa_status st =
      put_turn(p, q, k, B, N, d, positions, axis_stride, batch_stride, spec, 1.0f);
  if (st != FA_OK) return st;
  if (!put_norm(p, norm)) return FA_ERR_INVALID_ARGUMENT;
  return launch_norm<kTurnOnly>(p, d, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_norm_rotary_backward_workspace_bytes(int d) {
  return d == 64 || d == 96 || d == 128 || d == 256 ? fa::workspace_bytes(d) : 0;
}

fa_status fa_norm_rotary_backward(const fa_rotary_rows* dq, const fa_rotary_rows* dk,
                                  const fa_rotary_rows* q, const fa_rotary_rows* k, int B, int N,
                                  int d, const fa_head_norm* norm, float* dq_weight,
                                  float* dk_weight, const int* positions, long long axis_stride,
                                  long long batch_stride, const fa_rotary_spec* spec,
                                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace fa;
  NormGradParams p{};
  const fa_status st =
      put_turn(p.t, dq, dk, B, N, d, positions, axis_stride, batch_stride, spec, -1.0f);
  if (st != FA_OK) return st;
  if (!put_norm(p.t, norm) || !q || !dk != !k || !put_inputs(p.qx, *q, dq->heads) ||
      (k && !put_inputs(p.kx, *k, dk->heads)) || (dk_weight && !dk))
    return FA_ERR_INVALID_ARGUMENT;
  for (const void* x : {static_cast<const void*>(dq_weight), static_cast<const void*>(dk_weight)})
    if (reinterpret_cast<uintptr_t>(x) & 3u) return FA_ERR_INVALID_ARGUMENT;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes == 0 ||
      workspace_bytes < fa::workspace_bytes(d))
    return FA_ERR_INVALID_ARGUMENT;
  p.part = static_cast<float*>(workspace);
  const cudaError_t e = d == 64    ? launch_grad_d<64>(p, dq_weight, dk_weight, stream)
                        : d == 96  ? launch_grad_d<96>(p, dq_weight, dk_weight, stream)
                        : d == 128 ? launch_grad_d<128>(p, dq_weight, dk_weight, stream)
                                   : launch_grad_d<256>(p, dq_weight, dk_weight, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_paged_append_norm(const fa_paged_cache* cache, const fa_paged_batch* batch,
                               const void* k, long long k_token, long long k_head, const void* v,
                               long long v_token, long long v_head, int T, const void* q,
                               long long q_token, long long q_head, void* q_out, long long qo_token,
                               long long qo_head, int H_q, const fa_head_norm* norm,
                               const fa_rotary_spec* spec, const int* positions,
                               long long axis_stride, cudaStream_t stream) {
  using namespace fa;
  TurnParams p{};
  if (!put_norm(p, norm)) return FA_ERR_INVALID_ARGUMENT;
  bool nothing = false;
  const fa_status st =
      put_append(p, cache, batch, k, k_token, k_head, v, v_token, v_head, T, q, q_token, q_head,
                 q_out, qo_token, qo_head, H_q, spec, positions, axis_stride, &nothing);
  if (st != FA_OK || nothing) return st;
  const cudaError_t e = cache->dtype == FA_CACHE_BF16
                            ? launch_norm<kToBf16>(p, cache->d, stream)
                            : launch_norm<kToE4m3>(p, cache->d, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
