// Norms of each head's rows of q and k with the position rotation in the same pass, their
// gradients, and the same on the way into a paged cache.
//
//     u = x / sqrt(mean x^2 + eps),   y = R(a) (u o w)
// and from g = R(-a) dy:
//     dw = sum over rows of g o u,    dx = r (g o w - u mean(g o w o u)),  r = u / x.
// The forward kernel is fa_rotary.cuh's with NORM.  The gradient's, here, recomputes r and u
// from x, which it has to read anyway: bound by memory, three rows' bytes a row.
//
// A thread keeps the sum for dw of its 16 values of a row over all rows that it goes
// through, in fp32; the threads of a block are added in a fixed order through shared
// memory, and the blocks' sums in a fixed order by a second kernel, so that results repeat to
// the bit.  Blocks are shared out between q and k by their rows, so that a block has one
// tensor's weights and sums.

#include <algorithm>

#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kMaxTok = 16;  // positions a block of the gradient's takes at a time, at most

struct NormGradParams {
  TurnParams t;  // rows: in = dy, out = dx
  TurnRows qx, kx;  // in = x
  int q_blocks;     // blocks of q; the others are k's
  int q_tok, k_tok; // log2 of the positions that a block takes at a time
  float* part;      // [block][D]
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    fa_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int LANES = row_lanes(D, true);
  constexpr int SLOTS = kThreads / LANES;  // rows at a time
  __shared__ __align__(16) float2 cs[kMaxTok][kMaxPairs];
  __shared__ uint64_t fraction[kMaxPairs];
  static_assert(sizeof(cs) >= sizeof(float) * SLOTS * D, "the sums take the angles' place");

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
  const int u = tid % LANES, slot = tid / LANES;
  const int tt = slot & (tok - 1), hg = slot >> tok_log, HG = SLOTS >> tok_log;
  const bool lane_on = LANES * 16 == D || u < D / 16;
  const bool turned = u < half / 8 && lane_on;
  const int first = t.interleaved ? 16 * u : u < half / 8 ? 8 * u : 2 * half + 16 * (u - half / 8);
  const int gap = t.interleaved || u >= half / 8 ? 8 : half;

  float wx[8], wy[8], ax[8], ay[8];
  const void* w = lane_on ? (is_k ? t.k_weight : t.q_weight) : nullptr;
  load_weights(w, t.weight_bf16, first, wx);
  load_weights(w, t.weight_bf16, first + gap, wy);
#pragma unroll
  for (int e = 0; e < 8; ++e) ax[e] = ay[e] = 0.0f;
  if (tid < half) fraction[tid] = turn_fraction(t.inv_freq[tid]);

  for (long long t0 = static_cast<long long>(block) << tok_log; t0 < t.tokens;
       t0 += static_cast<long long>(blocks) << tok_log) {
    __syncthreads();
    for (int i = tid; i < tok * half; i += kThreads) {
      const int wi = i / half, pair = i - wi * half;
      const long long tw = t0 + wi;
      if (tw >= t.tokens) break;
      const long long bw = static_cast<uint32_t>(tw) / static_cast<uint32_t>(t.N);
      const int pos =
          t.positions[t.axis[pair] * t.axis_stride + bw * t.batch_stride + (tw - bw * t.N)];
      cs[wi][pair] = cos_sin(pos, fraction[pair], -1.0f);
    }
    __syncthreads();
    const long long tn = t0 + tt;
    if (tn >= t.tokens) continue;  // (a row's lanes together)
    const long long b = static_cast<uint32_t>(tn) / static_cast<uint32_t>(t.N);
    const long long n = tn - b * t.N;
    float2 t8[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 v = *reinterpret_cast<const float4*>(&cs[tt][turned ? 8 * u + 2 * e : 0]);
      t8[2 * e] = make_float2(v.x, v.y);
      t8[2 * e + 1] = make_float2(v.z, v.w);
    }
    const __nv_bfloat16* g_in = dy.in + (b * dy.ib + n * dy.ip + hg * dy.ih + first);
    const __nv_bfloat16* x_in = xr.in + (b * xr.ib + n * xr.ip + hg * xr.ih + first);
    __nv_bfloat16* out = dy.out + (b * dy.ob + n * dy.op + hg * dy.oh + first);
    uint4 g0{}, g1{}, x0{}, x1{};
    auto load = [&]() {
      g0 = *reinterpret_cast<const uint4*>(g_in);
      g1 = *reinterpret_cast<const uint4*>(g_in + gap);
      x0 = *reinterpret_cast<const uint4*>(x_in);
      x1 = *reinterpret_cast<const uint4*>(x_in + gap);
      g_in += dy.ih * HG;
      x_in += xr.ih * HG;
    };
    if (lane_on && hg < dy.heads) load();
    for (int h = hg; h < dy.heads; h += HG) {
      float gx[8], gy[8], xx[8], xy[8];
      unpack8(g0, gx);
      unpack8(g1, gy);
      unpack8(x0, xx);
      unpack8(x1, xy);
      if (lane_on && h + HG < dy.heads) load();  // the next head's, while this one is summed
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(xx[e], xx[e], fmaf(xy[e], xy[e], ss));
      const float r = rsqrtf(row_sum<LANES>(ss) * (1.0f / D) + t.eps);
      if (turned) {
        if (t.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = gx[2 * e], a1 = gx[2 * e + 1], b0 = gy[2 * e], b1 = gy[2 * e + 1];
            gx[2 * e] = a0 * t8[e].x - a1 * t8[e].y;
            gx[2 * e + 1] = a0 * t8[e].y + a1 * t8[e].x;
            gy[2 * e] = b0 * t8[e + 4].x - b1 * t8[e + 4].y;
            gy[2 * e + 1] = b0 * t8[e + 4].y + b1 * t8[e + 4].x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a0 = gx[e], b0 = gy[e];
            gx[e] = a0 * t8[e].x - b0 * t8[e].y;
            gy[e] = a0 * t8[e].y + b0 * t8[e].x;
          }
        }
      }
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xx[e] *= r;  // u
        xy[e] *= r;
        ax[e] = fmaf(gx[e], xx[e], ax[e]);
        ay[e] = fmaf(gy[e], xy[e], ay[e]);
        gx[e] *= wx[e];
        gy[e] *= wy[e];
        dot = fmaf(gx[e], xx[e], fmaf(gy[e], xy[e], dot));
      }
      const float mean = row_sum<LANES>(dot) * (1.0f / D);
      if (lane_on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          gx[e] = r * fmaf(-mean, xx[e], gx[e]);
          gy[e] = r * fmaf(-mean, xy[e], gy[e]);
        }
        *reinterpret_cast<uint4*>(out) = pack8(gx);
        *reinterpret_cast<uint4*>(out + gap) = pack8(gy);
      }
      out += dy.oh * HG;
    }
  }
  // The block's sums, its rows in order.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(cs);
  if (lane_on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[slot * D + first + e] = ax[e];
      sums[slot * D + first + gap + e] = ay[e];
    }
  }
  __syncthreads();
  for (int i = tid; i < D; i += kThreads) {
    float s = 0.0f;
    for (int k = 0; k < SLOTS; ++k) s += sums[k * D + i];
    p.part[static_cast<long long>(blockIdx.x) * D + i] = s;
  }
}

// dw of q (block 0) and of k (block 1): the sums of their blocks, added in order by eight
// threads a value.
constexpr int kSumThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kSumThreads)
    fa_norm_weight_kernel(const float* part, int q_blocks, int blocks, float* dqw, float* dkw) {
  constexpr int GROUPS = kSumThreads / D;
  __shared__ float sums[GROUPS][D];
  grid_launch_dependents();
  grid_dependency_wait();
  float* out = blockIdx.x == 0 ? dqw : dkw;
  if (out == nullptr) return;  // (the whole block)
  const int b0 = blockIdx.x == 0 ? 0 : q_blocks, b1 = blockIdx.x == 0 ? q_blocks : blocks;
  const int i = threadIdx.x % D, g = threadIdx.x / D;
  if (g < GROUPS) {
    float s = 0.0f;
#pragma unroll 4
    for (int b = b0 + g; b < b1; b += GROUPS) s += part[static_cast<long long>(b) * D + i];
    sums[g][i] = s;
  }
  __syncthreads();
  if (g == 0) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) s += sums[k][i];
    out[i] = s;
  }
}

// Blocks of the gradient's kernel, and so of its workspace.
int grad_blocks() { return 2 * sm_count(); }

template <int D>
cudaError_t launch_grad_d(NormGradParams& p, float* dqw, float* dkw, cudaStream_t stream) {
  // Positions at a time: as many as leave a thread four heads or more to go through..
  constexpr int SLOTS = kThreads / row_lanes(D, true);
  auto tok_for = [&](int heads) {
    int log = 0;
    while ((2 << log) <= kMaxTok && (2 << log) <= SLOTS && (SLOTS >> log) * 4 > heads) ++log;
    return log;
  };
  p.q_tok = tok_for(p.t.q.heads);
  p.k_tok = tok_for(std::max(p.t.k.heads, 1));
  const int most = grad_blocks();
  if (most < 2) return cudaErrorInvalidDevice;
  auto need = [&](int tok) {
    return static_cast<int>(std::min<long long>((p.t.tokens + (1 << tok) - 1) >> tok, most));
  };
  int kb = 0;
  int qb = std::min(need(p.q_tok), most);
  if (p.t.k.heads > 0) {
    // blocks in proportion to rows, one at least
    kb = static_cast<int>(static_cast<long long>(most) * p.t.k.heads /
                          (p.t.q.heads + p.t.k.heads));
    kb = std::min(std::max(kb, 1), std::min(need(p.k_tok), most - 1));
    qb = std::min(qb, most - kb);
  }
  p.q_blocks = qb;
  const cudaError_t e = launch_dependent(fa_norm_grad_kernel<D>, dim3(qb + kb), dim3(kThreads), 0,
                                         stream, p);
  if (e != cudaSuccess || (!dqw && !dkw)) return e;
  return launch_dependent(fa_norm_weight_kernel<D>, dim3(2), dim3(kSumThreads), 0, stream,
                          static_cast<const float*>(p.part), qb, qb + kb, dqw, dkw);
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
  return launch_turn<kTurnOnly, true>(p, d, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
                            ? launch_turn<kToBf16, true>(p, cache->d, stream)
                            : launch_turn<kToE4m3, true>(p, cache->d, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
