// Entry points of attention with shaped scores: checks, the choice of kernels, and the pass
// that tells the dK/dV kernel which query tiles see which keys.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "fa_internal.h"
#include "fa_paged_host.h"
#include "fa_scores.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

// The union of the spans of each query tile's rows, tiles[b][i], one block a tile: the dK/dV
// kernel finds the query tiles of its keys in it (8 bytes for every 128 queries).
__global__ void __launch_bounds__(128) fa_span_tiles_kernel(const ScoreParams p, int2* tiles,
                                                            int n_qtiles) {
  __shared__ KeySpan hulls[4];
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.x / n_qtiles;
  const int i = blockIdx.x - b * n_qtiles;
  const KeySpan h = warp_hull(row_span(p, b, i * 128 + static_cast<int>(threadIdx.x)));
  if ((threadIdx.x & 31) == 0) hulls[threadIdx.x >> 5] = h;
  __syncthreads();
  if (threadIdx.x == 0)
    tiles[blockIdx.x] =
        make_int2(min(min(hulls[0].lo, hulls[1].lo), min(hulls[2].lo, hulls[3].lo)),
                  max(max(hulls[0].hi, hulls[1].hi), max(hulls[2].hi, hulls[3].hi)));
}

// dV (block row 0) and dK (1): the sums of `split` CTAs, added in order; four values a thread.
__global__ void __launch_bounds__(256) fa_scores_sum_kernel(const float4* part, int split,
                                                            long long n4, uint2* dv, uint2* dk) {
  grid_launch_dependents();
  grid_dependency_wait();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4* src = part + blockIdx.y * split * n4 + i;
  float4 s = src[0];
  for (int c = 1; c < split; ++c) {
    const float4 x = src[c * n4];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  (blockIdx.y == 0 ? dv : dk)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// CTAs that share a key tile in the dK/dV kernel: 1, 2, 4 or 8, for which the longest of them
// and the average SM finish first, in steps of 128 queries by one key tile (about 1.5 us): a
// CTA's start and end cost some three, and the shares' sums what their bytes take.  Windows and
// the masks that spans bring are not known here: the steps are those of the causal mask, or all,
// and no split has been timed under the others.  The whole backward with 1 / 2 / 4 / 8 (us; q and key heads, positions): 16/4, 8192, d = 128, causal: 644
// / 637 / 683 / 777; 16/4, 4096, d = 64: 227 / 151 / 158 / 182; 8/1, 4096, d = 128, full: 446 / 265 /
// 181 / 192; 32/32, 2048, d = 128: 131 / 208 / 305 / 477.  The choice loses 6 % to the best of
// the four on two of ten shapes, and nothing on the others.
int dkdv_split(const ScoreParams& p, int d, int sms) {
  const long long keys = d == 256 ? 64 : 128;
  const long long n_k = (p.Nk + keys - 1) / keys, n_q = (p.Nq + 127) / 128;
  const long long units = n_k * p.B * p.Hkv;
  const double longest = static_cast<double>(p.G) * n_q;
  const double total = longest * units * (p.causal && p.q_offset == 0 ? 0.5 : 1.0);
  int best = 1;
  double least = 0.0;
  for (int split : {1, 2, 4, 8}) {
    const double ctas = static_cast<double>(units) * split;
    const double each = longest / split + 3.0;
    const double average = (total + 3.0 * ctas) / sms;
    const double sums =
        split == 1 ? 0.0
                   : 2.0 + 2.0 * split * p.B * p.Hkv * static_cast<double>(p.Nk) * d / (6e3 * sms);
    // (the last CTAs of a causal order are short ones; of any other, as long as all)
    const double t = std::max(each, average + (p.causal ? 0.25 : 0.5) * each) + sums;
    if (split == 1 || t < least) {
      best = split;
      least = t;
    }
  }
  return best;
}

// D, the tiles' spans and the shares' sums, each on a 256-byte boundary.
struct Scratch {
  size_t tiles, part, total;
  int split;
};
Scratch scratch_of(const ScoreParams& p, int d, int sms) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Scratch s;
  s.split = dkdv_split(p, d, sms);
  s.tiles = up(static_cast<size_t>(p.B) * p.Hq * p.Nq * sizeof(float));
  s.part = s.tiles + up(static_cast<size_t>(p.B) * ((p.Nq + 127) / 128) * sizeof(int2));
  s.total = s.part + (s.split > 1 ? 2ull * s.split * p.B * p.Hkv * p.Nk * d * sizeof(float) : 0) +
            240;
  return s;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

fa_status put_scores(ScoreParams* p, const fa_score_spec* spec, float scale) {
  p->scale = scale;
  p->f = score_factors(scale * kScoreLog2e, 0.0f);
  p->slopes = nullptr;
  p->window = 0;
  if (!std::isfinite(p->f.k) || !(p->f.k > 0.0f)) return FA_ERR_INVALID_ARGUMENT;
  if (!spec) return FA_OK;
  if (!std::isfinite(spec->softcap) || spec->softcap < 0.0f || spec->window < 0)
    return FA_ERR_INVALID_ARGUMENT;
  if (spec->softcap > 0.0f) {
    const float k = scale / spec->softcap, cap2 = spec->softcap * kScoreLog2e;
    // (the tanh takes 2 log2(e) k)
    if (!std::isfinite(3.0f * k) || !(k >= 1.2e-38f) || !std::isfinite(2.0f * cap2) ||
        !(cap2 >= 1.2e-38f))
      return FA_ERR_INVALID_ARGUMENT;
    p->f = score_factors(k, cap2);
  }
  if (!aligned(spec->slopes, 4)) return FA_ERR_INVALID_ARGUMENT;
  p->slopes = spec->slopes;
  p->window = spec->window;
  return FA_OK;
}

int score_mode(const ScoreParams& p) {
  return (p.f.cap2 > 0.0f ? kScoreCap : 0) + (p.slopes ? kScoreBias : 0);
}

namespace {

fa_status check(ScoreParams* p, int B, int H_q, int H_kv, int N_q, int N_kv, int d, float scale,
                int causal, int q_offset, const fa_score_spec* spec, const fa_key_spans* spans) {
  fa_status st = validate(B, H_q, H_kv, N_q, d, scale, causal);
  if (st != FA_OK) return st;
  if (N_kv < 1 || q_offset < 0) return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<double>(q_offset) + N_q + 128 >= 2147483647.0 || N_kv > 2147483647 - 256)
    return FA_ERR_INVALID_ARGUMENT;
  if (static_cast<double>(B) * H_kv * N_kv * d >= 1099511627776.0) return FA_ERR_INVALID_ARGUMENT;
  st = put_scores(p, spec, scale);
  if (st != FA_OK) return st;
  p->first = p->end = nullptr;
  p->span_batch = 0;
  if (spans) {
    if (!aligned(spans->first, 4) || !aligned(spans->end, 4) || spans->batch_stride < 0)
      return FA_ERR_INVALID_ARGUMENT;
    p->first = spans->first;
    p->end = spans->end;
    p->span_batch = spans->batch_stride;
  }
  p->causal = causal;
  p->q_offset = q_offset;
  p->Nq = N_q;
  p->Nk = N_kv;
  p->Hq = H_q;
  p->Hkv = H_kv;
  p->G = H_q / H_kv;
  p->B = B;
  return FA_OK;
}

bool maps(ScoreMaps* m, const void* q, const void* k, const void* v, const void* dO,
          const ScoreParams& p, int d) {
  const long long qplanes = static_cast<long long>(p.B) * p.Hq;
  const long long kvplanes = static_cast<long long>(p.B) * p.Hkv;
  return encode_map_bf16(&m->q, q, d, p.Nq, qplanes) &&
         (!dO || encode_map_bf16(&m->dO, dO, d, p.Nq, qplanes)) &&
         encode_map_kv_bf16(&m->k, k, d, p.Nk, kvplanes) &&
         encode_map_kv_bf16(&m->v, v, d, p.Nk, kvplanes);
}

// dQ first: it may sum D anew (fa_scores_dq.cuh), for the dK/dV kernel as well.
template <int D>
cudaError_t backward_d(const ScoreMaps& m, const float* lse, float* Dv, const int2* tiles, void* dq,
                       void* dk, void* dv, float* part, int split, const ScoreParams& p,
                       cudaStream_t stream) {
  const int mode = score_mode(p);
  cudaError_t e = launch_scores_dq<D>(m, lse, Dv, dq, p, mode, stream);
  if (e == cudaSuccess)
    e = launch_scores_dkdv<D>(m, lse, Dv, tiles, dk, dv, part, split, p, mode, stream);
  if (e != cudaSuccess || split == 1) return e;
  const long long n4 = static_cast<long long>(p.B) * p.Hkv * p.Nk * (D / 4);
  const long long blocks = (n4 + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(fa_scores_sum_kernel, dim3(static_cast<unsigned>(blocks), 2), dim3(256),
                          0, stream, reinterpret_cast<const float4*>(part), split, n4,
                          static_cast<uint2*>(dv), static_cast<uint2*>(dk));
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_forward_scores(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                            int H_q, int H_kv, int N_q, int N_kv, int d, float scale, int causal,
                            int q_offset, const fa_score_spec* spec, const fa_key_spans* spans,
                            cudaStream_t stream) {
  using namespace fa;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARGUMENT;
  ScoreParams p;
  const fa_status st =
      check(&p, B, H_q, H_kv, N_q, N_kv, d, scale, causal, q_offset, spec, spans);
  if (st != FA_OK) return st;
  for (const void* x : {q, k, v, static_cast<const void*>(o)})
    if (!aligned(x, 16)) return FA_ERR_INVALID_ARGUMENT;
  if (!aligned(lse, 4)) return FA_ERR_INVALID_ARGUMENT;
  p.err = device_error_word();
  if (!p.err) return FA_ERR_CUDA;
  ScoreMaps m;
  if (!maps(&m, q, k, v, nullptr, p, d)) return FA_ERR_CUDA;
  const int mode = score_mode(p);
  const cudaError_t e = d == 64    ? launch_scores_forward<64>(m, o, lse, p, mode, stream)
                        : d == 96  ? launch_scores_forward<96>(m, o, lse, p, mode, stream)
                        : d == 128 ? launch_scores_forward<128>(m, o, lse, p, mode, stream)
                                   : launch_scores_forward<256>(m, o, lse, p, mode, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_backward_scores(const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dO, void* dq, void* dk, void* dv, int B,
                             int H_q, int H_kv, int N_q, int N_kv, int d, float scale, int causal,
                             int q_offset, const fa_score_spec* spec, const fa_key_spans* spans,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace fa;
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID_ARGUMENT;
  ScoreParams p;
  const fa_status st =
      check(&p, B, H_q, H_kv, N_q, N_kv, d, scale, causal, q_offset, spec, spans);
  if (st != FA_OK) return st;
  for (const void* x : {q, k, v, o, dO, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!aligned(x, 16)) return FA_ERR_INVALID_ARGUMENT;
  if (!aligned(lse, 4)) return FA_ERR_INVALID_ARGUMENT;
  const long long rows = static_cast<long long>(B) * H_q * N_q;
  const int n_qtiles = (N_q + 127) / 128;
  const long long n_tiles = static_cast<long long>(B) * n_qtiles;
  if (n_tiles > 0x7fffffffLL) return FA_ERR_INVALID_ARGUMENT;
  if (!workspace || !aligned(workspace, 16)) return FA_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  const Scratch at = scratch_of(p, d, sms);
  if (workspace_bytes < at.total) return FA_ERR_INVALID_ARGUMENT;
  if (sms < 1) return FA_ERR_CUDA;
  p.err = device_error_word();
  if (!p.err) return FA_ERR_CUDA;
  ScoreMaps m;
  if (!maps(&m, q, k, v, dO, p, d)) return FA_ERR_CUDA;
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) &
                                     ~static_cast<uintptr_t>(255));
  float* Dv = reinterpret_cast<float*>(ws);
  int2* tiles = reinterpret_cast<int2*>(ws + at.tiles);
  float* part = reinterpret_cast<float*>(ws + at.part);
  cudaError_t e = launch_dependent(fa_span_tiles_kernel, dim3(static_cast<unsigned>(n_tiles)),
                                   dim3(128), 0, stream, p, tiles, n_qtiles);
  if (e == cudaSuccess) e = launch_preprocess(o, dO, Dv, rows, d, stream);
  if (e == cudaSuccess)
    e = d == 64    ? backward_d<64>(m, lse, Dv, tiles, dq, dk, dv, part, at.split, p, stream)
        : d == 96  ? backward_d<96>(m, lse, Dv, tiles, dq, dk, dv, part, at.split, p, stream)
        : d == 128 ? backward_d<128>(m, lse, Dv, tiles, dq, dk, dv, part, at.split, p, stream)
                   : backward_d<256>(m, lse, Dv, tiles, dq, dk, dv, part, at.split, p, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_backward_scores_workspace_bytes(int B, int H_q, int H_kv, int N_q, int N_kv, int d,
                                          int causal, int q_offset) {
  using namespace fa;
  ScoreParams p;
  if (check(&p, B, H_q, H_kv, N_q, N_kv, d, 1.0f, causal, q_offset, nullptr, nullptr) != FA_OK)
    return 0;
  return scratch_of(p, d, sm_count()).total;
}

}  // extern "C"
