// Host side of the shaped-score entry points, between their translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

// What a score is multiplied by, and its tanh.
struct ScoreFactors {
  float k;      // CAP: the tanh's factor of q.k, scale / softcap; otherwise scale log2(e)
  float cap2;   // softcap log2(e); 0: none
  // cap2 tanh(s k) = s (a0 + a1 s^2 + a2 s^4 + a3 s^6) for |s| <= range; below 0: these do not
  // hold the polynomial
  float a[4];
  float range;
  float neg_inv_cap_sq;  // -1 / cap2^2
};

// tanh(y) = y (c0 + c1 y^2 + c2 y^4 + c3 y^6) for |y| <= kTanhRange (fa_scores.cuh).
constexpr float kTanhRange = 0.4f;
constexpr float kTanhC0 = 0.9999999019009195f;
constexpr float kTanhC1 = -0.33331362458867403f;
constexpr float kTanhC2 = 0.13270976757985897f;
constexpr float kTanhC3 = -0.04755360359006216f;

// For k = 1 the coefficients are the tanh's own times cap2.  Otherwise they hold caps up to some
// thousands at usual scales; beyond (and where any of them leaves fp32's range otherwise) range is
// -1, and shape_columns takes each score by itself; as it is for caps so small that 1 / cap2^2,
// from which the polynomial's way has 1 - tanh^2, would leave it.
__host__ __device__ inline ScoreFactors score_factors(float k, float cap2) {
  ScoreFactors f;
  f.k = k;
  f.cap2 = cap2;
  const float k2 = k * k;
  f.a[0] = kTanhC0 * cap2 * k;
  f.a[1] = kTanhC1 * cap2 * k * k2;
  f.a[2] = kTanhC2 * cap2 * k * k2 * k2;
  f.a[3] = kTanhC3 * cap2 * k * k2 * k2 * k2;
  const float last = f.a[3] < 0.0f ? -f.a[3] : f.a[3];
  const bool holds =
      k == 1.0f || (k2 > 1e-18f && k2 < 1e12f && last > 1e-30f && last < 1e30f);
  f.range = cap2 > 1e-15f && holds ? kTanhRange / k : -1.0f;
  f.neg_inv_cap_sq = cap2 > 0.0f ? -1.0f / (cap2 * cap2) : 0.0f;
  return f;
}

// What the kernels get of fa_score_spec, fa_key_spans and the call's sizes.
struct ScoreParams {
  float scale;    // of Q K^T
  ScoreFactors f;
  const float* slopes;  // [Hq], nullptr: none
  const int* first;
  const int* end;
  long long span_batch;
  int window, causal, q_offset;
  int Nq, Nk, Hq, Hkv, G;
  int B;
  uint32_t* err;
};

// Kinds of kernels: what is done to a score.
enum ScoreMode { kScorePlain = 0, kScoreBias = 1, kScoreCap = 2, kScoreCapBias = 3 };

struct ScoreMaps {
  CUtensorMap q, dO;  // boxes of 64 columns x 128 rows
  CUtensorMap k, v;   // boxes of 64 columns x 128 rows (64 rows at d = 256)
};

// As encode_map_bf16 (fa_internal.h), with boxes of one key tile's rows (fa_api.cu).
bool encode_map_kv_bf16(CUtensorMap* m, const void* ptr, int d, int N, long long planes);

// Fills in what `spec` (may be NULL) and `scale` say; refuses what it cannot hold.
fa_status put_scores(ScoreParams* p, const fa_score_spec* spec, float scale);
int score_mode(const ScoreParams& p);

// Each by head dimension D (64, 96, 128, 256); instantiated one D a translation unit.
template <int D>
cudaError_t launch_scores_forward(const ScoreMaps& m, void* o, float* lse, const ScoreParams& p,
                                  int mode, cudaStream_t stream);
template <int D>
cudaError_t launch_scores_dkdv(const ScoreMaps& m, const float* lse, const float* Dv,
                               const int2* tiles, void* dk, void* dv, float* part, int split,
                               const ScoreParams& p, int mode, cudaStream_t stream);
template <>
cudaError_t launch_scores_dkdv<256>(const ScoreMaps& m, const float* lse, const float* Dv,
                                    const int2* tiles, void* dk, void* dv, float* part, int split,
                                    const ScoreParams& p, int mode, cudaStream_t stream);
template <int D>
cudaError_t launch_scores_dq(const ScoreMaps& m, const float* lse, float* Dv, void* dq,
                             const ScoreParams& p, int mode, cudaStream_t stream);

}  // namespace fa
