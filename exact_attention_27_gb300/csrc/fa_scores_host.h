// Host side of the shaped-score entry points, between their translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

// What the kernels get of fa_score_spec, fa_key_spans and the call's sizes.
struct ScoreParams {
  float scale;    // of Q K^T
  float scale2;   // scale log2(e)
  float y_scale;  // scale / softcap
  float cap2;     // softcap log2(e); 0: none
  // The factor of q.k that the kernels take.
  __host__ __device__ float factor(bool cap) const { return cap ? y_scale : scale2; }
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

// Fills in what `spec` (may be NULL) and `scale` say; refuses what it cannot hold.
fa_status put_scores(ScoreParams* p, const fa_score_spec* spec, float scale);
int score_mode(const ScoreParams& p);

// Each by head dimension D (64, 96, 128, 256); instantiated one D a translation unit.
template <int D>
cudaError_t launch_scores_forward(const ScoreMaps& m, void* o, float* lse, const ScoreParams& p,
                                  int mode, cudaStream_t stream);
template <int D>
cudaError_t launch_scores_dkdv(const ScoreMaps& m, const float* lse, const float* Dv,
                               const int2* tiles, void* dk, void* dv, const ScoreParams& p,
                               int mode, cudaStream_t stream);
template <>
cudaError_t launch_scores_dkdv<256>(const ScoreMaps& m, const float* lse, const float* Dv,
                                    const int2* tiles, void* dk, void* dv, const ScoreParams& p,
                                    int mode, cudaStream_t stream);
template <int D>
cudaError_t launch_scores_dq(const ScoreMaps& m, const float* lse, float* Dv, void* dq,
                             const ScoreParams& p, int mode, cudaStream_t stream);

}  // namespace fa
