// The kernels of attention with shaped scores at head dimension 256.
#include "fa_scores_dq.cuh"
#include "fa_scores_kv256.cuh"
#include "fa_scores_launch.cuh"

namespace fa {

template cudaError_t launch_scores_forward<256>(const ScoreMaps&, void*, float*, const ScoreParams&,
                                               int, cudaStream_t);
template cudaError_t launch_scores_dq<256>(const ScoreMaps&, const float*, float*, void*,
                                          const ScoreParams&, int, cudaStream_t);

}  // namespace fa
