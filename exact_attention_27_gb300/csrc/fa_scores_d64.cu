// The kernels of attention with shaped scores at head dimension 64.
#include "fa_scores_dkdv.cuh"
#include "fa_scores_dq.cuh"
#include "fa_scores_launch.cuh"

namespace fa {

template cudaError_t launch_scores_forward<64>(const ScoreMaps&, void*, float*, const ScoreParams&,
                                               int, cudaStream_t);
template cudaError_t launch_scores_dq<64>(const ScoreMaps&, const float*, float*, void*,
                                          const ScoreParams&, int, cudaStream_t);
template cudaError_t launch_scores_dkdv<64>(const ScoreMaps&, const float*, const float*,
                                            const int2*, void*, void*, float*, int,
                                            const ScoreParams&, int, cudaStream_t);

}  // namespace fa
