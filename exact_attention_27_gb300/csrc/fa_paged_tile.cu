// Instances of fa_paged_tile1.cuh for the unshaped call.
#include "fa_paged_tile1.cuh"

namespace fa {

cudaError_t launch_paged_tile(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                              bool e4m3, int ctas, cudaStream_t stream) {
  return e4m3 ? launch_tile1_t<256, true, false>(tk, tv, p, ctas, stream)
              : launch_tile1_t<256, false, false>(tk, tv, p, ctas, stream);
}

}  // namespace fa
