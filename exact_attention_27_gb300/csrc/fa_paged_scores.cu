// Instances of the kernels of paged attention for shaped scores: few rows a sequence, and d = 256.
#include "fa_paged_rows.cuh"
#include "fa_paged_tile1.cuh"

namespace fa {

cudaError_t launch_paged_rows_shaped(const CUtensorMap& tk, const CUtensorMap& tv,
                                     const PagedParams& p, int d, bool e4m3, int ctas,
                                     cudaStream_t stream) {
  return e4m3 ? launch_rows<true, true>(tk, tv, p, d, ctas, stream)
              : launch_rows<false, true>(tk, tv, p, d, ctas, stream);
}

cudaError_t launch_paged_tile_shaped(const CUtensorMap& tk, const CUtensorMap& tv,
                                     const PagedParams& p, bool e4m3, int ctas,
                                     cudaStream_t stream) {
  return e4m3 ? launch_tile1_t<256, true, true>(tk, tv, p, ctas, stream)
              : launch_tile1_t<256, false, true>(tk, tv, p, ctas, stream);
}

}  // namespace fa
