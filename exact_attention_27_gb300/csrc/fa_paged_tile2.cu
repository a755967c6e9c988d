// Instances of fa_paged_tile2.cuh for the unshaped call.
#include "fa_paged_tile2.cuh"

namespace fa {
namespace {

template <bool E4M3>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int d,
                     int ctas, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_tile2_t<64, E4M3, false>(tk, tv, p, ctas, stream);
    case 96: return launch_tile2_t<96, E4M3, false>(tk, tv, p, ctas, stream);
    case 128: return launch_tile2_t<128, E4M3, false>(tk, tv, p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_tile2(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                               int d, bool e4m3, int ctas, cudaStream_t stream) {
  return e4m3 ? launch_d<true>(tk, tv, p, d, ctas, stream)
              : launch_d<false>(tk, tv, p, d, ctas, stream);
}

}  // namespace fa
