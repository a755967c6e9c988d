// Launches of fa_forward_paged's kernels, between its translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

struct PagedParams;

// Rows of an item and keys of a tile of the tile kernel (fa_paged_tile.cu).
constexpr int kPagedTileRows = 128;
constexpr int paged_tile_keys(int d) { return d == 256 ? 64 : 128; }

// Enqueues the tile kernel on `ctas` CTAs; K and V maps have boxes of
// min(page size, keys of a tile) rows.
cudaError_t launch_paged_tile(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                              int d, bool e4m3, int ctas, cudaStream_t stream);

}  // namespace fa
