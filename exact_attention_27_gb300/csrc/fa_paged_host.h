// Host side of the paged-cache entry points, between their translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

struct PagedParams;

// Bit of the device error word that is no timeout: a paged call met a length
// past its block table's row or a page outside its cache.
constexpr uint32_t kErrBadPage = 1u << 5;

// Checks a paged cache, a step's batch and its number of tokens (fa_rotary.cu);
// T = 0 or S = 0 needs no pointers.
fa_status validate_cache(const fa_paged_cache* c, const fa_paged_batch* b, int T);

// Multiprocessors of the current device, 0 if CUDA gives none (fa_paged.cu).
int sm_count();

// The pages (k or v) of a paged cache as bytes (d, row, head, page), boxes of
// 128 bytes x box_rows rows, 128-byte swizzle (fa_api.cu).
bool encode_map_pages(CUtensorMap* m, const fa_paged_cache& c, const void* pages, int box_rows);

// Rows of an item and keys of a tile of the tcgen05 kernels: 256 x 128 at d =
// 64, 96 and 128 (fa_paged_tile2.cu), 128 x 64 at d = 256 (fa_paged_tile.cu).
constexpr int paged_tile_rows(int d) { return d == 256 ? 128 : 256; }
constexpr int paged_tile_keys(int d) { return d == 256 ? 64 : 128; }

// Enqueue those kernels on `ctas` CTAs; K and V maps have boxes of min(page
// size, keys of a tile) rows.
cudaError_t launch_paged_tile(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                              bool e4m3, int ctas, cudaStream_t stream);
cudaError_t launch_paged_tile2(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                               int d, bool e4m3, int ctas, cudaStream_t stream);
// The same kernels for shaped scores (fa_paged_scores.cu).
cudaError_t launch_paged_rows_shaped(const CUtensorMap& tk, const CUtensorMap& tv,
                                     const PagedParams& p, int d, bool e4m3, int ctas,
                                     cudaStream_t stream);
cudaError_t launch_paged_tile_shaped(const CUtensorMap& tk, const CUtensorMap& tv,
                                     const PagedParams& p, bool e4m3, int ctas,
                                     cudaStream_t stream);
cudaError_t launch_paged_tile2_shaped(const CUtensorMap& tk, const CUtensorMap& tv,
                                      const PagedParams& p, int d, bool e4m3, int ctas,
                                      cudaStream_t stream);

}  // namespace fa
