// The entry of fa_forward_paged and its shaped form: checks, the choice of kernels (few rows a
// sequence: fa_paged_rows.cuh; more: fa_paged_tile2.cuh, and fa_paged_tile1.cuh at d = 256),
// and the joining of what the CTAs share.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_paged_host.h"
#include "fa_paged_rows.cuh"
#include "fa_ptx.cuh"
#include "fa_scores_host.h"

namespace fa {
namespace {

// Joins the parts of the items that several CTAs share: blocks (c, y) those of
// the item that starts in CTA c and is not finished there.  A group of D / 4
// threads runs over parts with a running maximum, four loads in flight.  Few
// parts, or rows for more groups than the item's blocks have: each group has a row
// of its own.  Many parts and few rows (a long history): the block's groups share a
// row's parts and join through shared memory.  Either way the order is that of the
// CTAs.  (512 rows of 30,000 keys, d = 64: 27.2 us, 46.4 us when items of all
// heights of many parts share rows.)  The blocks an item are fixed, however few items
// there are: one item of 256 rows in 152 parts (64 tokens of 4 heads over 100,000 keys
// of one head, d = 128) keeps 16 blocks busy while the others idle, 63 us in all for
// 7.6 us of bytes.
constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 12;
constexpr int kJoinRowsBlocks = 4, kJoinTileBlocks = 16;

template <int D, bool TILE>
__global__ void __launch_bounds__(kJoinThreads)
    fa_paged_join_kernel(const PagedParams p, int tile_rows) {
  constexpr int LANES = D / 4;
  constexpr int GROUPS = kJoinThreads / LANES;
  __shared__ float4 acc[GROUPS][LANES];
  __shared__ float2 state[GROUPS];
  grid_launch_dependents();
  grid_dependency_wait();
  const int cta = blockIdx.x;
  const PagedNote note = p.notes[cta];
  if (note.last < 0) return;
  const int rows = min(tile_rows, note.rows - note.tile0);
  const int grp = threadIdx.x / LANES, lane = threadIdx.x - grp * LANES;
  const int parts = note.last - cta + 1;
  float m = -INFINITY, l = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float2& ml, const float4& x) {
    const float m_new = fmaxf(m, ml.x);
    const float ref = m_new == -INFINITY ? 0.0f : m_new;
    const float f = ex2_approx(m - ref), e = ex2_approx(ml.x - ref);
    a.x = a.x * f + x.x * e;
    a.y = a.y * f + x.y * e;
    a.z = a.z * f + x.z * e;
    a.w = a.w * f + x.w * e;
    l = l * f + ml.y * e;
    m = m_new;
  };
  auto run = [&](int row, int k0, int step) {
    m = -INFINITY;
    l = 0.0f;
    a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int N = 4;
    for (int k = k0; k < parts; k += N * step) {
      float2 ml[N];
      float4 x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int part = k + i * step;
        if (part < parts) {
          const long long at =
              (static_cast<long long>(cta + part) * 2 + (part == 0)) * tile_rows + row;
          ml[i] = p.part_ml[at];
          x[i] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (k + i * step < parts) add(ml[i], x[i]);
    }
  };
  auto store = [&](int row) {
    const int r = note.tile0 + row;
    const int tok = r / p.G;
    const long long token = note.q0 + tok;
    const int head = note.head * p.G + (r - tok * p.G);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    *reinterpret_cast<uint2*>(p.o + token * p.o_token + head * p.o_head + 4 * lane) =
        make_uint2(pack_bf16x2(a.x * inv * p.v_scale, a.y * inv * p.v_scale),
                   pack_bf16x2(a.z * inv * p.v_scale, a.w * inv * p.v_scale));
    if (lane == 0 && p.lse)
      p.lse[token * p.Hq + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kPagedLn2;
  };
  if (parts <= kJoinFew || (TILE && rows > 2 * kJoinTileBlocks)) {
    if (grp < GROUPS)
      for (int row = blockIdx.y * GROUPS + grp; row < rows; row += gridDim.y * GROUPS) {
        run(row, 0, 1);
        store(row);
      }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    if (grp < GROUPS) {
      run(row, grp, GROUPS);
      acc[grp][lane] = a;
      if (lane == 0) state[grp] = make_float2(m, l);
    }
    __syncthreads();
    if (grp == 0) {
      for (int k = 1; k < GROUPS; ++k) add(state[k], acc[k][lane]);
      store(row);
    }
    __syncthreads();
  }
}

// Rows of an item, which says the kernel: sequences of at most 16 rows go to the
// kernel above, anything longer to the tcgen05 kernels (64 sequences of 100 to
// 8000 keys, 32 rows each, d = 128: 213 us there, 269 us 32 rows a time here;
// 348 us as two items of 16).  The longest sequence decides for the whole step, so
// the single tokens of a mixed step fill 128-row tiles: 3 chunks among 21 tokens,
// 16 / 4 heads, d = 64, take 40.9 us, the chunks on their own 29.9, and single
// tokens of all 24 sequences in the kernel above 22.1.
int rows_for(long long most, int d) { return most <= 16 ? 16 : paged_tile_rows(d); }

// CTAs of a launch with `rows` rows an item.
int ctas_for(int sms, int rows, int d, bool e4m3) {
  return sms * (rows == 16 ? rows_occupancy(d, e4m3) : 1);
}

// Workspace: notes, (m, l), O; each part on a 256-byte boundary (parts of O are
// stored 32 bytes at a time), the first that the caller's 16-byte aligned memory has.
struct PartLayout {
  size_t ml, o, total;
};
PartLayout part_layout(int ctas, int rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  PartLayout l;
  l.ml = up(static_cast<size_t>(ctas) * sizeof(PagedNote));
  l.o = l.ml + up(static_cast<size_t>(ctas) * 2 * rows * sizeof(float2));
  l.total = l.o + static_cast<size_t>(ctas) * 2 * rows * d * sizeof(float) + 240;
  return l;
}

template <bool TILE>
cudaError_t launch_join(const PagedParams& p, int rows, int d, int ctas, cudaStream_t stream) {
  auto kern = d == 64    ? fa_paged_join_kernel<64, TILE>
              : d == 96  ? fa_paged_join_kernel<96, TILE>
              : d == 128 ? fa_paged_join_kernel<128, TILE>
                         : fa_paged_join_kernel<256, TILE>;
  return launch_dependent(kern, dim3(ctas, TILE ? kJoinTileBlocks : kJoinRowsBlocks),
                          dim3(kJoinThreads), 0, stream, p, rows);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];  // by device; 0: not asked yet
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool slot = dev >= 0 && dev < 64;
  if (slot && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (slot) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

fa_status forward_paged(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* q,
                        long long q_token, long long q_head, void* o, long long o_token,
                        long long o_head, float* lse, int T, int H_q, float scale, int causal,
                        const fa_score_spec* spec, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  const fa_status st = validate_cache(cache, batch, T);
  if (st != FA_OK) return st;
  const int d = cache->d, H = cache->H_kv;
  if (H_q < 1 || H_q % H != 0) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARGUMENT;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARGUMENT;
  const float s_eff = scale * cache->k_descale;
  if (!std::isfinite(s_eff * kPagedLog2e) || !(s_eff > 0.0f)) return FA_ERR_INVALID_ARGUMENT;
  ScoreParams shape;
  if (put_scores(&shape, spec, s_eff) != FA_OK) return FA_ERR_INVALID_ARGUMENT;
  const bool shaped = shape.f.cap2 > 0.0f || shape.slopes || shape.window > 0;
  if (static_cast<long long>(T) * H_q >= 0x7fffff00LL) return FA_ERR_INVALID_ARGUMENT;
  if (T == 0 || batch->S == 0) return FA_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FA_ERR_INVALID_ARGUMENT;
  for (long long s : {q_token, q_head, o_token, o_head})
    if (s < 0 || s % 8 != 0) return FA_ERR_INVALID_ARGUMENT;
  if ((o_token == 0 && T > 1) || (o_head == 0 && H_q > 1)) return FA_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms < 1) return FA_ERR_CUDA;
  const int G = H_q / H;
  const long long most = static_cast<long long>(std::min(T, batch->max_q_len)) * G;
  const int rows = rows_for(most, d);
  const int ctas = ctas_for(sms, rows, d, cache->dtype == FA_CACHE_E4M3);
  const PartLayout lay = part_layout(ctas, rows, d);
  if (!workspace || !aligned16(workspace) || workspace_bytes < lay.total)
    return FA_ERR_INVALID_ARGUMENT;
  PagedParams p{};
  p.err = device_error_word();
  if (!p.err) return FA_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_token = q_token;
  p.q_head = q_head;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o_token = o_token;
  p.o_head = o_head;
  p.lse = lse;
  p.table = batch->block_table;
  p.table_stride = batch->table_stride;
  p.q_start = batch->q_start;
  p.kv_len = batch->kv_len;
  p.S = batch->S;
  p.T = T;
  p.Hq = H_q;
  p.Hkv = H;
  p.G = G;
  p.page_shift = 31 - __builtin_clz(cache->page_size);
  p.max_pages = batch->max_pages;
  p.n_pages = cache->n_pages;
  p.causal = causal;
  // A CTA starts for one tile of 64 keys (two sequences of a thousand keys: 10.8 us,
  // 13 to 19 us with 2 to 8 at least), but for more of the tcgen05 kernels, whose
  // parts are larger: two tiles at d = 256 (128 tokens of 32 heads without a
  // history: 13.0 us, 15.0 with three, 17.3 with four), and otherwise six units, two
  // or three tiles (128 rows of 4096 keys, d = 128: 15.0 us, 15.7 us with eight).
  // Ranges then hold at least three units there, so each CTA between an item's first
  // and last has a tile of it.
  p.min_units = rows == 16 ? 1 : d == 256 ? 2 : 6;
  p.scale_log2 = s_eff * kPagedLog2e;
  p.v_scale = cache->v_descale;
  p.cap2 = shape.f.cap2;
  p.f = cache->dtype == FA_CACHE_E4M3 ? score_factors(1.0f, shape.f.cap2) : shape.f;
  p.slopes = shape.slopes;
  p.window = shape.window;
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) &
                                     ~static_cast<uintptr_t>(255));
  p.notes = reinterpret_cast<PagedNote*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
  p.part_o = reinterpret_cast<float*>(ws + lay.o);
  CUtensorMap tk, tv;
  const bool tile = rows > 16;
  const bool e4m3 = cache->dtype == FA_CACHE_E4M3;
  const int box = std::min(cache->page_size, tile ? paged_tile_keys(d) : kTK);
  if (!encode_map_pages(&tk, *cache, cache->k, box) || !encode_map_pages(&tv, *cache, cache->v, box))
    return FA_ERR_CUDA;
  cudaError_t e;
  if (shaped)
    e = !tile      ? launch_paged_rows_shaped(tk, tv, p, d, e4m3, ctas, stream)
        : d == 256 ? launch_paged_tile_shaped(tk, tv, p, e4m3, ctas, stream)
                   : launch_paged_tile2_shaped(tk, tv, p, d, e4m3, ctas, stream);
  else
    e = tile   ? d == 256 ? launch_paged_tile(tk, tv, p, e4m3, ctas, stream)
                          : launch_paged_tile2(tk, tv, p, d, e4m3, ctas, stream)
        : e4m3 ? launch_rows<true, false>(tk, tv, p, d, ctas, stream)
               : launch_rows<false, false>(tk, tv, p, d, ctas, stream);
  if (e == cudaSuccess)
    e = tile ? launch_join<true>(p, rows, d, ctas, stream)
             : launch_join<false>(p, rows, d, ctas, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_forward_paged_workspace_bytes(int H_q, int H_kv, int d, int T, int max_q_len) {
  using namespace fa;
  if (H_q < 1 || H_kv < 1 || H_q % H_kv != 0 || T < 0 || max_q_len < 0) return 0;
  if (d != 64 && d != 96 && d != 128 && d != 256) return 0;
  const long long most = static_cast<long long>(std::min(T, max_q_len)) * (H_q / H_kv);
  const int rows = rows_for(most, d);
  return part_layout(ctas_for(sm_count(), rows, d, true), rows, d).total;  // (the most)
}

fa_status fa_forward_paged(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* q,
                           long long q_token, long long q_head, void* o, long long o_token,
                           long long o_head, float* lse, int T, int H_q, float scale, int causal,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return fa::forward_paged(cache, batch, q, q_token, q_head, o, o_token, o_head, lse, T, H_q, scale,
                           causal, nullptr, workspace, workspace_bytes, stream);
}

fa_status fa_forward_paged_scores(const fa_paged_cache* cache, const fa_paged_batch* batch,
                                  const void* q, long long q_token, long long q_head, void* o,
                                  long long o_token, long long o_head, float* lse, int T, int H_q,
                                  float scale, int causal, const fa_score_spec* spec,
                                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return fa::forward_paged(cache, batch, q, q_token, q_head, o, o_token, o_head, lse, T, H_q, scale,
                           causal, spec, workspace, workspace_bytes, stream);
}

}  // extern "C"
