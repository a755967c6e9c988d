// Launches of the forward with shaped scores: the kernel by its mode, one query tile a CTA or two.
#pragma once

#include "fa_internal.h"
#include "fa_paged_host.h"
#include "fa_scores_fwd.cuh"
#include "fa_scores_fwd2.cuh"

namespace fa {
namespace {

// Caps up to here (log2 domain; 55 in scores) have a fixed reference, 0: weights from 2^-80 to
// 2^80.
constexpr float kFixedCap = 80.0f;

// One query tile a CTA or two: as the unshaped forward chooses (forward_rows_for: it estimates
// when either grid ends, at that kernel's costs).  16 heads of 8192, causal, one / two: d = 64 187 /
// 152 us, with slopes 241 / 207; d = 96 197 / 170, 259 / 219; d = 128 200 / 225, 276 / 287.  Only
// that grid was timed.  At d = 128, where one tile is the faster there, and is chosen, larger grids
// still get two; and neither windows nor the masks that spans bring are known here.
bool two_tiles(const ScoreParams& s, int d) {
  const int sms = sm_count();
  AttnShape a{s.B, s.Hq, s.Hkv, s.Nq, d, s.scale, s.causal};
  a.Nk = s.Nk;
  a.q_offset = s.q_offset;
  return sms > 0 && forward_rows_for(a, sms) == 256;
}

template <int D, bool CAP, bool BIAS, bool FIXED>
cudaError_t launch_scores_fwd_t(const ScoreMaps& m, void* o, float* lse, const ScoreParams& s,
                                cudaStream_t stream) {
  ScoreFwdParams p;
  p.s = s;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.n_qtiles = (s.Nq + 127) / 128;
  p.n_heads = s.B * s.Hq;
  p.heads_per_group = static_cast<int>(heads_per_group(s.Nk, D, 2.0, s.G, p.n_heads));
  if constexpr (D <= 128 && !FIXED) {
    if (two_tiles(s, D)) {
      using C = ScoreFwd2Cfg<D>;
      const cudaError_t e =
          set_smem_limit_once<fa_scores_fwd2_kernel<D, CAP, BIAS>>(C::SMEM_BYTES);
      if (e != cudaSuccess) return e;
      const long long grid = static_cast<long long>(p.n_heads) * ((p.n_qtiles + 1) / 2);
      if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
      return launch_dependent(fa_scores_fwd2_kernel<D, CAP, BIAS>,
                              dim3(static_cast<unsigned>(grid)), dim3(C::THREADS), C::SMEM_BYTES,
                              stream, m.q, m.k, m.v, p);
    }
  }
  using C = ScoreFwdCfg<D, FIXED>;
  const cudaError_t e =
      set_smem_limit_once<fa_scores_fwd_kernel<D, CAP, BIAS, FIXED>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.n_heads) * p.n_qtiles;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(fa_scores_fwd_kernel<D, CAP, BIAS, FIXED>,
                          dim3(static_cast<unsigned>(grid)), dim3(C::THREADS), C::SMEM_BYTES,
                          stream, m.q, m.k, m.v, p);
}

}  // namespace

template <int D>
cudaError_t launch_scores_forward(const ScoreMaps& m, void* o, float* lse, const ScoreParams& p,
                                  int mode, cudaStream_t stream) {
  switch (mode) {
    case kScorePlain: return launch_scores_fwd_t<D, false, false, false>(m, o, lse, p, stream);
    case kScoreBias: return launch_scores_fwd_t<D, false, true, false>(m, o, lse, p, stream);
    case kScoreCap:
      if (p.f.cap2 <= kFixedCap)
        return launch_scores_fwd_t<D, true, false, true>(m, o, lse, p, stream);
      [[fallthrough]];  // (no slopes: a slope of 0)
    default: return launch_scores_fwd_t<D, true, true, false>(m, o, lse, p, stream);
  }
}

}  // namespace fa
