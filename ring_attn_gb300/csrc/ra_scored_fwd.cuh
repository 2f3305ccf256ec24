// Launcher of the ring forward with changed scores.  Each ra_scored_fwd_*.cu makes it for one
// kind of change, so that they compile side by side.
#pragma once

#include "ra_fwd.cuh"

namespace ra {
namespace {

template <int SC, int D, bool VL>
cudaError_t launch_fwd_sdv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdParams& p,
                           const ScoreParams& sc, cudaStream_t st) {
  FwdParamsT<VL, SC> pv;
  static_cast<FwdParams&>(pv) = p;
  pv.sc = sc;
  return launch_fwd_v<D, VL, SC>(tq, tk, tv, pv, st);
}

}  // namespace

template <int SC>
cudaError_t launch_fwd_score(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const FwdParams& p, const ScoreParams& sc, cudaStream_t st) {
  if (D == 64)
    return p.cu ? launch_fwd_sdv<SC, 64, true>(tq, tk, tv, p, sc, st)
                : launch_fwd_sdv<SC, 64, false>(tq, tk, tv, p, sc, st);
  return p.cu ? launch_fwd_sdv<SC, 128, true>(tq, tk, tv, p, sc, st)
              : launch_fwd_sdv<SC, 128, false>(tq, tk, tv, p, sc, st);
}

}  // namespace ra
