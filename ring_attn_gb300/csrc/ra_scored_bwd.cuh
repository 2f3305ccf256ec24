// Launcher of the ring backward with changed scores.  Each ra_scored_bwd_*.cu makes it for one
// kind of change, so that they compile side by side.
#pragma once

#include "ra_bwd.cuh"

namespace ra {
namespace {

template <int SC, int D, bool VL>
cudaError_t launch_bwd_sdv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                           const BwdParams& p, const ScoreParams& sc, int which, const LseView& lse, cudaStream_t st) {
  BwdParamsT<VL, SC> pv;
  static_cast<BwdParams&>(pv) = p;
  pv.sc = sc;
  if (which == 2)
    return launch_rowdot_v<D, VL, SC>(tq, tk, tv, tdo, pv, lse, const_cast<float*>(p.nD), const_cast<float*>(p.nlse2), st);
  return launch_bwd_v<D, VL, SC>(tq, tk, tv, tdo, pv, which, st);
}

}  // namespace

template <int SC>
cudaError_t launch_bwd_score(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo, const BwdParams& p, const ScoreParams& sc, int which,
                             const LseView& lse, cudaStream_t st) {
  if (D == 64)
    return p.cu ? launch_bwd_sdv<SC, 64, true>(tq, tk, tv, tdo, p, sc, which, lse, st)
                : launch_bwd_sdv<SC, 64, false>(tq, tk, tv, tdo, p, sc, which, lse, st);
  return p.cu ? launch_bwd_sdv<SC, 128, true>(tq, tk, tv, tdo, p, sc, which, lse, st)
              : launch_bwd_sdv<SC, 128, false>(tq, tk, tv, tdo, p, sc, which, lse, st);
}

}  // namespace ra
