// The ring backward with plain scores (the kernels: ra_bwd.cuh).
#include "ra_bwd.cuh"

namespace ra {
namespace {

template <int D, bool VL>
cudaError_t launch_plain(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                         const BwdParams& p, int which, cudaStream_t st) {
  BwdParamsT<VL> pv;
  static_cast<BwdParams&>(pv) = p;
  return which == 0 ? launch_dkdv_v<D, VL, 0>(tq, tk, tv, tdo, pv, st) : launch_dq_v<D, VL>(tq, tk, tv, tdo, pv, st);
}

}  // namespace

cudaError_t launch_bwd(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const BwdParams& p, int which, cudaStream_t st) {
  if (D == 64)
    return p.cu ? launch_plain<64, true>(tq, tk, tv, tdo, p, which, st)
                : launch_plain<64, false>(tq, tk, tv, tdo, p, which, st);
  return p.cu ? launch_plain<128, true>(tq, tk, tv, tdo, p, which, st)
              : launch_plain<128, false>(tq, tk, tv, tdo, p, which, st);
}

}  // namespace ra
