// The ring forward with plain scores (the kernel: ra_fwd.cuh).
#include "ra_fwd.cuh"

namespace ra {
namespace {

template <int D, bool VL>
cudaError_t launch_plain(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdParams& p,
                         cudaStream_t st) {
  FwdParamsT<VL> pv;
  static_cast<FwdParams&>(pv) = p;
  return launch_fwd_v<D, VL, 0>(tq, tk, tv, pv, st);
}

}  // namespace

size_t fwd_smem_bytes(int D) { return D == 64 ? FwdLayout<64>::kAlloc : FwdLayout<128>::kAlloc; }

cudaError_t launch_fwd(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const FwdParams& p, cudaStream_t st) {
  if (D == 64) return p.cu ? launch_plain<64, true>(tq, tk, tv, p, st) : launch_plain<64, false>(tq, tk, tv, p, st);
  return p.cu ? launch_plain<128, true>(tq, tk, tv, p, st) : launch_plain<128, false>(tq, tk, tv, p, st);
}

}  // namespace ra
