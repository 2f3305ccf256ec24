// Chunks over the paged cache with a bias by distance.
#include "ra_cache_chunk.cuh"

namespace ra {

template <>
cudaError_t launch_cache_chunk_score<SC_ON | SC_BIAS>(const CacheAttnPlan& p, cudaStream_t st) {
  return p.args.d == 64 ? launch_chunk<64, SC_ON | SC_BIAS>(p, st) : launch_chunk<128, SC_ON | SC_BIAS>(p, st);
}

}  // namespace ra
