// Attention of few new tokens over the paged cache with changed scores.
#include "ra_cache_attn.cuh"

namespace ra {

cudaError_t launch_cache_attn_scored(const CacheAttnPlan& p, cudaStream_t st) { return launch_few<true>(p, st); }

}  // namespace ra
