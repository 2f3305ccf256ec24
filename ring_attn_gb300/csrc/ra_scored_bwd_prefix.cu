// The ring backward with a prefix that all tokens see, scores as they are.
#include "ra_scored_bwd.cuh"

template cudaError_t ra::launch_bwd_score<ra::SC_ON>(
    int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const ra::BwdParams&,
    const ra::ScoreParams&, int, cudaStream_t);
