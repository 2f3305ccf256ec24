// The ring backward with capped scores.
#include "ra_scored_bwd.cuh"

template cudaError_t ra::launch_bwd_score<ra::SC_ON | ra::SC_CAP>(
    int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const ra::BwdParams&,
    const ra::ScoreParams&, int, cudaStream_t);
