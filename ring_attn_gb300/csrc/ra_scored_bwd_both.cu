// The ring backward with capped scores and a bias by distance.
#include "ra_scored_bwd.cuh"

template cudaError_t ra::launch_bwd_score<ra::SC_ON | ra::SC_CAP | ra::SC_BIAS>(
    int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const ra::BwdParams&,
    const ra::ScoreParams&, int, cudaStream_t);
