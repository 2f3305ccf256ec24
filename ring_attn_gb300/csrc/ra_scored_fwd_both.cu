// The ring forward with capped scores and a bias by distance.
#include "ra_scored_fwd.cuh"

template cudaError_t ra::launch_fwd_score<ra::SC_ON | ra::SC_CAP | ra::SC_BIAS>(
    int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const ra::FwdParams&, const ra::ScoreParams&,
    cudaStream_t);
