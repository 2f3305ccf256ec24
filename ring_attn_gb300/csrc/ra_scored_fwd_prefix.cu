// The ring forward with a prefix that all tokens see, scores as they are.
#include "ra_scored_fwd.cuh"

template cudaError_t ra::launch_fwd_score<ra::SC_ON>(
    int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const ra::FwdParams&, const ra::ScoreParams&,
    cudaStream_t);
