// Instances of the attention over 8-bit caches with plain scores.
#include "ripe_score_kernel.cuh"

namespace ripe {

cudaError_t launch_score_q8(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
    switch (d) {
        case 64: return ScoreSet<64, true, 0>::launch(t, grid, a, s);
        case 96: return ScoreSet<96, true, 0>::launch(t, grid, a, s);
        case 128: return ScoreSet<128, true, 0>::launch(t, grid, a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t set_score_q8_attributes() {
    cudaError_t e = ScoreSet<64, true, 0>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<96, true, 0>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<128, true, 0>::set_attr();
    return e;
}

}  // namespace ripe
