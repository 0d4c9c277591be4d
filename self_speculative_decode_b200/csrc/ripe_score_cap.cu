// Instances of the attention over bf16 caches with a cap from kCapSeries on.
#include "ripe_score_kernel.cuh"

namespace ripe {

cudaError_t launch_score_cap(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
    switch (d) {
        case 64: return ScoreSet<64, false, 2>::launch(t, grid, a, s);
        case 96: return ScoreSet<96, false, 2>::launch(t, grid, a, s);
        case 128: return ScoreSet<128, false, 2>::launch(t, grid, a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t set_score_cap_attributes() {
    cudaError_t e = ScoreSet<64, false, 2>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<96, false, 2>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<128, false, 2>::set_attr();
    return e;
}

}  // namespace ripe
