// Instances of the attention over 8-bit caches, with plain and with capped or biased scores.
#include "ripe_score_kernel.cuh"

namespace ripe {
namespace {

template <bool MOD>
cudaError_t launch_d(int d, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
    switch (d) {
        case 64: return ScoreSet<64, true, MOD>::launch(t, grid, a, s);
        case 96: return ScoreSet<96, true, MOD>::launch(t, grid, a, s);
        case 128: return ScoreSet<128, true, MOD>::launch(t, grid, a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_score_q8(int d, bool mod, const LaunchTarget &t, int grid, const ScoreArgs &a, cudaStream_t s) {
    return mod ? launch_d<true>(d, t, grid, a, s) : launch_d<false>(d, t, grid, a, s);
}

cudaError_t set_score_q8_attributes() {
    cudaError_t e = ScoreSet<64, true, false>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<96, true, false>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<128, true, false>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<64, true, true>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<96, true, true>::set_attr();
    if (e == cudaSuccess) e = ScoreSet<128, true, true>::set_attr();
    return e;
}

}  // namespace ripe
