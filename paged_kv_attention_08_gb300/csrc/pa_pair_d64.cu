// Instantiations of the two-tile kernel for head_dim 64.
#include "pa_pair.cuh"

namespace pa {
cudaError_t launch_pair_d64(const AttnLaunch& L, cudaStream_t stream) {
    return launch_pair_for_d<64>(L, stream);
}
}  // namespace pa
