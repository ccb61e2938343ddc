// Instantiations of the two-tile kernel for head_dim 128.
#include "pa_pair.cuh"

namespace pa {
cudaError_t launch_pair_d128(const AttnLaunch& L, cudaStream_t stream) {
    return launch_pair_for_d<128>(L, stream);
}
}  // namespace pa
