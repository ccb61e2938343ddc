// Instantiations of the attention over the latent cache for latent_dim 256.
#include "pa_latent.cuh"

namespace pa {
cudaError_t launch_latent_r256(const LatentLaunch& L, cudaStream_t stream) {
    return launch_latent_for_r<256>(L, stream);
}
}  // namespace pa
