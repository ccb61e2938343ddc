// Instantiations of the attention over the latent cache for latent_dim 128.
#include "pa_latent.cuh"

namespace pa {
cudaError_t launch_latent_r128(const LatentLaunch& L, cudaStream_t stream) {
    return launch_latent_for_r<128>(L, stream);
}
}  // namespace pa
