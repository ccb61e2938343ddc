// Instantiations of the decode kernel for head_dim 256 with row statistics,
// scores, a shared prefix or a limit of the tokens.
#include "pa_attn.cuh"

namespace pa {
cudaError_t launch_attn_d256_extended(const AttnLaunch& L, cudaStream_t stream) {
    return L.p.q_len > 1 ? launch_attn_for_d<256, true, true>(L, stream)
                         : launch_attn_for_d<256, false, true>(L, stream);
}
}  // namespace pa
