// Instantiations of the decode kernel for head_dim 64 with row statistics,
// scores, a shared prefix or a limit of the tokens.
#include "pa_attn.cuh"

namespace pa {
cudaError_t launch_attn_d64_extended(const AttnLaunch& L, cudaStream_t stream) {
    return L.p.q_len > 1 ? launch_attn_for_d<64, true, true>(L, stream)
                         : launch_attn_for_d<64, false, true>(L, stream);
}
}  // namespace pa
