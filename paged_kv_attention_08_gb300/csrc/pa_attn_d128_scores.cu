// Instantiations of the decode kernel that store the scores, for head_dim 128.
#include "pa_attn.cuh"

namespace pa {
cudaError_t launch_attn_d128_scores(const AttnLaunch& L, cudaStream_t stream) {
    return L.p.q_len > 1 ? launch_attn_for_d<128, true, true>(L, stream)
                         : launch_attn_for_d<128, false, true>(L, stream);
}
}  // namespace pa
