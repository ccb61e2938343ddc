// Instantiations of the decode kernel for head_dim 128 with a shared prefix in
// front of each sequence's own pages.
#include "pa_attn.cuh"

namespace pa {
cudaError_t launch_attn_d128_prefixed(const AttnLaunch& L, cudaStream_t stream) {
    return L.p.q_len > 1 ? launch_attn_for_d<128, true, false, true>(L, stream)
                         : launch_attn_for_d<128, false, false, true>(L, stream);
}
}  // namespace pa
