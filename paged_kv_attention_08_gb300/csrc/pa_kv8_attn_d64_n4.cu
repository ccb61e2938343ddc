// Instantiations of the attention over the 8-bit cache for head_dim 64 and up to
// 32 query rows of a CTA.
#include "pa_kv8_attn.cuh"

namespace pa {
cudaError_t launch_kv8_d64_n4(const Kv8Launch& L, cudaStream_t stream) {
    return launch_kv8_for<64, 4>(L, stream);
}
int kv8_ctas_d64_n4() { return kv8_ctas<64, 4>; }
}  // namespace pa
