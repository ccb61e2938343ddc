// Instantiations of the attention over the 8-bit cache for head_dim 128.
#include "pa_kv8_attn.cuh"

namespace pa {
cudaError_t launch_kv8_d128(const Kv8Launch& L, cudaStream_t stream) {
    return launch_kv8_for_d<128>(L, stream);
}
}  // namespace pa
