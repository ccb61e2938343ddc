// Instantiations of the tcgen05 tile kernel for compact units (head_dim 256, at
// most 16 rows) with row statistics, a shared prefix or a limit of the tokens.
#include "pa_tile.cuh"

namespace pa {
cudaError_t launch_tile_d256_compact_extended(const AttnLaunch& L, cudaStream_t stream) {
    return launch_tile_extended_for_d<256, kTileCompactQRows>(L, stream);
}
}  // namespace pa
