// Instantiations of the tcgen05 tile kernel for head_dim 64 with row
// statistics, a shared prefix or a limit of the tokens.
#include "pa_tile.cuh"

namespace pa {
cudaError_t launch_tile_d64_extended(const AttnLaunch& L, cudaStream_t stream) {
    return launch_tile_extended_for_d<64, kTileRows>(L, stream);
}
}  // namespace pa
