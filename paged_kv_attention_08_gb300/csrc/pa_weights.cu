// Accumulated attention weights from stored scores (pa_weights.cuh) where the rows'
// statistics are known when the attention kernel ends; those of partitions
// are joined beside the combine (pa_combine.cu).
#include "pa_weights.cuh"

namespace pa {

namespace {

__global__ void __launch_bounds__(kSThreads) weights_of_scores_kernel(const WeightParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    add_scored_weights(p, blockIdx.x, gridDim.x, blockIdx.y, blockIdx.z);
}

}  // namespace

cudaError_t launch_weights_of_scores(const WeightParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(weight_tiles(p)),
                       (unsigned)p.num_kv_heads, (unsigned)p.batch);
    cfg.blockDim = dim3(kSThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, weights_of_scores_kernel, p);
}

}  // namespace pa
