// Attention over the latent cache, simplest form: a warp to a query row.
#include "pa_device.cuh"

namespace pa {

namespace {

template <typename T>
__global__ void __launch_bounds__(128) latent_attention_kernel(const LatentParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)p.q_len * p.num_heads) return;
    const int qi = (int)(row / p.num_heads), h = (int)(row % p.num_heads);
    const int R = p.latent_dim, W = R + 64;
    const size_t at = ((size_t)b * p.q_len + qi) * p.num_heads + h;
    float q[18], acc[16];
    for (int i = 0; i < 18; ++i)
        q[i] = i < W / 32 ? (float)static_cast<const T*>(p.q)[at * W + lane + i * 32] : 0.f;
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    const int reach = min(reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size), p.token_limit);
    const int limit = min(reach, max(__ldg(p.context_lens + b), 0) - p.q_len + qi + 1);
    float m = -INFINITY, l = 0.f;
    for (int t = 0; t < limit; ++t) {
        const int e = __ldg(p.block_tables + (size_t)b * p.max_blocks + t / p.block_size);
        if (e < 0 || (int64_t)e >= p.num_blocks) continue;
        const T* c = static_cast<const T*>(p.cache) + ((size_t)e * p.block_size + t % p.block_size) * W;
        float s = 0.f, v[18];
        for (int i = 0; i < W / 32; ++i) {
            v[i] = (float)c[lane + i * 32];
            s = fmaf(q[i], v[i], s);
        }
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        s *= p.qscale;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * f + w;
        for (int i = 0; i < R / 32; ++i) acc[i] = acc[i] * f + w * v[i];
    }
    for (int i = 0; i < R / 32; ++i)
        static_cast<T*>(p.out)[at * R + lane + i * 32] = (T)(l == 0.f ? 0.f : acc[i] / l);
}

}  // namespace

cudaError_t launch_latent_attention(const LatentParams& p, bool bf16, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)p.q_len * p.num_heads + 3) / 4), (unsigned)p.batch);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return bf16 ? cudaLaunchKernelEx(&cfg, latent_attention_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, latent_attention_kernel<__half>, p);
}

}  // namespace pa
