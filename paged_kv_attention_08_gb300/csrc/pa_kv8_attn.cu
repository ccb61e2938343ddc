// Attention over the 8-bit cache, simplest form: a warp to a query row.
#include "pa_kv8.cuh"

namespace pa {

namespace {

template <typename T>
__global__ void __launch_bounds__(128) kv8_attention_kernel(const Kv8Params p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)p.q_len * p.num_heads) return;
    const int qi = (int)(row / p.num_heads), h = (int)(row % p.num_heads);
    const int D = p.head_dim, n = D / 32, kvh = h / p.group;
    const size_t at = (((size_t)b * p.q_len + qi) * p.num_heads + h) * D;
    float q[8], acc[8];
    for (int i = 0; i < 8; ++i) {
        q[i] = i < n ? (float)static_cast<const T*>(p.q)[at + lane + i * 32] : 0.f;
        acc[i] = 0.f;
    }
    const int reach = min(reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size), p.token_limit);
    const int limit = min(reach, max(__ldg(p.context_lens + b), 0) - p.q_len + qi + 1);
    float m = -INFINITY, l = 0.f;
    for (int t = 0; t < limit; ++t) {
        const int e = __ldg(p.block_tables + (size_t)b * p.max_blocks + t / p.block_size);
        if (e < 0 || (int64_t)e >= p.num_blocks) continue;
        const size_t c = (((size_t)e * p.block_size + t % p.block_size) * p.num_kv_heads + kvh) * D;
        float s = 0.f, v[8];
        for (int i = 0; i < n; ++i) {
            float k0, unused;
            Mma<__half>::unpack(decode2(p.k_cache[c + lane + i * 32]), k0, unused);
            Mma<__half>::unpack(decode2(p.v_cache[c + lane + i * 32]), v[i], unused);
            s = fmaf(q[i], k0, s);
        }
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        s *= p.qscale * __ldg(p.k_scales + (size_t)e * p.num_kv_heads + kvh);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        const float vs = w * __ldg(p.v_scales + (size_t)e * p.num_kv_heads + kvh);
        m = mn;
        l = l * f + w;
        for (int i = 0; i < n; ++i) acc[i] = acc[i] * f + vs * v[i];
    }
    for (int i = 0; i < n; ++i)
        store_out(p.out, at + lane + i * 32, l == 0.f ? 0.f : acc[i] / l, p.out_dtype);
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8Params& p, bool bf16, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)p.q_len * p.num_heads + 3) / 4), (unsigned)p.batch);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return bf16 ? cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__half>, p);
}

}  // namespace pa
