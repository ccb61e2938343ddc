// Accumulated attention weights: after an attention call has left each query
// row's statistics lse = m + log2 l, every cached token's weight
//     weights[b, kvh, t] += sum over the rows r of the kv head of 2^(s_rt - lse_r),
//     s_rt = q_r . K_t * scale * log2(e),
// is added by reading the keys once more.
//
// The tokens are the 16 rows of a warp-level m16n8k16 MMA and the query rows
// its columns, so that a token's sum over the query rows stays in one quad's
// registers.  A contraction may take its terms in any order: lane `tig` of a
// quad takes the eight neighbouring elements 8 tig .. 8 tig + 7 of every 32
// (one 16-byte load of a key row, one of a query row) as its share of two MMA
// steps, so keys go from memory to the fragments' registers with no staging.
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kWThreads = 256;
constexpr int kWWarps = kWThreads / 32;
constexpr int kWRows = 64;  // query rows in shared memory at a time

// One CTA per (run of 16-token tiles, kv head, sequence), one tile per warp at a time.
template <int D, typename KV>
__global__ void __launch_bounds__(kWThreads) weights_kernel(const WeightParams p) {
    constexpr int C = D / 32;        // 32-element column groups
    constexpr int QS = D + 8;        // row stride in shared memory: 16 bytes more than the row
    __shared__ __align__(16) KV qs[kWRows * QS];
    __shared__ float ls[kWRows];
    __shared__ int lim[kWRows];      // tokens each row attends to
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.group, rows = p.q_len * G;
    grid_dependency_wait();
    grid_launch_dependents();

    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int ctx = max(__ldg(p.context_lens + b), 0);
    const int npages = (T + p.block_size - 1) / p.block_size;
    const int32_t* table_row = p.block_tables + (size_t)b * p.max_blocks;
    const size_t unit = ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * p.block_size;
    const int tiles = (T + 15) / 16;
    for (int first = blockIdx.x * kWWarps; first < tiles; first += gridDim.x * kWWarps) {
        const int t0 = (first + warp) * 16;
        const int phys = t0 < T ? page_phys(table_row, t0 / p.block_size, npages, p.num_blocks) : -1;
        // keys of tokens g and g + 8, in the fragments' order
        uint4 ka[C], kb[C];
        if (phys >= 0) {
            const size_t slot = (size_t)phys * p.block_size + t0 % p.block_size;
            const KV* k = static_cast<const KV*>(p.k_cache) +
                          ((slot + g) * p.num_kv_heads + kvh) * D + tig * 8;
            const size_t down = (size_t)8 * p.num_kv_heads * D;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                ka[c] = *reinterpret_cast<const uint4*>(k + c * 32);
                kb[c] = *reinterpret_cast<const uint4*>(k + down + c * 32);
            }
        }
        float sum0 = 0.f, sum1 = 0.f;  // tokens g and g + 8
        for (int r0 = 0; r0 < rows; r0 += kWRows) {
            __syncthreads();  // the previous rows have been used
            for (int i = tid; i < kWRows * (D / 8); i += kWThreads) {
                const int r = i / (D / 8), c = i % (D / 8), u = r0 + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (u < rows)
                    v = __ldg(reinterpret_cast<const uint4*>(
                                  static_cast<const KV*>(p.q) +
                                  (((size_t)b * p.q_len + u / G) * p.num_heads + kvh * G + u % G) * D) +
                              c);
                *reinterpret_cast<uint4*>(qs + r * QS + c * 8) = v;
            }
            if (tid < kWRows) {
                const int u = r0 + tid;
                ls[tid] = u < rows ? p.lse[((size_t)b * p.q_len + u / G) * p.num_heads + kvh * G + u % G]
                                   : INFINITY;
                lim[tid] = u < rows ? min(min(T, p.token_limit), ctx - p.q_len + u / G + 1) : 0;
            }
            __syncthreads();
            if (phys < 0) continue;
            const int n8 = (min(rows - r0, kWRows) + 7) / 8;
            for (int n = 0; n < n8; ++n) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 qv = *reinterpret_cast<const uint4*>(qs + (n * 8 + g) * QS + c * 32 + tig * 8);
                    const uint32_t a0[4] = {ka[c].x, kb[c].x, ka[c].y, kb[c].y};
                    const uint32_t a1[4] = {ka[c].z, kb[c].z, ka[c].w, kb[c].w};
                    Mma<KV>::mma(s, a0, qv.x, qv.y);
                    Mma<KV>::mma(s, a1, qv.z, qv.w);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + tig * 2 + e;
                    const float l = ls[r];
                    const int end = lim[r];
                    // (a row that attends to nothing has lse = +inf: weight 0)
                    if (t0 + g < end) sum0 += fast_exp2(fmaf(s[e], p.qscale, -l));
                    if (t0 + g + 8 < end) sum1 += fast_exp2(fmaf(s[2 + e], p.qscale, -l));
                }
            }
        }
        sum0 += __shfl_xor_sync(kFullMask, sum0, 1);
        sum1 += __shfl_xor_sync(kFullMask, sum1, 1);
        sum0 += __shfl_xor_sync(kFullMask, sum0, 2);
        sum1 += __shfl_xor_sync(kFullMask, sum1, 2);
        if (tig < 2) {
            const int t = t0 + g + 8 * tig;
            if (t < T) p.weights_out[unit + t] = p.weights_in[unit + t] + (tig ? sum1 : sum0);
        }
    }
}

// From scores that the attention left: one thread per four neighbouring tokens
// of a kv head.  Bound: memory, 4 bytes per (row, token) and 8 per token.
constexpr int kSThreads = 256;

__global__ void __launch_bounds__(kSThreads) weights_of_scores_kernel(const WeightParams p) {
    __shared__ float ls[16];
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.group, rows = p.q_len * G;
    grid_dependency_wait();
    grid_launch_dependents();
    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int t0 = blockIdx.x * (kSThreads * 4) + tid * 4;
    if (tid < rows)
        ls[tid] = p.lse[((size_t)b * p.q_len + tid / G) * p.num_heads + kvh * G + tid % G];
    __syncthreads();
    if (t0 >= T) return;
    const int npages = (T + p.block_size - 1) / p.block_size;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t0 < p.token_limit && page_phys(p.block_tables + (size_t)b * p.max_blocks, t0 / p.block_size,
                                        npages, p.num_blocks) >= 0) {
        const float* s = p.scores + ((size_t)b * p.num_kv_heads + kvh) * rows * p.score_width + t0;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(s + (size_t)r * p.score_width));
            const float l = ls[r];  // (+inf where the row attends to nothing: weight 0)
            sum.x += fast_exp2(fmaf(x.x, p.qscale, -l));
            sum.y += fast_exp2(fmaf(x.y, p.qscale, -l));
            sum.z += fast_exp2(fmaf(x.z, p.qscale, -l));
            sum.w += fast_exp2(fmaf(x.w, p.qscale, -l));
        }
    }
    const size_t at = ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * p.block_size + t0;
    const float* in = p.weights_in + at;
    float* out = p.weights_out + at;
    if (t0 + 4 <= T && ((reinterpret_cast<uintptr_t>(p.weights_in) |
                         reinterpret_cast<uintptr_t>(p.weights_out)) & 15) == 0) {
        const float4 w = *reinterpret_cast<const float4*>(in);
        *reinterpret_cast<float4*>(out) =
            make_float4(w.x + sum.x, w.y + sum.y, w.z + sum.z, w.w + sum.w);
    } else {
        const float d[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t0 + e < T) out[e] = in[e] + d[e];
    }
}

template <int D>
cudaError_t launch_d(const WeightParams& p, int kv_dtype, const cudaLaunchConfig_t& cfg) {
    return kv_dtype == PA_BF16 ? cudaLaunchKernelEx(&cfg, weights_kernel<D, __nv_bfloat16>, p)
                               : cudaLaunchKernelEx(&cfg, weights_kernel<D, __half>, p);
}

}  // namespace

cudaError_t launch_weights_of_scores(const WeightParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // every token of the table: those past the scores take a weight of 0
    const int64_t tokens = (int64_t)p.max_blocks * p.block_size;
    cfg.gridDim = dim3((unsigned)((tokens + kSThreads * 4 - 1) / (kSThreads * 4)),
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

cudaError_t launch_weights(const WeightParams& p, int head_dim, int kv_dtype, int max_tokens,
                           bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    const int per_cta = kWWarps * 16;
    cfg.gridDim = dim3((unsigned)((max_tokens + per_cta - 1) / per_cta), (unsigned)p.num_kv_heads,
                       (unsigned)p.batch);
    cfg.blockDim = dim3(kWThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    switch (head_dim) {
        case 64: return launch_d<64>(p, kv_dtype, cfg);
        case 128: return launch_d<128>(p, kv_dtype, cfg);
        default: return launch_d<256>(p, kv_dtype, cfg);
    }
}

}  // namespace pa
