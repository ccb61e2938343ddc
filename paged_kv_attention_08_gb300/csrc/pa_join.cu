// Joins the partitions of an attention over the 8-bit or the latent cache: with
// (m, l, acc) of each partition,
//     M = max m,  out = sum 2^(m - M) acc / sum 2^(m - M) l,
// zeros for a row without a token.
//
// Bound by the partials' bytes, which the attention has just written (they come
// from L2), and by the latency of the three steps: statistics, sums, join.  A
// CTA takes 128 columns of a row: 32 threads hold four columns each, and four such
// groups (at 64 columns, eight of 16) share the partitions.
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kJoinThreads = 128;

template <int COLS>  // columns of a CTA: 128 or 64
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinParams p) {
    constexpr int LANES = COLS / 4, GROUPS = kJoinThreads / LANES;
    extern __shared__ float weight[];  // [partitions]
    __shared__ float red[kJoinThreads / 32];
    __shared__ float4 sums[GROUPS][LANES];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slabs = p.width / COLS;
    const int row = blockIdx.x / slabs, col = blockIdx.x % slabs * COLS;
    const int kvh = blockIdx.y, b = blockIdx.z;   // row: (query token, head of the group)
    const int reach = min(reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size), p.token_limit);
    const int pages = (reach + p.block_size - 1) / p.block_size;
    const int parts = min((pages + p.part_pages - 1) / p.part_pages, p.num_parts);
    // partition x of the row
    const size_t first = ((size_t)b * gridDim.y + kvh) * p.num_parts * p.unit_rows + row;
    float m = -INFINITY;
    for (int x = tid; x < parts; x += kJoinThreads) {
        const float v = p.part_ml[(first + (size_t)x * p.unit_rows) * 2];
        weight[x] = v;
        m = fmaxf(m, v);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, k));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    const float M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float l = 0.f;
    for (int x = tid; x < parts; x += kJoinThreads) {
        const float w = weight[x] == -INFINITY ? 0.f : fast_exp2(weight[x] - M);
        weight[x] = w;
        l = fmaf(w, p.part_ml[(first + (size_t)x * p.unit_rows) * 2 + 1], l);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(kFullMask, l, k);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    const float L = red[0] + red[1] + red[2] + red[3];
    const int c = tid % LANES, grp = tid / LANES;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = grp; x < parts; x += GROUPS) {
        const float w = weight[x];
        const float4 v = *reinterpret_cast<const float4*>(
            p.part_acc + (first + (size_t)x * p.unit_rows) * p.width + col + c * 4);
        if (w != 0.f) {
            a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y);
            a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
        }
    }
    sums[grp][c] = a;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int x = 1; x < GROUPS; ++x) {
            const float4 v = sums[x][c];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        const int qi = row / p.group, h = kvh * p.group + row % p.group;
        const size_t at = (((size_t)b * (p.unit_rows / p.group) + qi) * gridDim.y * p.group + h) * p.width + col + c * 4;
        const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) store_out(p.out, at + i, L == 0.f ? 0.f : v[i] / L, p.out_dtype);
    }
}

}  // namespace

cudaError_t launch_join(const JoinParams& p, int batch, int num_kv_heads, bool pdl, cudaStream_t stream) {
    auto kern = p.width == 64 ? join_kernel<64> : join_kernel<128>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.unit_rows * (p.width == 64 ? 1 : p.width / 128)),
                       (unsigned)num_kv_heads, (unsigned)batch);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = (size_t)p.num_parts * 4;  // (at most kMaxJoinParts: 32 KB)
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pa
