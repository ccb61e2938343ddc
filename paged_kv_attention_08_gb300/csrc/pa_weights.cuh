// Accumulated attention weights from scores that the attention kernel left:
//     weights[b, kvh, t] += sum over the rows r of the kv head of 2^(s_rt - lse_r),
//     s_rt = q_r . K_t * scale * log2(e),   lse_r = m_r + log2 l_r.
// (pa_weights_tile.cu forms the scores again, for more rows than are worth storing.)
#pragma once

#include "pa_device.cuh"

namespace pa {

// One thread per four neighbouring tokens of a kv head.  Bound: memory, 4 bytes
// per (row, token) and 8 per token: 4 rows of 1M (token, kv head) pairs, 25 MB, in
// 10.7 us cold, 14.0 with the combine of 1024 rows in the same launch.  The scores
// are stored in fp32, as they were formed.  (Reading the keys again instead took 79
// us there, and 135 us for 2M pairs.)
constexpr int kSThreads = 256;
// Tokens that a CTA of kSThreads threads takes.
constexpr int kSTokens = kSThreads * 4;

__host__ __device__ inline int weight_tiles(const WeightParams& p) {
    return (int)((p.score_width + kSTokens - 1) / kSTokens);
}

// The CTA's share: tokens number `tile` of `tiles` of a kv head of a sequence.
__device__ __forceinline__ void add_scored_weights(const WeightParams& p, int tile, int tiles, int kvh,
                                                   int b) {
    __shared__ float ls[16];
    const int tid = threadIdx.x;
    const int G = p.group, rows = p.q_len * G;
    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int t0 = tile * kSTokens + tid * 4;
    if (tile * kSTokens >= T) return;
    const size_t unit = ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * p.block_size;
    if (tile == tiles - 1)  // tokens past the scores: nothing to add
        for (int t = tiles * kSTokens + tid; t < T; t += kSThreads)
            p.weights_out[unit + t] = p.weights_in[unit + t];
    const int npages = (T + p.block_size - 1) / p.block_size;
    if (p.part_ml) {
        // m + log2 l over the partitions that hold tokens: a warp per row in turn
        const int parts = min((npages + p.part_pages - 1) / p.part_pages, p.num_parts);
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml) +
                           ((size_t)b * p.num_kv_heads + kvh) * p.num_parts * rows;
        const int lane = tid & 31;
        for (int r = tid >> 5; r < rows; r += kSThreads / 32) {
            float m = -INFINITY, l = 0.f;
            for (int q = lane; q < parts; q += 32) {
                const float2 v = ml[(size_t)q * rows + r];
                if (v.x == -INFINITY) continue;
                const float n = fmaxf(m, v.x);
                l = l * (m == -INFINITY ? 0.f : exp2f(m - n)) + v.y * exp2f(v.x - n);
                m = n;
            }
            float M = m;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, d));
            l *= m == -INFINITY ? 0.f : exp2f(m - M);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(kFullMask, l, d);
            if (lane == 0) ls[r] = row_lse(M, l);
        }
    } else if (tid < rows) {
        ls[tid] = p.lse[((size_t)b * p.q_len + tid / G) * p.num_heads + kvh * G + tid % G];
    }
    __syncthreads();
    if (t0 >= T) return;
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
    const float* in = p.weights_in + unit + t0;
    float* out = p.weights_out + unit + t0;
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

}  // namespace pa
