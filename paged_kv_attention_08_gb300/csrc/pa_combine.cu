// Split-KV combine and page-walk export.
//
// Combine (flash-decoding-bench "design.md": each chunk's local max, sum and
// weighted values are reduced into the final output): for query head h of
// query token qi of sequence b, with partitions p holding (m_p, l_p, acc_p)
// in base-2 units,
//     M = max_p m_p,   L = sum_p 2^(m_p - M) l_p,
//     out = sum_p 2^(m_p - M) acc_p / L.
// Partitions past the sequence's context are never read; an empty partition
// (m = -inf, l = 0, acc = 0) contributes nothing; a sequence with no attended
// token gets zeros.
#include "pa_device.cuh"
#include "pa_weights.cuh"

namespace pa {

namespace {

// One CTA of 256 threads per (query token and head, sequence).  Every thread loads the
// (m, l) of a few partitions; two block reductions give the maximum and the
// weighted normaliser.  The threads then form PGRP groups over the
// partitions, each thread a 16-byte slice of the head dimension, so that all
// acc loads of a head are in flight at once; a shared-memory sum over the
// groups finishes the head.  Two dependent memory round trips in all.
constexpr int kCombineThreads = 256;

// x: query token and head; LSE: the rows' statistics are wanted too (p.lse).
template <int D, bool LSE>
__device__ __forceinline__ void combine_row(const CombineParams& p, int x, int b) {
    constexpr int SLICES = D / 4;                      // float4 slices of one row
    constexpr int PGRP = kCombineThreads / SLICES;     // partition groups
    constexpr float NEG_INF = -INFINITY;
    extern __shared__ float weight[];                  // [num_parts]
    __shared__ float red[kCombineThreads / 32];
    __shared__ float4 part[PGRP][SLICES];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = x % p.num_heads, qi = x / p.num_heads;
    const int kvh = h / p.group;
    const int U = p.q_len * p.group, u = qi * p.group + h % p.group;  // rows of a unit; this row
    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int npages = (T + p.block_size - 1) / p.block_size;
    const int nparts = min((npages + p.part_pages - 1) / p.part_pages, p.num_parts);

    const size_t row0 = ((size_t)b * p.num_kv_heads + kvh) * p.num_parts;  // partition 0 of (b, kvh)
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);

    float mx = NEG_INF;
    for (int q = tid; q < nparts; q += kCombineThreads) mx = fmaxf(mx, ml[(row0 + q) * U + u].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, m));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = red[0];
#pragma unroll
    for (int w = 1; w < kCombineThreads / 32; ++w) mx = fmaxf(mx, red[w]);
    __syncthreads();

    float ls = 0.f;
    for (int q = tid; q < nparts; q += kCombineThreads) {
        const float2 v = ml[(row0 + q) * U + u];
        const float w = (v.x == NEG_INF) ? 0.f : exp2f(v.x - mx);
        weight[q] = w;
        ls = fmaf(w, v.y, ls);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ls += __shfl_xor_sync(kFullMask, ls, m);
    if (lane == 0) red[warp] = ls;
    __syncthreads();  // also publishes `weight`
    ls = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) ls += red[w];

    const bool empty = (mx == NEG_INF) || !(ls > 0.f);
    const int pg = tid / SLICES, sl = tid % SLICES;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!empty) {
        const float4* src = reinterpret_cast<const float4*>(p.part_acc + (row0 * U + u) * D) + sl;
        const size_t stride = (size_t)U * SLICES;  // float4s between partitions
#pragma unroll 4
        for (int q = pg; q < nparts; q += PGRP) {
            const float w = weight[q];
            const float4 x = src[(size_t)q * stride];
            a.x = fmaf(w, x.x, a.x);
            a.y = fmaf(w, x.y, a.y);
            a.z = fmaf(w, x.z, a.z);
            a.w = fmaf(w, x.w, a.w);
        }
    }
    part[pg][sl] = a;
    __syncthreads();
    if (pg == 0) {
        for (int k = 1; k < PGRP; ++k) {
            const float4 x = part[k][sl];
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
        const float inv = empty ? 0.f : 1.f / ls;
        const size_t o = (((size_t)b * p.q_len + qi) * p.num_heads + h) * D + sl * 4;
        if (LSE && sl == 0) p.lse[o / D] = empty ? INFINITY : row_lse(mx, ls);
        store_out(p.out, o, a.x * inv, p.out_dtype);
        store_out(p.out, o + 1, a.y * inv, p.out_dtype);
        store_out(p.out, o + 2, a.z * inv, p.out_dtype);
        store_out(p.out, o + 3, a.w * inv, p.out_dtype);
    }
}

template <int D, bool LSE>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
    grid_dependency_wait();                            // partials come from the attention kernel
    grid_launch_dependents();
    combine_row<D, LSE>(p, blockIdx.x, blockIdx.y);
}

// The combine and, beside it in the same launch, the tokens' weights from the
// scores and the partitions' statistics: both need the attention kernel alone,
// and both wait for it.
template <int D>
__global__ void __launch_bounds__(kCombineThreads)
    combine_weights_kernel(const CombineParams p, const WeightParams w) {
    static_assert(kCombineThreads == kSThreads, "CTAs of both kinds");
    grid_dependency_wait();
    grid_launch_dependents();
    const int rows = p.q_len * p.num_heads;
    const int x = (int)blockIdx.x - rows, tiles = weight_tiles(w);
    if (x < 0) combine_row<D, false>(p, blockIdx.x, blockIdx.y);
    else add_scored_weights(w, x % tiles, tiles, x / tiles, blockIdx.y);
}

// Combine for the balanced split: the attention kernel's CTA c covered pages
// [c*W/C, (c+1)*W/C) of the flattened (sequence, kv head, page) order and
// wrote every unit it covered whole; a unit spread over CTAs c0..c1 left one
// record in each: slot 1 of c0 when the unit began inside c0's range (slot 0
// when exactly at its start), slot 0 of every later CTA whose share is not
// empty (with more CTAs than pages, some CTAs take no page and write nothing).  One CTA per (query
// head, sequence) finds its unit's CTAs from the same arithmetic and merges
// their records as the partition combine does.  Records hold every row of a
// unit: [C][2][Q * G].
template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_balanced_kernel(const CombineParams p) {
    constexpr int SLICES = D / 4;
    constexpr int PGRP = kCombineThreads / SLICES;
    constexpr float NEG_INF = -INFINITY;
    extern __shared__ float weight[];                  // [records]
    __shared__ float red[kCombineThreads / 32];
    __shared__ float4 part[PGRP][SLICES];
    __shared__ long long span[2];                      // W, flat start of sequence b
    grid_dependency_wait();
    grid_launch_dependents();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = (int)blockIdx.x % p.num_heads, qi = (int)blockIdx.x / p.num_heads;
    const int b = blockIdx.y;
    const int Hkv = p.num_kv_heads;
    const int kvh = h / p.group;
    const int U = p.q_len * p.group, u = qi * p.group + h % p.group;
    if (warp == 0) {
        long long all = 0, before = 0;
        for (int b0 = lane; b0 < p.batch; b0 += 32) {
            const int T = reachable_tokens(p.context_lens, b0, p.max_blocks, p.block_size);
            const int np = (T + p.block_size - 1) / p.block_size;
            all += np;
            if (b0 < b) before += np;
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            all += __shfl_xor_sync(kFullMask, all, m);
            before += __shfl_xor_sync(kFullMask, before, m);
        }
        if (lane == 0) {
            span[0] = all * Hkv;
            span[1] = before * Hkv;
        }
    }
    __syncthreads();
    const long long W = span[0];
    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int np = (T + p.block_size - 1) / p.block_size;
    const size_t o = (((size_t)b * p.q_len + qi) * p.num_heads + h) * D;
    if (np == 0) {  // no page, no CTA: the empty-context result
        for (int d = tid; d < D; d += kCombineThreads) store_out(p.out, o + d, 0.f, p.out_dtype);
        return;
    }
    const long long Cn = p.num_ctas;
    const long long A = span[1] + (long long)kvh * np, E = A + np;
    const long long c0 = ((A + 1) * Cn - 1) / W, c1 = (E * Cn - 1) / W;
    if (c0 == c1) return;  // one CTA covered the unit and wrote it
    const int nrec = (int)(c1 - c0 + 1);
    const bool c0_tail = A != c0 * W / Cn;
    auto rec_row = [&](int k) -> size_t {
        const long long c = c0 + k;
        const int slotk = (k == 0 && c0_tail) ? 1 : 0;
        return ((size_t)c * 2 + slotk) * U + u;
    };
    // CTA c0 + k wrote a record only if its share [c*W/C, (c+1)*W/C) is not empty
    auto live = [&](int k) -> bool {
        const long long c = c0 + k;
        return (c + 1) * W / Cn > c * W / Cn;
    };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);

    float mx = NEG_INF;
    for (int k = tid; k < nrec; k += kCombineThreads)
        if (live(k)) mx = fmaxf(mx, ml[rec_row(k)].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, m));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = red[0];
#pragma unroll
    for (int w = 1; w < kCombineThreads / 32; ++w) mx = fmaxf(mx, red[w]);
    __syncthreads();
    float ls = 0.f;
    for (int k = tid; k < nrec; k += kCombineThreads) {
        float w = 0.f;
        if (live(k)) {
            const float2 v = ml[rec_row(k)];
            w = (v.x == NEG_INF) ? 0.f : exp2f(v.x - mx);
            ls = fmaf(w, v.y, ls);
        }
        weight[k] = w;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ls += __shfl_xor_sync(kFullMask, ls, m);
    if (lane == 0) red[warp] = ls;
    __syncthreads();  // also publishes `weight`
    ls = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) ls += red[w];

    const bool empty = (mx == NEG_INF) || !(ls > 0.f);
    const int pg = tid / SLICES, sl = tid % SLICES;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!empty) {
        for (int k = pg; k < nrec; k += PGRP) {
            const float w = weight[k];
            if (w == 0.f) continue;  // no record (or an empty one): nothing to add
            const float4 x = reinterpret_cast<const float4*>(p.part_acc + rec_row(k) * D)[sl];
            a.x = fmaf(w, x.x, a.x);
            a.y = fmaf(w, x.y, a.y);
            a.z = fmaf(w, x.z, a.z);
            a.w = fmaf(w, x.w, a.w);
        }
    }
    part[pg][sl] = a;
    __syncthreads();
    if (pg == 0) {
        for (int k = 1; k < PGRP; ++k) {
            const float4 x = part[k][sl];
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
        const float inv = empty ? 0.f : 1.f / ls;
        store_out(p.out, o + sl * 4, a.x * inv, p.out_dtype);
        store_out(p.out, o + sl * 4 + 1, a.y * inv, p.out_dtype);
        store_out(p.out, o + sl * 4 + 2, a.z * inv, p.out_dtype);
        store_out(p.out, o + sl * 4 + 3, a.w * inv, p.out_dtype);
    }
}

// Joining a shared prefix with the sequences' own tokens: a query row has
// partials (m, l, acc) of the prefix's partitions, in the prefix's rows (its
// n sequences' query tokens in order), and of its own sequence's.  With x over
// both, out = sum_x 2^(m_x - M) acc_x / sum_x 2^(m_x - M) l_x: the softmax over
// the tokens of prefix and sequence as one.  Partitions past the tokens are
// never read.
//
// One warp per row: a lane holds the statistics of one partition (32 at a
// time, M and the sums carried along when there are more) and D / 32 columns
// of the result, and the accs of eight partitions are in flight before their
// weights are known.  Bound: the latency of lengths, statistics and accs in
// turn.  (A CTA per row, as in combine_kernel, took 17.5 us for 4096 rows of 6
// partitions at head_dim 128 and 19.4 us for 4096 of 6 at 256.)
template <int D>
__global__ void __launch_bounds__(kCombineThreads) prefix_combine_kernel(const PrefixCombineParams p) {
    constexpr int F = D / 32;   // columns of a lane, in groups of V, 32 V columns apart
    constexpr int V = F < 4 ? F : 4;
    constexpr int AHEAD = D == 256 ? 4 : 8;
    constexpr float NEG_INF = -INFINITY;
    grid_dependency_wait();
    grid_launch_dependents();

    const int lane = threadIdx.x & 31;
    const int rows = p.q_len * p.num_heads;
    const int x = blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5);
    if (x >= rows) return;
    const int h = x % p.num_heads, qi = x / p.num_heads;
    const int b = blockIdx.y, pre = b / p.per_prefix;
    const int kvh = h / p.group, hg = h % p.group;
    const int own_rows = p.q_len * p.group, pre_rows = p.per_prefix * own_rows;
    const int Tp = reachable_tokens(p.prefix_lens, pre, p.max_prefix_blocks, p.block_size);
    const int To = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const int np_pages = (Tp + p.block_size - 1) / p.block_size;
    const int no_pages = (To + p.block_size - 1) / p.block_size;
    const int np = min((np_pages + p.prefix_part_pages - 1) / p.prefix_part_pages, p.prefix_parts);
    const int no = min((no_pages + p.own_part_pages - 1) / p.own_part_pages, p.own_parts);
    // rows of partition q of the prefix, and of the sequence
    const size_t rp = ((size_t)pre * p.num_kv_heads + kvh) * p.prefix_parts * pre_rows +
                      ((b - pre * p.per_prefix) * p.q_len + qi) * p.group + hg;
    const size_t ro = ((size_t)b * p.num_kv_heads + kvh) * p.own_parts * own_rows + qi * p.group + hg;
    const int parts = np + no;

    float M = NEG_INF, L = 0.f, a[F];
#pragma unroll
    for (int f = 0; f < F; ++f) a[f] = 0.f;
    for (int q0 = 0; q0 < parts; q0 += 32) {
        const int count = min(parts - q0, 32);
        auto acc_of = [&](int q, float (&v)[F]) {  // partition q0 + q's acc, this lane's columns
            const int i = q0 + q;
            const float* src = i < np ? p.prefix_acc + (rp + (size_t)i * pre_rows) * D
                                      : p.own_acc + (ro + (size_t)(i - np) * own_rows) * D;
#pragma unroll
            for (int f = 0; f < F; f += V) {
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(src + f * 32 + lane * 4);
                    v[f] = y.x, v[f + 1] = y.y, v[f + 2] = y.z, v[f + 3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(src + f * 32 + lane * 2);
                    v[f] = y.x, v[f + 1] = y.y;
                }
            }
        };
        float2 st = make_float2(NEG_INF, 0.f);
        if (lane < count) {
            const int i = q0 + lane;
            st = i < np ? reinterpret_cast<const float2*>(p.prefix_ml)[rp + (size_t)i * pre_rows]
                        : reinterpret_cast<const float2*>(p.own_ml)[ro + (size_t)(i - np) * own_rows];
        }
        float v[AHEAD][F];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (q < count) acc_of(q, v[q]);
        float mx = st.x;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, m));
        mx = fmaxf(mx, M);
        if (mx == NEG_INF) continue;  // nothing so far (the same in every lane)
        const float keep = M == NEG_INF ? 0.f : exp2f(M - mx);
        const float w = st.x == NEG_INF ? 0.f : exp2f(st.x - mx);
        float l = w * st.y;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) l += __shfl_xor_sync(kFullMask, l, m);
        L = fmaf(L, keep, l);
        M = mx;
#pragma unroll
        for (int f = 0; f < F; ++f) a[f] *= keep;
        for (int q1 = 0; q1 < count; q1 += AHEAD) {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                if (q1 + q >= count) break;
                const float wq = __shfl_sync(kFullMask, w, q1 + q);
                if (q1 > 0) acc_of(q1 + q, v[q]);
#pragma unroll
                // (an empty partition's acc is zeros)
                for (int f = 0; f < F; ++f) a[f] = fmaf(wq, v[q][f], a[f]);
            }
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const size_t o = ((size_t)b * rows + x) * D;
#pragma unroll
    for (int f = 0; f < F; f += V) {
        const size_t at = o + f * 32 + lane * V;
        if (p.out_dtype == PA_F32) {
            float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int e = 0; e < V; e += 2)
                *reinterpret_cast<float2*>(dst + e) = make_float2(a[f + e] * inv, a[f + e + 1] * inv);
        } else {
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
            for (int e = 0; e < V; e += 2)
                dst[e / 2] = p.out_dtype == PA_F16
                                 ? Mma<__half>::pack(a[f + e] * inv, a[f + e + 1] * inv)
                                 : Mma<__nv_bfloat16>::pack(a[f + e] * inv, a[f + e + 1] * inv);
        }
    }
}

// Append of one new token per sequence (MiniVLLM docs "Decoding Benchmark":
// each decode step stores the new token's keys/values in the block the table
// assigns, at slot position % block_size).  One CTA per sequence copies the
// token's row for all kv heads (contiguous in both the new-token array and
// the cache slot) with 16-byte vectors.  Positions outside the table row and
// masked entries write nothing.
__global__ void __launch_bounds__(128) append_kernel(uint4* k_cache, uint4* v_cache,
                                                    const uint4* k_new, const uint4* v_new,
                                                    const int32_t* block_tables,
                                                    const int32_t* positions, int32_t max_blocks,
                                                    int32_t block_size, int64_t num_blocks,
                                                    int32_t row_vecs) {
    grid_dependency_wait();  // the new rows may come from the previous kernel
    grid_launch_dependents();
    const int b = blockIdx.x;
    const int pos = __ldg(positions + b);
    if (pos < 0 || pos >= max_blocks * block_size) return;
    const int e = __ldg(block_tables + (size_t)b * max_blocks + pos / block_size);
    if (e < 0 || (int64_t)e >= num_blocks) return;
    const size_t dst = ((size_t)e * block_size + pos % block_size) * row_vecs;
    const size_t src = (size_t)b * row_vecs;
    for (int i = threadIdx.x; i < row_vecs; i += blockDim.x) {
        k_cache[dst + i] = __ldg(k_new + src + i);
        v_cache[dst + i] = __ldg(v_new + src + i);
    }
}

// Self-test of the bounded wait: an mbarrier that nothing ever arrives at.
// The wait gives up after `timeout_ns` and records PA_ERR_TIMEOUT, exactly as
// the decode kernels do when their copy pipeline stops delivering.
__global__ void wait_timeout_kernel(int32_t* err, uint64_t timeout_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        mbar_init_fence();
    }
    __syncthreads();
    const bool ok = mbar_wait_bounded(smem_u32(&bar), 0u, timeout_ns);
    if (!ok && threadIdx.x == 0) record_error(err, PA_ERR_TIMEOUT);
}

__global__ void resolve_kernel(int32_t* out_phys, const int32_t* block_tables,
                               const int32_t* context_lens, int32_t batch, int32_t max_blocks,
                               int32_t block_size, int64_t num_blocks) {
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= (int64_t)batch * max_blocks) return;
    const int b = (int)(idx / max_blocks), j = (int)(idx % max_blocks);
    const int T = reachable_tokens(context_lens, b, max_blocks, block_size);
    const int npages = (T + block_size - 1) / block_size;
    out_phys[idx] = page_phys(block_tables + (size_t)b * max_blocks, j, npages, num_blocks);
}

}  // namespace

cudaError_t launch_combine(const CombineParams& p, int head_dim, dim3 grid, bool pdl,
                           cudaStream_t stream) {
    void (*kern)(const CombineParams);
    switch (head_dim) {
        case 64: kern = p.lse ? combine_kernel<64, true> : combine_kernel<64, false>; break;
        case 128: kern = p.lse ? combine_kernel<128, true> : combine_kernel<128, false>; break;
        default: kern = p.lse ? combine_kernel<256, true> : combine_kernel<256, false>; break;
    }
    const uint32_t smem = (uint32_t)p.num_parts * sizeof(float);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_combine_weights(const CombineParams& p, const WeightParams& w, int head_dim,
                                   bool pdl, cudaStream_t stream) {
    void (*kern)(const CombineParams, const WeightParams);
    switch (head_dim) {
        case 64: kern = combine_weights_kernel<64>; break;
        case 128: kern = combine_weights_kernel<128>; break;
        default: kern = combine_weights_kernel<256>; break;
    }
    const uint32_t smem = (uint32_t)p.num_parts * sizeof(float);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t ctas =
        (int64_t)p.q_len * p.num_heads + (int64_t)weight_tiles(w) * p.num_kv_heads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)p.batch);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, w);
}

cudaError_t launch_combine_balanced(const CombineParams& p, int head_dim, dim3 grid, bool pdl,
                                    cudaStream_t stream) {
    void (*kern)(const CombineParams);
    switch (head_dim) {
        case 64: kern = combine_balanced_kernel<64>; break;
        case 128: kern = combine_balanced_kernel<128>; break;
        default: kern = combine_balanced_kernel<256>; break;
    }
    const uint32_t smem = (uint32_t)(p.num_ctas + 1) * sizeof(float);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_prefix_combine(const PrefixCombineParams& p, int head_dim, int batch, bool pdl,
                                  cudaStream_t stream) {
    void (*kern)(const PrefixCombineParams);
    switch (head_dim) {
        case 64: kern = prefix_combine_kernel<64>; break;
        case 128: kern = prefix_combine_kernel<128>; break;
        default: kern = prefix_combine_kernel<256>; break;
    }
    cudaLaunchConfig_t cfg = {};
    const int per_cta = kCombineThreads / 32;  // rows
    cfg.gridDim = dim3((unsigned)((p.q_len * p.num_heads + per_cta - 1) / per_cta), (unsigned)batch);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                          const int32_t* block_tables, const int32_t* positions, int32_t batch,
                          int32_t max_blocks, int32_t block_size, int64_t num_blocks,
                          int32_t row_bytes, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)batch);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, append_kernel, static_cast<uint4*>(k_cache),
                              static_cast<uint4*>(v_cache), static_cast<const uint4*>(k_new),
                              static_cast<const uint4*>(v_new), block_tables, positions,
                              max_blocks, block_size, num_blocks, row_bytes / 16);
}

cudaError_t launch_wait_timeout(int32_t* err, uint64_t timeout_ns, cudaStream_t stream) {
    wait_timeout_kernel<<<1, 32, 0, stream>>>(err, timeout_ns);
    return cudaGetLastError();
}

cudaError_t launch_resolve(int32_t* out_phys, const int32_t* block_tables,
                           const int32_t* context_lens, int32_t batch, int32_t max_blocks,
                           int32_t block_size, int64_t num_blocks, cudaStream_t stream) {
    const int64_t n = (int64_t)batch * max_blocks;
    if (n == 0) return cudaSuccess;
    const int threads = 256;
    const unsigned blocks = (unsigned)((n + threads - 1) / threads);
    resolve_kernel<<<blocks, threads, 0, stream>>>(out_phys, block_tables, context_lens, batch,
                                                   max_blocks, block_size, num_blocks);
    return cudaGetLastError();
}

}  // namespace pa
