// Eviction from the paged cache by accumulated attention weight.
//
// Each kv head of a sequence keeps its own tokens, at most `budget` of them:
// the first `sink` and the last `recent` ones always, then those of the
// largest weights, equal weights by the lowest index.  The kept tokens stay
// in their order and are packed from slot 0 of the new pages on.
//
//   evict_select_kernel  finds the budget's threshold in a row of weights by
//                        radix selection on the order-preserving integer image
//                        of the floats, then lists the kept tokens in order;
//   evict_copy_kernel    moves keys, values and weights of the listed tokens
//                        to other pages, all rows at once;
//   evict_pack_kernel    the same within the same pages.
//
// Bound: memory (the weights are read, each kept row is read and written).
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kSelThreads = 1024;

// Integers that order as the weights do: NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of one int per thread; *total gets the sum.
// `scratch` holds 33 ints; a barrier follows its last read.
__device__ __forceinline__ int block_exclusive(int v, int* scratch, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = lane < (int)(blockDim.x >> 5) ? scratch[lane] : 0;
        const int own = s;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int y = __shfl_up_sync(kFullMask, s, m);
            if (lane >= m) s += y;
        }
        scratch[lane] = s - own;
        if (lane == 31) scratch[32] = s;
    }
    __syncthreads();
    const int r = x - v + scratch[warp];
    *total = scratch[32];
    __syncthreads();
    return r;
}

// One CTA per (kv head, sequence).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
    __shared__ int hist[256];
    __shared__ int scratch[33];
    __shared__ int chosen[2];  // digit of the threshold, tokens still wanted of it
    const int tid = threadIdx.x;
    const int kvh = blockIdx.x, b = blockIdx.y;
    grid_dependency_wait();
    grid_launch_dependents();

    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const float* w = p.weights + ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * p.block_size;
    int32_t* kept = p.kept + ((size_t)b * p.num_kv_heads + kvh) * p.budget;
    const int32_t* row = p.block_tables + (size_t)b * p.max_blocks;
    const int npages = (T + p.block_size - 1) / p.block_size;
    auto held = [&](int t) { return page_phys(row, t / p.block_size, npages, p.num_blocks) >= 0; };
    auto always = [&](int t) { return t < p.sink || t >= T - p.recent; };

    // tokens of readable pages, and those kept whatever their weight
    int mine = 0, forced = 0;
    for (int t = tid; t < T; t += kSelThreads)
        if (held(t)) {
            ++mine;
            forced += always(t);
        }
    int valid, must;
    (void)block_exclusive(mine, scratch, &valid);
    (void)block_exclusive(forced, scratch, &must);
    const int n = min(valid, p.budget);
    int want = n - must;  // to be chosen by weight

    // the largest key of which at least `want` free tokens are as large, digit by digit
    uint32_t prefix = 0, mask = 0;
    const bool all = valid <= p.budget;
    if (!all) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int t = tid; t < T; t += kSelThreads) {
                if (always(t) || !held(t)) continue;
                const uint32_t k = weight_key(w[t]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = want, d = 255;
                for (; d > 0 && hist[d] < left; --d) left -= hist[d];
                chosen[0] = d;
                chosen[1] = left;
            }
            __syncthreads();
            prefix |= (uint32_t)chosen[0] << shift;
            mask |= 255u << shift;
            want = chosen[1];
            __syncthreads();
        }
    }
    // the kept tokens in order; `want` of those equal to the threshold, lowest first
    int at = 0, equals = 0;
    for (int t0 = 0; t0 < T; t0 += kSelThreads) {
        const int t = t0 + tid;
        bool keep = false, equal = false;
        if (t < T && held(t)) {
            keep = all || always(t);
            if (!keep) {
                const uint32_t k = weight_key(w[t]);
                keep = k > prefix;
                equal = k == prefix;
            }
        }
        int total;
        const int rank = equals + block_exclusive(equal, scratch, &total);
        equals += total;
        keep = keep || (equal && rank < want);
        const int j = at + block_exclusive(keep, scratch, &total);
        at += total;
        if (keep) kept[j] = t;
    }
    for (int j = n + tid; j < p.budget; j += kSelThreads) kept[j] = -1;
    if (kvh == 0 && tid == 0) p.new_lens[b] = n;
}

// A row (slot) of the cache, in 16-byte vectors, of token t of a table row;
// -1 where the table has no page for it.
__device__ __forceinline__ long long slot_of(const int32_t* row, int t, int block_size, int max_blocks,
                                             int64_t num_blocks) {
    if (t < 0 || t / block_size >= max_blocks) return -1;
    const int e = __ldg(row + t / block_size);
    if (e < 0 || (int64_t)e >= num_blocks) return -1;
    return (long long)e * block_size + t % block_size;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;  // tokens of one kv head per CTA

// One CTA per (64 tokens of the new row, kv head, sequence).
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p) {
    __shared__ long long src[kCopyRows], dst[kCopyRows];
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int j0 = blockIdx.x * kCopyRows;
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t unit = (size_t)b * p.num_kv_heads + kvh;
    const int vecs = p.head_dim / 8;
    if (tid < kCopyRows) {
        const int j = j0 + tid;
        const int t = j < p.budget ? p.kept[unit * p.budget + j] : -1;
        long long s = -1, d = -1;
        if (t >= 0) {
            s = slot_of(p.block_tables + (size_t)b * p.max_blocks, t, p.block_size, p.max_blocks,
                        p.num_blocks);
            d = slot_of(p.new_block_tables + (size_t)b * p.new_max_blocks, j, p.block_size,
                        p.new_max_blocks, p.num_blocks);
        }
        src[tid] = s;
        dst[tid] = d;
        const size_t width = (size_t)p.max_blocks * p.block_size;
        const size_t new_width = (size_t)p.new_max_blocks * p.block_size;
        if ((size_t)j < new_width)
            p.new_weights[unit * new_width + j] = t >= 0 ? p.weights[unit * width + t] : 0.f;
    }
    __syncthreads();
    const long long row = (long long)p.num_kv_heads * vecs;
    for (int i = tid; i < kCopyRows * 2 * vecs; i += kCopyThreads) {
        const int r = i / (2 * vecs), c = i % (2 * vecs);
        if (src[r] < 0 || dst[r] < 0) continue;
        uint4* cache = static_cast<uint4*>(c < vecs ? p.k_cache : p.v_cache);
        const int at = kvh * vecs + (c < vecs ? c : c - vecs);
        cache[dst[r] * row + at] = cache[src[r] * row + at];
    }
}

constexpr int kPackThreads = 256;
constexpr int kPackRows = kPackThreads / 8;  // rows of 64 columns moved at a time
constexpr int kPackSteps = 8;

// In place: token j of the new row comes from slot kept[j] >= j of the same
// row, so a chunk of rows may be written once all of it has been read, and
// no later chunk reads what it writes.  One CTA per (64 columns of the keys
// or of the values, kv head, sequence) takes the chunks in order; columns
// do not meet, so the CTAs need no order among them.  The first slice's CTA
// packs the weights as well.
__global__ void __launch_bounds__(kPackThreads) evict_pack_kernel(const EvictParams p) {
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int slices = p.head_dim / 64;
    const int slice = blockIdx.x % slices;
    uint4* cache = static_cast<uint4*>((int)blockIdx.x < slices ? p.k_cache : p.v_cache);
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t unit = (size_t)b * p.num_kv_heads + kvh;
    const int32_t* kept = p.kept + unit * p.budget;
    const int32_t* old_row = p.block_tables + (size_t)b * p.max_blocks;
    const int32_t* new_row = p.new_block_tables + (size_t)b * p.new_max_blocks;
    const int n = p.new_lens[b];
    const long long row = (long long)p.num_kv_heads * (p.head_dim / 8);
    const int col = kvh * (p.head_dim / 8) + slice * 8 + (tid & 7);
    for (int j0 = 0; j0 < n; j0 += kPackRows * kPackSteps) {
        uint4 v[kPackSteps];
        long long dst[kPackSteps];
#pragma unroll
        for (int k = 0; k < kPackSteps; ++k) {
            const int j = j0 + k * kPackRows + (tid >> 3);
            dst[k] = -1;
            if (j < n) {
                const long long s = slot_of(old_row, kept[j], p.block_size, p.max_blocks, p.num_blocks);
                const long long d = slot_of(new_row, j, p.block_size, p.new_max_blocks, p.num_blocks);
                if (s >= 0 && d >= 0 && s != d) {
                    dst[k] = d;
                    v[k] = cache[s * row + col];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPackSteps; ++k)
            if (dst[k] >= 0) cache[dst[k] * row + col] = v[k];
    }
    if (blockIdx.x == 0) {
        const float* w = p.weights + unit * p.max_blocks * p.block_size;
        const int new_width = p.new_max_blocks * p.block_size;
        float* nw = p.new_weights + unit * new_width;
        for (int j0 = 0; j0 < n; j0 += kPackThreads) {
            const int j = j0 + tid;
            const float x = j < n ? w[kept[j]] : 0.f;
            __syncthreads();
            if (j < n) nw[j] = x;
        }
        for (int j = n + tid; j < new_width; j += kPackThreads) nw[j] = 0.f;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, bool in_place, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cfg.gridDim = dim3((unsigned)p.num_kv_heads, (unsigned)p.batch);
    cfg.blockDim = dim3(kSelThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    if (e != cudaSuccess) return e;
    if (in_place) {
        cfg.gridDim = dim3((unsigned)(2 * p.head_dim / 64), (unsigned)p.num_kv_heads, (unsigned)p.batch);
        cfg.blockDim = dim3(kPackThreads);
        return cudaLaunchKernelEx(&cfg, evict_pack_kernel, p);
    }
    const int width = max(p.budget, p.new_max_blocks * p.block_size);
    cfg.gridDim = dim3((unsigned)((width + kCopyRows - 1) / kCopyRows), (unsigned)p.num_kv_heads,
                       (unsigned)p.batch);
    cfg.blockDim = dim3(kCopyThreads);
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
}

}  // namespace pa
