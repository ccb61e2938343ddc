// Rotary positions and the append to the 8-bit cache (pa_rope_append_kv8).
//
// The new tokens' queries and keys turn as in pa_rope.cu.  The turned keys and
// the values, in fp32, go to e4m3 codes on the scale of their page and kv head:
//     s_new = the smallest power of two that brings the new tokens' largest
//             finite magnitude in the page to 448 or below,
//     s     = s_new where the call begins the page, else max(s_old, s_new),
// and where s is above s_old the page's older tokens move to the new scale.  A
// power of two changes a code's exponent and nothing else: the older tokens
// lose nothing but what falls under e4m3's smallest normal number (2^-6, of
// 448), however often the scale rises.  A scale for the magnitude itself would
// round them anew each time.
//
// One CTA takes a sequence's new tokens of one page: its tokens' sines and
// cosines are made once for all heads, a warp takes all tokens of one kv head's
// keys or values, finds their largest magnitude and reads them a second time
// (from L1 or L2) to write them.  So nothing is shared between CTAs and no
// scale is written by two.
//
// Bound: memory.  16,004 tokens of 32 + 2 x 8 heads of 128 (361 MB): 73 us, 4.9 TB/s,
// as the 16-bit append reaches; eight tokens: 5 us a launch.  Loading more of a
// thread's queries ahead costs the warps that hide the rest (74 to 105 us).
#include "pa_kv8.cuh"
#include "pa_turn.cuh"

namespace pa {

namespace {

constexpr int kAppend8Threads = 256;

template <typename T>
__global__ void __launch_bounds__(kAppend8Threads) append8_kernel(const Append8Params p) {
    extern __shared__ float4 cs[];  // [tokens of the CTA][4][octets]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int BS = p.block_size, D = p.head_dim, Q = p.q_len;
    const int per_head = D / 16, octets = p.rotary_dim / 16, half = p.rotary_dim / 2;
    const int b = blockIdx.y;

    grid_dependency_wait();
    grid_launch_dependents();

    // The CTA's tokens: those of the call at positions [page * BS, page * BS + BS).
    // Positions before 0 (padding) form pages of their own, which are not stored.
    const long long start = (long long)max(__ldg(p.context_lens + b), 0) - Q;  // token 0's position
    const long long page = (start >= 0 ? start / BS : -((-start + BS - 1) / BS)) + blockIdx.x;
    const int i0 = (int)max(page * BS - start, 0ll);
    const int i1 = (int)min(page * BS + BS - start, (long long)Q);
    if (i0 >= i1) return;
    const int n = i1 - i0;
    const long long t0 = (long long)b * Q + i0;          // first token of the flattened order
    const int slot0 = (int)(start + i0 - page * BS);     // its slot in the page
    int phys = -1;
    if (page >= 0 && page < p.max_blocks) {
        phys = __ldg(p.block_tables + (size_t)b * p.max_blocks + page);
        if (phys < 0 || (int64_t)phys >= p.num_blocks) phys = -1;
    }

    const long long tokens = (long long)p.batch * Q;
    for (int i = tid; i < n * half; i += kAppend8Threads) {
        const int t = i / half, j = i - t * half;
        const int ax = __ldg(p.axes + j);
        float2 w = make_float2(1.f, 0.f);
        if (ax >= 0 && ax < p.num_axes)
            w = turn_angle(__ldg(p.positions + (size_t)ax * tokens + t0 + t), __ldg(p.phases + j));
        *turn_entry(cs, octets, t, j) = w;
    }
    __syncthreads();

    // ---- the keys and values: one (kv head, K or V) to a warp at a time ----
    if (phys >= 0) {
        const int rows = 32 / per_head;                  // tokens of a warp's step
        const int sub = lane / per_head, oct = lane % per_head;
        const size_t token_codes = (size_t)p.num_kv_heads * D;
        for (int task = warp; task < 2 * p.num_kv_heads; task += kAppend8Threads / 32) {
            const bool is_k = task < p.num_kv_heads;
            const int h = is_k ? task : task - p.num_kv_heads;
            const T* src = static_cast<const T*>(is_k ? p.k_new : p.v_new) + h * D;
            const int64_t stride = is_k ? p.k_stride : p.v_stride;
            uint8_t* codes = (is_k ? p.k_cache : p.v_cache) + (size_t)phys * BS * token_codes +
                             (size_t)h * D;
            float* scale = (is_k ? p.k_scales : p.v_scales) + (size_t)phys * p.num_kv_heads + h;
            const float s_old = slot0 > 0 ? *scale : 0.f;
            const bool turned = is_k && oct < octets;
            const bool split = turned && !p.interleaved;
            const int lo_at = split ? oct * 8 : oct * 16, hi_at = split ? half + oct * 8 : oct * 16 + 8;
            auto load = [&](int t, float (&x)[16]) {
                const T* row = src + (t0 + t) * stride;
                const uint4 lo = *reinterpret_cast<const uint4*>(row + lo_at);
                const uint4 hi = *reinterpret_cast<const uint4*>(row + hi_at);
                widen8<T>(lo, hi, x);
                if (turned) turn8(x, cs + t * 4 * octets + oct, octets, p.interleaved);
            };
            float amax = 0.f;
#pragma unroll 4
            for (int t = sub; t < n; t += rows) {
                float x[16];
                load(t, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float a = fabsf(x[e]);
                    amax = a < INFINITY ? fmaxf(amax, a) : amax;
                }
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, m));
            const float s = fmaxf(s_old, scale_for(amax));
            const float inv = 1.f / s;                   // (exact for powers of two)
            __syncwarp();                                // every lane has read the old scale
            if (lane == 0) *scale = s;
            if (slot0 > 0 && s > s_old) {
                const float ratio = s_old * inv;
                for (int t = sub; t < slot0; t += rows) {
                    uint4* at = reinterpret_cast<uint4*>(codes + (size_t)t * token_codes + oct * 16);
                    const uint4 v = *at;
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x0, x1, x2, x3;
                        Mma<__half>::unpack(decode2((uint16_t)w[i]), x0, x1);
                        Mma<__half>::unpack(decode2((uint16_t)(w[i] >> 16)), x2, x3);
                        w[i] = encode2(x0 * ratio, x1 * ratio) |
                               (encode2(x2 * ratio, x3 * ratio) << 16);
                    }
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
#pragma unroll 2
            for (int t = sub; t < n; t += rows) {
                float x[16];
                load(t, x);
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = encode2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                           (encode2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
                uint8_t* dst = codes + (size_t)(slot0 + t) * token_codes;
                *reinterpret_cast<uint2*>(dst + lo_at) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(dst + hi_at) = make_uint2(w[2], w[3]);
            }
        }
    }

    // ---- the queries ----
    const int q_items = p.num_heads * per_head;
#pragma unroll 4
    for (int i = tid; i < n * q_items; i += kAppend8Threads) {
        const int t = i / q_items, rem = i - t * q_items;
        const int h = rem / per_head, oct = rem - h * per_head;
        const bool turned = oct < octets, split = turned && !p.interleaved;
        const int lo_at = h * D + (split ? oct * 8 : oct * 16);
        const int hi_at = h * D + (split ? half + oct * 8 : oct * 16 + 8);
        const T* src = static_cast<const T*>(p.q) + (t0 + t) * p.q_stride;
        uint4 lo = *reinterpret_cast<const uint4*>(src + lo_at);
        uint4 hi = *reinterpret_cast<const uint4*>(src + hi_at);
        if (turned) {
            float x[16];
            widen8<T>(lo, hi, x);
            turn8(x, cs + t * 4 * octets + oct, octets, p.interleaved);
            narrow8<T>(x, lo, hi);
        }
        T* dst = static_cast<T*>(p.q_out) + (t0 + t) * p.q_out_stride;
        *reinterpret_cast<uint4*>(dst + lo_at) = lo;
        *reinterpret_cast<uint4*>(dst + hi_at) = hi;
    }
}

}  // namespace

cudaError_t launch_append8(const Append8Params& p, bool bf16, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // pages that q_len tokens can touch
    cfg.gridDim = dim3((unsigned)((p.q_len + p.block_size - 2) / p.block_size + 1), (unsigned)p.batch);
    cfg.blockDim = dim3(kAppend8Threads);
    // at most 32 tokens of 128 pairs: 32 KB
    cfg.dynamicSmemBytes = (size_t)p.block_size * (p.rotary_dim / 2) * 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return bf16 ? cudaLaunchKernelEx(&cfg, append8_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, append8_kernel<__half>, p);
}

}  // namespace pa
