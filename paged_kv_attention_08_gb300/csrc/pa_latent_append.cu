// Append to the latent cache (pa_rope_append_latent): each new token's latent
// vector, normalised by its root mean square,
//     y = x / sqrt(mean(x^2) + eps) * w,
// and its positional key part, turned as in pa_rope.cu, go to the token's slot;
// the positional part of every head's query turns into q_out.  One launch: the
// norm, the turn and the store are a few elementary operations an element, the
// call is bound by its bytes: 16,002 tokens of 32 heads (168 MB, the heads' parts in
// pieces of 128 bytes): 36 us, 4.7 TB/s; and, for single tokens, by its launch (3.3 us).
//
// A CTA takes `span` consecutive tokens; their sines and cosines are made once
// for the key and all heads.  A warp takes a token's row: 16 elements a lane at
// latent_dim 512, the sum of squares in fp32.
#include "pa_turn.cuh"

namespace pa {

namespace {

constexpr int kLatentAppendThreads = 256;
constexpr int kAhead = 4;  // query items that a thread loads ahead
constexpr int kLatentRope = 64;  // elements of the positional part

// Every load is issued before the sines are made: a thread's items of the queries
// (kAhead of them, the rest behind), and a warp's token row.
template <typename T>
__global__ void __launch_bounds__(kLatentAppendThreads, 3) append_latent_kernel(const LatentAppendParams p) {
    constexpr int OCT = kLatentRope / 16, HALF = kLatentRope / 2;
    extern __shared__ float4 cs[];  // [span][4][OCT]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long tokens = (long long)p.batch * p.q_len;
    const long long t0 = (long long)blockIdx.x * p.span;
    const int n = (int)min((long long)p.span, tokens - t0);
    const int lo_of = p.interleaved ? 16 : 8, hi_off = p.interleaved ? 8 : HALF;  // an item's two vectors

    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the queries' positional parts: items of eight pairs ----
    const int q_items = p.num_heads * OCT, total = n * q_items;
    auto q_at = [&](int i, int& t, int& oct, int64_t token_stride, int64_t head_stride) -> int64_t {
        t = i / q_items;
        const int rem = i - t * q_items;
        oct = rem % OCT;
        return (t0 + t) * token_stride + (rem / OCT) * head_stride + oct * lo_of;
    };
    uint4 lo[kAhead], hi[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = tid + k * kLatentAppendThreads;
        if (i < total) {
            int t, oct;
            const T* src = static_cast<const T*>(p.q) + q_at(i, t, oct, p.q_token_stride, p.q_head_stride);
            lo[k] = *reinterpret_cast<const uint4*>(src);
            hi[k] = *reinterpret_cast<const uint4*>(src + hi_off);
        }
    }
    // ---- the cache rows: a warp to a token ----
    const int R = p.latent_dim, W = R + kLatentRope;
    T* dst = nullptr;
    uint4 v[2], klo, khi;
    if (warp < n) {
        const long long token = t0 + warp;
        const int b = (int)(token / p.q_len), i = (int)(token - (long long)b * p.q_len);
        const long long at = (long long)max(__ldg(p.context_lens + b), 0) - p.q_len + i;
        const T* src = static_cast<const T*>(p.latent_new) + token * p.new_stride;
        // lane's vectors of eight: lane, lane + 32 (latent_dim 128: the first 16 lanes)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = (lane + k * 32) * 8 < R ? *reinterpret_cast<const uint4*>(src + (lane + k * 32) * 8)
                                           : make_uint4(0, 0, 0, 0);
        if (lane < OCT) {
            klo = *reinterpret_cast<const uint4*>(src + R + lane * lo_of);
            khi = *reinterpret_cast<const uint4*>(src + R + lane * lo_of + hi_off);
        }
        if (at >= 0 && at < (long long)p.max_blocks * p.block_size) {
            const int e = __ldg(p.block_tables + (size_t)b * p.max_blocks + at / p.block_size);
            if (e >= 0 && (int64_t)e < p.num_blocks)
                dst = static_cast<T*>(p.cache) + ((size_t)e * p.block_size + at % p.block_size) * W;
        }
    }

    for (int i = tid; i < n * HALF; i += kLatentAppendThreads) {
        const int t = i / HALF, j = i % HALF;
        *turn_entry(cs, OCT, t, j) = turn_angle(__ldg(p.positions + t0 + t), __ldg(p.phases + j));
    }
    __syncthreads();

    if (dst) {
        if (lane < OCT) {
            float x[16];
            widen8<T>(klo, khi, x);
            turn8(x, cs + warp * 4 * OCT + lane, OCT, p.interleaved);
            narrow8<T>(x, klo, khi);
            *reinterpret_cast<uint4*>(dst + R + lane * lo_of) = klo;
            *reinterpret_cast<uint4*>(dst + R + lane * lo_of + hi_off) = khi;
        }
        float f = 1.f;
        if (p.norm_weight) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x0, x1;
                    Mma<T>::unpack(a[c], x0, x1);
                    sum = fmaf(x0, x0, fmaf(x1, x1, sum));
                }
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
            f = 1.f / sqrtf(sum / (float)R + p.eps);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if ((lane + k * 32) * 8 >= R) continue;
            if (p.norm_weight) {
                const uint4 g = *reinterpret_cast<const uint4*>(
                    static_cast<const T*>(p.norm_weight) + (lane + k * 32) * 8);
                const uint32_t a[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                const uint32_t w[4] = {g.x, g.y, g.z, g.w};
                uint32_t y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x0, x1, w0, w1;
                    Mma<T>::unpack(a[c], x0, x1);
                    Mma<T>::unpack(w[c], w0, w1);
                    y[c] = Mma<T>::pack(x0 * f * w0, x1 * f * w1);
                }
                v[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
            *reinterpret_cast<uint4*>(dst + (lane + k * 32) * 8) = v[k];
        }
    }

    auto finish = [&](int i, uint4& a, uint4& b) {
        int t, oct;
        T* out = static_cast<T*>(p.q_out) + q_at(i, t, oct, p.q_out_token_stride, p.q_out_head_stride);
        float x[16];
        widen8<T>(a, b, x);
        turn8(x, cs + t * 4 * OCT + oct, OCT, p.interleaved);
        narrow8<T>(x, a, b);
        *reinterpret_cast<uint4*>(out) = a;
        *reinterpret_cast<uint4*>(out + hi_off) = b;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (tid + k * kLatentAppendThreads < total) finish(tid + k * kLatentAppendThreads, lo[k], hi[k]);
    for (int i = tid + kAhead * kLatentAppendThreads; i < total; i += kLatentAppendThreads) {
        int t, oct;
        const T* src = static_cast<const T*>(p.q) + q_at(i, t, oct, p.q_token_stride, p.q_head_stride);
        uint4 a = *reinterpret_cast<const uint4*>(src), b = *reinterpret_cast<const uint4*>(src + hi_off);
        finish(i, a, b);
    }
}

}  // namespace

cudaError_t launch_append_latent(LatentAppendParams p, bool bf16, int num_sms, bool pdl,
                                 cudaStream_t stream) {
    const long long tokens = (long long)p.batch * p.q_len;
    // a token to a CTA until the SMs hold several, then up to eight (a warp's row
    // each), fewer where the heads' items then pass what the threads load ahead
    long long span = tokens / (4ll * num_sms);
    const int most = kAhead * kLatentAppendThreads / (p.num_heads * (kLatentRope / 16));
    if (span > most) span = most;
    p.span = (int)(span < 1 ? 1 : span > 8 ? 8 : span);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tokens + p.span - 1) / p.span));
    cfg.blockDim = dim3(kLatentAppendThreads);
    cfg.dynamicSmemBytes = (size_t)p.span * (kLatentRope / 2) * 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return bf16 ? cudaLaunchKernelEx(&cfg, append_latent_kernel<__nv_bfloat16>, p)
                : cudaLaunchKernelEx(&cfg, append_latent_kernel<__half>, p);
}

}  // namespace pa
