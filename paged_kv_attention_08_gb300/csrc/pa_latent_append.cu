// Append to the latent cache (pa_rope_append_latent): each new token's latent
// vector, normalised by its root mean square,
//     y = x / sqrt(mean(x^2) + eps) * w,
// and its positional key part, turned as in pa_rope.cu, go to the token's slot;
// the positional part of every head's query turns into q_out.  One launch: the
// norm, the turn and the store are a few elementary operations an element, the
// call is bound by its bytes (and, for single tokens, by its launch).
//
// A CTA takes `span` consecutive tokens; their sines and cosines are made once
// for the key and all heads.  A warp takes a token's row: 16 elements a lane at
// latent_dim 512, the sum of squares in fp32.
#include "pa_turn.cuh"

namespace pa {

namespace {

constexpr int kLatentAppendThreads = 256;
constexpr int kLatentRope = 64;  // elements of the positional part

template <typename T>
__global__ void __launch_bounds__(kLatentAppendThreads) append_latent_kernel(const LatentAppendParams p) {
    constexpr int OCT = kLatentRope / 16, HALF = kLatentRope / 2;
    extern __shared__ float4 cs[];  // [span][4][OCT]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long tokens = (long long)p.batch * p.q_len;
    const long long t0 = (long long)blockIdx.x * p.span;
    const int n = (int)min((long long)p.span, tokens - t0);

    grid_dependency_wait();
    grid_launch_dependents();

    for (int i = tid; i < n * HALF; i += kLatentAppendThreads) {
        const int t = i / HALF, j = i % HALF;
        *turn_entry(cs, OCT, t, j) = turn_angle(__ldg(p.positions + t0 + t), __ldg(p.phases + j));
    }
    __syncthreads();

    // ---- the cache rows: a warp to a token ----
    const int R = p.latent_dim, W = R + kLatentRope;
    for (int t = warp; t < n; t += kLatentAppendThreads / 32) {
        const long long token = t0 + t;
        const int b = (int)(token / p.q_len), i = (int)(token - (long long)b * p.q_len);
        const long long at = (long long)max(__ldg(p.context_lens + b), 0) - p.q_len + i;
        if (at < 0 || at >= (long long)p.max_blocks * p.block_size) continue;
        const int e = __ldg(p.block_tables + (size_t)b * p.max_blocks + at / p.block_size);
        if (e < 0 || (int64_t)e >= p.num_blocks) continue;
        const T* src = static_cast<const T*>(p.latent_new) + token * p.new_stride;
        T* dst = static_cast<T*>(p.cache) + ((size_t)e * p.block_size + at % p.block_size) * W;
        // lane's vectors of eight: lane, lane + 32 (latent_dim 128: the first 16 lanes)
        uint4 v[2];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if ((lane + k * 32) * 8 < R) {
                v[k] = *reinterpret_cast<const uint4*>(src + (lane + k * 32) * 8);
                const uint32_t a[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x0, x1;
                    Mma<T>::unpack(a[c], x0, x1);
                    sum = fmaf(x0, x0, fmaf(x1, x1, sum));
                }
            }
        }
        if (lane < OCT) {
            const int lo_at = R + (p.interleaved ? lane * 16 : lane * 8);
            const int hi_at = R + (p.interleaved ? lane * 16 + 8 : HALF + lane * 8);
            uint4 lo = *reinterpret_cast<const uint4*>(src + lo_at);
            uint4 hi = *reinterpret_cast<const uint4*>(src + hi_at);
            float x[16];
            widen8<T>(lo, hi, x);
            turn8(x, cs + t * 4 * OCT + lane, OCT, p.interleaved);
            narrow8<T>(x, lo, hi);
            *reinterpret_cast<uint4*>(dst + lo_at) = lo;
            *reinterpret_cast<uint4*>(dst + hi_at) = hi;
        }
        float f = 1.f;
        if (p.norm_weight) {
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
            f = 1.f / sqrtf(sum / (float)R + p.eps);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if ((lane + k * 32) * 8 < R) {
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
    }

    // ---- the queries' positional parts ----
    const int q_items = p.num_heads * OCT;
#pragma unroll 4
    for (int i = tid; i < n * q_items; i += kLatentAppendThreads) {
        const int t = i / q_items, rem = i - t * q_items;
        const int h = rem / OCT, oct = rem % OCT;
        const int lo_at = p.interleaved ? oct * 16 : oct * 8;
        const int hi_at = p.interleaved ? oct * 16 + 8 : HALF + oct * 8;
        const T* src = static_cast<const T*>(p.q) + (t0 + t) * p.q_token_stride + h * p.q_head_stride;
        uint4 lo = *reinterpret_cast<const uint4*>(src + lo_at);
        uint4 hi = *reinterpret_cast<const uint4*>(src + hi_at);
        float x[16];
        widen8<T>(lo, hi, x);
        turn8(x, cs + t * 4 * OCT + oct, OCT, p.interleaved);
        narrow8<T>(x, lo, hi);
        T* dst = static_cast<T*>(p.q_out) + (t0 + t) * p.q_out_token_stride + h * p.q_out_head_stride;
        *reinterpret_cast<uint4*>(dst + lo_at) = lo;
        *reinterpret_cast<uint4*>(dst + hi_at) = hi;
    }
}

}  // namespace

cudaError_t launch_append_latent(LatentAppendParams p, bool bf16, int num_sms, bool pdl,
                                 cudaStream_t stream) {
    const long long tokens = (long long)p.batch * p.q_len;
    // a token to a CTA until the SMs hold several, then up to eight (a warp's row each)
    long long span = tokens / (4ll * num_sms);
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
