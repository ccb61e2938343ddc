// Rotary positions with several axes, joined with the append to the paged
// cache: the new tokens' queries and keys are turned, and the keys and values
// written to the slots that the block tables give them.
//
// Pair j of a head (elements j and j + R/2 of the rotary part, or 2j and
// 2j + 1) turns by the angle pos[axis_j] * f_j:
//     (x, y) -> (x cos a - y sin a, x sin a + y cos a).
// The frequency arrives as a 64-bit fraction of a turn, F_j = f_j / 2 pi *
// 2^64.  pos * F_j, wrapped at 64 bits, is then the angle modulo one turn
// exactly up to F_j's own rounding: a far position loses nothing, where a
// 32-bit product of position and frequency would be off by 0.06 rad at a
// million tokens.  The top 32 bits go to the sine and cosine.
//
// Bound: memory (every element is read once and written once), and close behind
// it instruction issue (61 % of the cycles): an item's places, its products
// and its share of the sines.  A CTA takes a run of the flattened (token, item)
// order, an item being eight pairs (32 bytes) of one head; it issues all of its
// loads, computes each needed (token, pair) sine and cosine once into shared
// memory while they fly, and then turns and stores.  So a token's angles cost
// one evaluation for all of its H + Hkv heads.  24,002 tokens of 16 + 2 x 4 heads
// of 64 (148 MB moved): 30.1 us, 4.9 TB/s; eight tokens of 32 + 2 x 8 heads of 128:
// 2.7 us a launch.
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;

template <typename T>
__device__ __forceinline__ void turn8(uint4& lo, uint4& hi, const float4* cs, int cs_stride,
                                      bool interleaved) {
    uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w};
    uint32_t b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // pairs 2c and 2c + 1 of the eight
        const float4 w = cs[c * cs_stride];  // cos, sin, cos, sin
        float x0, x1, y0, y1;
        if (interleaved) {  // words 2c and 2c + 1 of the 16 elements
            uint32_t& u = c < 2 ? a[2 * c] : b[2 * c - 4];
            uint32_t& v = c < 2 ? a[2 * c + 1] : b[2 * c - 3];
            Mma<T>::unpack(u, x0, y0);
            Mma<T>::unpack(v, x1, y1);
            u = Mma<T>::pack(x0 * w.x - y0 * w.y, x0 * w.y + y0 * w.x);
            v = Mma<T>::pack(x1 * w.z - y1 * w.w, x1 * w.w + y1 * w.z);
        } else {
            Mma<T>::unpack(a[c], x0, x1);
            Mma<T>::unpack(b[c], y0, y1);
            a[c] = Mma<T>::pack(x0 * w.x - y0 * w.y, x1 * w.z - y1 * w.w);
            b[c] = Mma<T>::pack(x0 * w.y + y0 * w.x, x1 * w.w + y1 * w.z);
        }
    }
    lo = make_uint4(a[0], a[1], a[2], a[3]);
    hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// IPT: items per thread (1 spreads a decode step's few tokens over the SMs).
//
// Four CTAs to an SM: with the item's place kept in registers instead of found
// again after the barrier, and four items to a thread, only two fitted (92
// registers), and 24,002 tokens of 24 heads took 37.6 us.
template <typename T, int IPT>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(const RopeParams p) {
    extern __shared__ float4 cs[];  // [tokens of the CTA][4][pair octets] (cos, sin) x 2
    const int tid = threadIdx.x;
    const int per_head = p.head_dim / 16;                    // items of a head
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    const int per_token = heads * per_head;
    const int octets = p.rotary_dim / 16;                    // rotated items of a head
    long long* slot_of = reinterpret_cast<long long*>(cs + p.max_cta_tokens * 4 * octets);

    const long long tokens = (long long)p.batch * p.q_len;
    const long long first = (long long)blockIdx.x * (kRopeThreads * IPT);
    const long long t0 = first < (1ll << 31) ? (int)first / per_token  // the CTA's first token
                                             : first / per_token;
    const int skip = (int)(first - t0 * per_token);
    int ntok = (skip + kRopeThreads * IPT + per_token - 1) / per_token;
    if (ntok > tokens - t0) ntok = (int)(tokens - t0);

    grid_dependency_wait();
    grid_launch_dependents();

    // token of the CTA, head and octet of its item number i (below per_token + 512):
    // a head has a power of two of items; a token's are divided by as a product
    const int hshift = __ffs(per_head) - 1;
    auto place = [&](int k, int& tok, int& head, int& oct) {
        const int i = skip + tid + k * kRopeThreads;
        tok = per_token >= 512 ? (i >= per_token) : (int)__umulhi((uint32_t)i, p.per_token_inverse);
        const int rem = i - tok * per_token;
        head = rem >> hshift;
        oct = rem & (per_head - 1);
    };

    uint4 lo[IPT], hi[IPT];
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        int tok, h, oct;
        place(k, tok, h, oct);
        if (tok >= ntok) continue;
        // the two 8-element vectors of the item: both halves of the rotary
        // part, or 16 neighbours (interleaved pairs, the untouched rest, values)
        const T* src;
        bool turned = oct < octets;
        if (h < p.num_heads) {
            src = static_cast<const T*>(p.q) + (t0 + tok) * p.q_stride;
        } else if (h < p.num_heads + p.num_kv_heads) {
            h -= p.num_heads;
            src = static_cast<const T*>(p.k_new) + (t0 + tok) * p.k_stride;
        } else {
            h -= p.num_heads + p.num_kv_heads;
            turned = false;
            src = static_cast<const T*>(p.v_new) + (t0 + tok) * p.v_stride;
        }
        const bool split = turned && !p.interleaved;
        src += h * p.head_dim + (split ? oct * 8 : oct * 16);
        lo[k] = *reinterpret_cast<const uint4*>(src);
        hi[k] = *reinterpret_cast<const uint4*>(src + (split ? p.rotary_dim / 2 : 8));
    }

    // where each token's keys and values go (-1: nowhere)
    for (int t = tid; t < ntok; t += kRopeThreads) {
        const long long token = t0 + t;
        const int b = (int)(token / p.q_len), i = (int)(token - (long long)b * p.q_len);
        const long long at = (long long)max(__ldg(p.context_lens + b), 0) - p.q_len + i;
        long long slot = -1;
        if (at >= 0 && at < (long long)p.max_blocks * p.block_size) {
            const int e = __ldg(p.block_tables + (size_t)b * p.max_blocks + at / p.block_size);
            if (e >= 0 && (int64_t)e < p.num_blocks)
                slot = (long long)e * p.block_size + at % p.block_size;
        }
        slot_of[t] = slot;
    }
    // the sines and cosines of the CTA's tokens
    const int half = p.rotary_dim / 2;
    for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int t = i / half, j = i - t * half;
        const int ax = __ldg(p.axes + j);
        float s = 0.f, c = 1.f;
        if (ax >= 0 && ax < p.num_axes) {
            const long long pos = __ldg(p.positions + (size_t)ax * tokens + t0 + t);
            const unsigned long long turn =
                (unsigned long long)pos * (unsigned long long)__ldg(p.phases + j);
            // the signed top 32 bits: a fraction of half a turn in [-1, 1)
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        }
        float2* at = reinterpret_cast<float2*>(cs + (t * 4 + ((j >> 1) & 3)) * octets + (j >> 3));
        at[j & 1] = make_float2(c, s);
    }
    __syncthreads();

#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        int tok, h, oct;
        place(k, tok, h, oct);
        if (tok >= ntok) continue;
        const bool is_q = h < p.num_heads, is_k = !is_q && h < p.num_heads + p.num_kv_heads;
        const bool turned = oct < octets && (is_q || is_k);
        if (turned)
            turn8<T>(lo[k], hi[k], cs + tok * 4 * octets + oct, octets, p.interleaved);
        T* dst;
        if (is_q) {
            dst = static_cast<T*>(p.q_out) + (t0 + tok) * p.q_out_stride;
        } else {
            const long long slot = slot_of[tok];
            if (slot < 0) continue;
            h -= is_k ? p.num_heads : p.num_heads + p.num_kv_heads;
            dst = static_cast<T*>(is_k ? p.k_cache : p.v_cache) +
                  slot * ((long long)p.num_kv_heads * p.head_dim);
        }
        const bool split = turned && !p.interleaved;
        dst += h * p.head_dim + (split ? oct * 8 : oct * 16);
        *reinterpret_cast<uint4*>(dst) = lo[k];
        *reinterpret_cast<uint4*>(dst + (split ? p.rotary_dim / 2 : 8)) = hi[k];
    }
}

template <typename T, int IPT>
cudaError_t launch_inst(RopeParams p, long long items, int per_token, bool pdl,
                        cudaStream_t stream) {
    const int span = kRopeThreads * IPT;
    // floor(i / per_token) = (i * inverse) >> 32 for i < 1024 and per_token < 512
    p.per_token_inverse = (uint32_t)((0x100000000ull + per_token - 1) / per_token);
    p.max_cta_tokens = (span + per_token - 2) / per_token + 1;
    // at most (512 / (3 D / 16) + 2) tokens of D / 2 pairs: 13 KB
    const size_t smem = (size_t)p.max_cta_tokens * (p.rotary_dim / 16 * 4 * sizeof(float4) + 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items + span - 1) / span));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<T, IPT>, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool bf16, int num_sms, bool pdl,
                               cudaStream_t stream) {
    const int per_token = (p.num_heads + 2 * p.num_kv_heads) * (p.head_dim / 16);
    const long long items = (long long)p.batch * p.q_len * per_token;
    const bool wide = items > (long long)num_sms * kRopeThreads * 4;  // more than a wave of one each
    if (bf16)
        return wide ? launch_inst<__nv_bfloat16, 2>(p, items, per_token, pdl, stream)
                    : launch_inst<__nv_bfloat16, 1>(p, items, per_token, pdl, stream);
    return wide ? launch_inst<__half, 2>(p, items, per_token, pdl, stream)
                : launch_inst<__half, 1>(p, items, per_token, pdl, stream);
}

}  // namespace pa
