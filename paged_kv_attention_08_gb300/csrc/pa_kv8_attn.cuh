// Attention over the 8-bit cache: one CTA per (sequence, kv head and chunk of up
// to 16 query rows, partition of the sequence's pages).
//
// The mathematics: with codes k8, v8 and the page's scales sk, sv,
//     s_t = scale * sk (q . k8_t),      out = sum_t 2^(s_t) sv v8_t / sum_t 2^(s_t)
// (s in base-2 units).  The value's scale goes into the weight's exponent,
//     w_t = 2^(s_t + log2 sv - m),  m the running maximum of s_t + log2 sv,
//     acc = sum_t w_t v8_t,         l = sum over pages of (1 / sv) sum_t w_t,
// so that a weight is as large as its token's share of the output can be: a page
// of tiny values keeps its precision where its tokens have all the weight, and
// no page's values are ever multiplied.
//
// What bounds it: memory; two bytes a head_dim element against the 16-bit
// cache's four, so the issue slots a byte count double.  The MMAs are warp-level
// m16n8k16 in fp16, to which e4m3 widens exactly (cvt.f16x2.e4m3x2, two codes
// an instruction); with at most 16 rows a tcgen05 tile would be 7/8 empty
// and its operands would have to go through shared memory a second time.
// Nothing is transposed or shuffled: a lane loads 16 consecutive codes of a
// token's key, and the products' k order, and the output's column order, are
// permuted to what the lanes hold (the queries are loaded in that order).
// Values go two tokens at a time through a byte permutation (prmt), four
// elements of each to a pair of registers that the conversion turns into the B
// operand.
// Weights are split into two fp16 parts, 2^kHalfLift up (pa_internal.h); the
// queries are brought to fp16 exactly, each row scaled by a power of two to
// below 2^15 (elements 2^-28 and less of the row's largest begin to round).
#pragma once

#include <type_traits>

#include "pa_kv8.cuh"

namespace pa {

template <int D, int BS>
struct Kv8Cfg {
    static constexpr int NW = 4;                    // warps
    static constexpr int DS = D == 256 ? 2 : 1;     // warps that split a page's output columns
    static constexpr int NT = NW / DS;              // token streams (page rings)
    static constexpr int DW = D / DS;               // output columns of a warp
    static constexpr int KSTEPS = D / 16;
    static constexpr int ONT = DW / 8;              // output n-tiles of a warp
    static constexpr int ROW = D < 128 ? D : 128;   // bytes of a row of a column block
    static constexpr int BLK = D / ROW;             // column blocks
    static constexpr uint32_t TILE = BS * D;        // bytes of a page's keys of one head
    static constexpr int CTAS = D == 256 ? 2 : 3;   // per SM
    static constexpr int NS_RAW = (int)((CTAS == 3 ? 72u : 104u) * 1024u / (NT * 2 * TILE));
    static constexpr int NS = NS_RAW > 8 ? 8 : NS_RAW;  // stages of a ring
    static constexpr uint32_t STAGES = NT * NS * 2 * TILE;
    static constexpr uint32_t SMEM = STAGES + 2 * 8 * NT * NS + 4 * NT * NS + kSmemAlignSlack;
};

// Byte offset of the 16-byte chunk c of row t in a column block as TMA writes
// it: rows of 128 bytes with the 128-byte swizzle, of 64 with the 64-byte one.
template <int ROW>
__device__ __forceinline__ uint32_t chunk8(int t, int c) {
    return ROW == 128 ? (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4))
                      : (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

template <int D, int BS, typename T>
__global__ void __launch_bounds__(128, Kv8Cfg<D, BS>::CTAS)
    kv8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
               const Kv8Params p) {
    using C = Kv8Cfg<D, BS>;
    constexpr int DS = C::DS, NT = C::NT, NS = C::NS, KSTEPS = C::KSTEPS, ONT = C::ONT, DW = C::DW;
    constexpr float NEG_INF = -INFINITY;
    constexpr float kSlack = 8.f;  // log2 units that weights may stand above 2^kHalfLift

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlignSlack - 1)) & ~uintptr_t(kSmemAlignSlack - 1));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES);
    uint64_t* empty = full + NT * NS;
    int32_t* phys_of = reinterpret_cast<int32_t*>(empty + NT * NS);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stream = warp / DS, ds = warp % DS;
    const int g = lane >> 2, tig = lane & 3;
    const int G = p.group, Hkv = p.num_kv_heads, Q = p.q_len;
    const int part = blockIdx.x, b = blockIdx.z;
    const int kvh = (int)blockIdx.y % Hkv, qi0 = (int)blockIdx.y / Hkv * p.q_chunk;
    const int R = min(p.q_chunk, Q - qi0) * G;

    if (tid == 0) {
        for (int i = 0; i < NT * NS; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), DS);
        }
        mbar_init_fence();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    const int ctx = max(__ldg(p.context_lens + b), 0);
    const int reach = min(min(ctx, p.max_blocks * BS), p.token_limit);  // tokens of the call
    const int pb = part * p.part_pages;
    const int pe = min(pb + p.part_pages, (reach + BS - 1) / BS);
    auto row_off = [&](int r) -> size_t {
        return (((size_t)b * Q + qi0 + r / G) * p.num_heads + kvh * G + r % G) * D;
    };
    if (pb >= pe && p.cluster <= 1) {
        if (p.num_parts <= 1)
            for (int i = tid; i < R * D; i += 128) store_out(p.out, row_off(i / D) + i % D, 0.f, p.out_dtype);
        return;  // (the join does not read partitions past the context)
    }

    // ---- the stream's pages: pb + stream, + NT, ...; each warp keeps 32 table
    // entries ahead, one a lane, and the scales of the pages that it consumes ----
    const int n_s = pe - pb > stream ? (pe - pb - stream + NT - 1) / NT : 0;
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks;
    auto fetch = [&](int chunk) -> int {
        const int j = pb + stream + (chunk * 32 + lane) * NT;
        const int e = j < pe ? __ldg(table + j) : -1;
        return e >= 0 && (int64_t)e < p.num_blocks ? e : -1;
    };
    float sk_ahead = 0.f, sv_ahead = 1.f;
    auto fetch_scales = [&](int e) {
        sk_ahead = e >= 0 ? __ldg(p.k_scales + (size_t)e * Hkv + kvh) : 0.f;
        sv_ahead = e >= 0 ? __ldg(p.v_scales + (size_t)e * Hkv + kvh) : 1.f;
    };
    int ent = fetch(0), ent_next = fetch(1);
    __syncthreads();  // barriers initialised
    // Whole warp: entry of local page i, and (the stream's first warp) its copies.
    auto issue = [&](int i) {
        if (i > 0 && (i & 31) == 0) {
            ent = ent_next;
            ent_next = fetch((i >> 5) + 1);
            fetch_scales(ent);  // (consumed from page i on, NS pages later)
        }
        const int e = __shfl_sync(kFullMask, ent, i & 31);
        if (ds == 0 && lane == 0) {
            const int sidx = stream * NS + i % NS;
            const uint32_t bar = smem_u32(full + sidx);
            phys_of[sidx] = e;
            if (e >= 0) {
                const uint64_t policy = l2_policy_evict_first();
                mbar_arrive_expect_tx(bar, 2 * C::TILE);
                const uint32_t dst = smem_u32(smem) + (uint32_t)sidx * 2 * C::TILE;
#pragma unroll
                for (int blk = 0; blk < C::BLK; ++blk) {
                    tma_load_4d(dst + blk * BS * C::ROW, &tmap_k, blk * C::ROW, kvh, 0, e, bar, policy);
                    tma_load_4d(dst + C::TILE + blk * BS * C::ROW, &tmap_v, blk * C::ROW, kvh, 0, e, bar,
                                policy);
                }
            } else {
                mbar_arrive(bar);
            }
        }
    };
    for (int i = 0; i < min(n_s, NS); ++i) issue(i);
    fetch_scales(ent);

    // ---- the queries, A operand of S = Q K^T: element order of a lane's keys,
    // rows g and g + 8, each scaled by a power of two ----
    const bool real0 = g < R, real1 = g + 8 < R;
    uint32_t qa[KSTEPS][4];
    float qk0, qk1;  // scale * log2(e), and the rows' powers of two taken out again
    {
        const T* q0 = static_cast<const T*>(p.q) + (real0 ? row_off(g) : row_off(0));
        const T* q1 = static_cast<const T*>(p.q) + (real1 ? row_off(g + 8) : row_off(0));
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) {
            const int d = k / (C::ROW / 16) * C::ROW + tig * (C::ROW / 4) + k % (C::ROW / 16) * 4;
            const uint2 x = real0 ? __ldg(reinterpret_cast<const uint2*>(q0 + d)) : make_uint2(0, 0);
            const uint2 y = real1 ? __ldg(reinterpret_cast<const uint2*>(q1 + d)) : make_uint2(0, 0);
            qa[k][0] = x.x, qa[k][2] = x.y, qa[k][1] = y.x, qa[k][3] = y.y;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float a, c;
                Mma<T>::unpack(qa[k][r], a, c);
                float& m = r & 1 ? m1 : m0;
                m = fmaxf(m, fmaxf(fabsf(a), fabsf(c)));
            }
        }
#pragma unroll
        for (int x = 1; x <= 2; x <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(kFullMask, m0, x));
            m1 = fmaxf(m1, __shfl_xor_sync(kFullMask, m1, x));
        }
        // 2^14 <= f * m < 2^15 (rows of less than 2^-112: f = 2^126)
        auto power = [](float m) { return min(141 + 127 - (int)(__float_as_uint(m) >> 23), 253); };
        const int e0 = max(power(m0), 1), e1 = max(power(m1), 1);
        const float f0 = __uint_as_float((uint32_t)e0 << 23), f1 = __uint_as_float((uint32_t)e1 << 23);
        qk0 = p.qscale * __uint_as_float((uint32_t)(254 - e0) << 23);
        qk1 = p.qscale * __uint_as_float((uint32_t)(254 - e1) << 23);
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float a, c;
                Mma<T>::unpack(qa[k][r], a, c);
                const float f = r & 1 ? f1 : f0;
                qa[k][r] = Mma<__half>::pack(a * f, c * f);
            }
    }
    // Tokens that a row attends to: its query token's causal limit.
    const int lim0 = min(reach, ctx - Q + qi0 + g / G + 1);
    const int lim1 = min(reach, ctx - Q + qi0 + (g + 8) / G + 1);
    const int lim_least = min(reach, ctx - Q + qi0 + 1);  // the first row's

    float m0 = real0 ? NEG_INF : 0.f, m1 = real1 ? NEG_INF : 0.f, l0 = 0.f, l1 = 0.f;
    float acc[ONT][4];
#pragma unroll
    for (int n = 0; n < ONT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

    float sk = 0.f, sv = 1.f;
    bool aborted = false;
    int issued = min(n_s, NS);
    for (int i = 0; i < n_s; ++i) {
        if ((i & 31) == 0) sk = sk_ahead, sv = sv_ahead;
        const int sidx = stream * NS + i % NS;
        if (!__all_sync(kFullMask, mbar_wait_bounded(smem_u32(full + sidx), (i / NS) & 1, p.timeout_ns))) {
            if (lane == 0) record_error(p.err, PA_ERR_TIMEOUT);
            aborted = true;
        }
        const float page_sk = __shfl_sync(kFullMask, sk, i & 31);
        const float page_sv = __shfl_sync(kFullMask, sv, i & 31);
        if (!aborted && phys_of[sidx] >= 0) {
            const int first = (pb + stream + i * NT) * BS;
            const int nvalid = reach - first;
            const uint32_t kt = smem_u32(smem) + (uint32_t)sidx * 2 * C::TILE, vt = kt + C::TILE;

            // ---- S = Q K^T: even and odd k-steps in chains of their own ----
            float s[BS / 8][4];
#pragma unroll
            for (int nt = 0; nt < BS / 8; ++nt) {
                float s2[4] = {0.f, 0.f, 0.f, 0.f};
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    // 16 codes: chunk c & 1 of the lane's pair (rows of 128 bytes), or its only one
                    const uint4 v = lds128(kt + (C::ROW == 128 ? (c >> 1) * BS * 128 : 0) +
                                           chunk8<C::ROW>(nt * 8 + g, C::ROW == 128 ? 2 * tig + (c & 1) : tig));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t k0 = decode2((uint16_t)w[x]), k1 = decode2((uint16_t)(w[x] >> 16));
                        Mma<__half>::mma(x & 1 ? s2 : s[nt], qa[c * 4 + x], k0, k1);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] += s2[e];
            }

            // ---- exponents s_t + log2 sv, their maxima, and a rescale where one rises ----
            const float svc = fminf(fmaxf(page_sv, kMinScale8), kMaxScale8);
            const float lv = __log2f(svc), c0 = qk0 * page_sk, c1 = qk1 * page_sk;
            const int v0 = lim0 - first, v1 = lim1 - first;
            float mx0 = NEG_INF, mx1 = NEG_INF;
            const bool masked = lim_least - first < BS;
#pragma unroll
            for (int nt = 0; nt < BS / 8; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[nt][e] = fmaf(s[nt][e], c0, lv);
                    s[nt][2 + e] = fmaf(s[nt][2 + e], c1, lv);
                    if (masked) {
                        const int t = nt * 8 + tig * 2 + e;
                        if (t >= v0) s[nt][e] = NEG_INF;
                        if (t >= v1) s[nt][2 + e] = NEG_INF;
                    }
                    mx0 = fmaxf(mx0, s[nt][e]);
                    mx1 = fmaxf(mx1, s[nt][2 + e]);
                }
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, x));
                mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, x));
            }
            const bool need = (real0 && mx0 > m0 + (kSlack + kHalfLift)) ||
                              (real1 && mx1 > m1 + (kSlack + kHalfLift));
            if (__any_sync(kFullMask, need)) {
                const float n0 = real0 ? fmaxf(m0, mx0 - kHalfLift) : m0;
                const float n1 = real1 ? fmaxf(m1, mx1 - kHalfLift) : m1;
                const float a0 = n0 == m0 ? 1.f : fast_exp2(m0 - n0);
                const float a1 = n1 == m1 ? 1.f : fast_exp2(m1 - n1);
                m0 = n0, m1 = n1;
                l0 *= a0, l1 *= a1;
#pragma unroll
                for (int n = 0; n < ONT; ++n) {
                    acc[n][0] *= a0, acc[n][1] *= a0;
                    acc[n][2] *= a1, acc[n][3] *= a1;
                }
            }
            // ---- weights (a row without a token so far has m = -inf and weights 0) ----
            const float e0 = m0 == NEG_INF ? 0.f : m0, e1 = m1 == NEG_INF ? 0.f : m1;
            float t0 = 0.f, t1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < BS / 8; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[nt][e] = real0 ? fast_exp2(s[nt][e] - e0) : 0.f;
                    s[nt][2 + e] = real1 ? fast_exp2(s[nt][2 + e] - e1) : 0.f;
                    t0 += s[nt][e];
                    t1 += s[nt][2 + e];
                }
            const float inv_sv = __frcp_rn(svc);
            l0 = fmaf(t0, inv_sv, l0);
            l1 = fmaf(t1, inv_sv, l1);

            // ---- O += P V ----
#pragma unroll
            for (int ks = 0; ks < BS / 16; ++ks) {
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x0 = s[2 * ks + (r >> 1)][(r & 1) * 2];
                    const float x1 = s[2 * ks + (r >> 1)][(r & 1) * 2 + 1];
                    ph[r] = Mma<__half>::pack(x0, x1);
                    float h0, h1;
                    Mma<__half>::unpack(ph[r], h0, h1);
                    pl[r] = Mma<__half>::pack(x0 - h0, x1 - h1);
                }
                // rows 2 tig, + 1, + 8, + 9 of the 16; ONT codes from g * ONT on
                constexpr int WORDS = ONT / 4;
                uint32_t v[4][WORDS];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = ks * 16 + tig * 2 + (r & 1) + (r >> 1) * 8;
                    if constexpr (WORDS == 4) {
                        const uint4 x = lds128(vt + ds * BS * 128 + chunk8<C::ROW>(t, g));
                        v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                    } else {
                        const uint2 x = lds64(vt + chunk8<C::ROW>(t, g >> 1) + (g & 1) * 8);
                        v[r][0] = x.x, v[r][1] = x.y;
                    }
                    if (nvalid < BS && t >= nvalid)  // slots past the context: 0 * NaN is not 0
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) v[r][w] = 0;
                }
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140);
                    const uint32_t a23 = __byte_perm(v[0][w], v[1][w], 0x7362);
                    const uint32_t b01 = __byte_perm(v[2][w], v[3][w], 0x5140);
                    const uint32_t b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
                    const uint32_t x[4] = {decode2((uint16_t)a01), decode2((uint16_t)(a01 >> 16)),
                                           decode2((uint16_t)a23), decode2((uint16_t)(a23 >> 16))};
                    const uint32_t y[4] = {decode2((uint16_t)b01), decode2((uint16_t)(b01 >> 16)),
                                           decode2((uint16_t)b23), decode2((uint16_t)(b23 >> 16))};
#pragma unroll
                    for (int n = 0; n < 4; ++n) Mma<__half>::mma(acc[w * 4 + n], ph, x[n], y[n]);
#pragma unroll
                    for (int n = 0; n < 4; ++n) Mma<__half>::mma(acc[w * 4 + n], pl, x[n], y[n]);
                }
            }
        }
        __syncwarp();
        if (DS > 1 && lane == 0) mbar_arrive(smem_u32(empty + sidx));
        if (i + NS < n_s && !aborted) {
            // the stage is free: the stream's page i + NS
            if (DS > 1 && ds == 0 &&
                !__all_sync(kFullMask, mbar_wait_bounded(smem_u32(empty + sidx), (i / NS) & 1, p.timeout_ns))) {
                if (lane == 0) record_error(p.err, PA_ERR_TIMEOUT);
                aborted = true;
            }
            if (!aborted) {
                fence_proxy_async_smem();
                issue(i + NS);
                ++issued;
            }
        }
        if (aborted) {
            // copies in flight land before the stages are used again
            if (ds == 0 && lane == 0)
                for (int k = i + 1; k < issued; ++k)
                    (void)mbar_wait_bounded(smem_u32(full + stream * NS + k % NS), (k / NS) & 1, p.timeout_ns);
            break;
        }
    }

    // ---- join the warps' results in the stage area ----
    l0 += __shfl_xor_sync(kFullMask, l0, 1);
    l1 += __shfl_xor_sync(kFullMask, l1, 1);
    l0 += __shfl_xor_sync(kFullMask, l0, 2);
    l1 += __shfl_xor_sync(kFullMask, l1, 2);
    float* macc = reinterpret_cast<float*>(smem);       // [4][R][DW]
    float* mm = macc + 4 * R * DW;                      // [4][R]
    float* ml = mm + 4 * R;                             // [4][R]
    float* cpart = ml + 4 * R;                          // cluster: acc [R][D], m [R], l [R]
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!(h ? real1 : real0)) continue;
        // a lane's columns: ONT from 2 tig * ONT on, and as many again
        float* at = macc + ((size_t)warp * R + g + h * 8) * DW + tig * 2 * ONT;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < ONT; n += 4)
                *reinterpret_cast<float4*>(at + e * ONT + n) =
                    make_float4(acc[n][h * 2 + e], acc[n + 1][h * 2 + e], acc[n + 2][h * 2 + e],
                                acc[n + 3][h * 2 + e]);
        if (tig == 0) {
            mm[warp * R + g + h * 8] = h ? m1 : m0;
            ml[warp * R + g + h * 8] = h ? l1 : l0;
        }
    }
    __syncthreads();
    const size_t row0 = (((size_t)b * Hkv + kvh) * p.num_parts + part) * ((size_t)Q * G) + (size_t)qi0 * G;
    for (int idx = tid; idx < R * D; idx += 128) {
        const int r = idx / D, d = idx % D, w0 = d / DW;
        float M = NEG_INF;
#pragma unroll
        for (int x = 0; x < NT; ++x) M = fmaxf(M, mm[(x * DS + w0) * R + r]);
        float A = 0.f, L = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int w = x * DS + w0;
            const float m = mm[w * R + r];
            const float f = m == NEG_INF ? 0.f : fast_exp2(m - M);
            A = fmaf(f, macc[((size_t)w * R + r) * DW + d % DW], A);
            L = fmaf(f, ml[w * R + r], L);
        }
        if (p.cluster > 1) {
            cpart[idx] = A;
            if (d == 0) cpart[R * D + r] = M, cpart[R * D + R + r] = L;
        } else if (p.num_parts > 1) {
            p.part_acc[(row0 + r) * D + d] = A;
            if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (row0 + r) * 2) = make_float2(M, L);
        } else {
            store_out(p.out, row_off(r) + d, L == 0.f ? 0.f : A / L, p.out_dtype);
        }
    }
    if (p.cluster > 1) {
        // the cluster's partitions, through distributed shared memory: each CTA
        // finishes a share of the outputs
        cluster_sync_release_acquire();
        const uint32_t cp = smem_u32(cpart);
        const int P = p.num_parts, share = (R * D + P - 1) / P;
        const int end = min((part + 1) * share, R * D);
        uint32_t base[kMaxClusterParts];
#pragma unroll
        for (int x = 0; x < kMaxClusterParts; ++x) base[x] = map_cluster_rank(cp, (uint32_t)(x < P ? x : 0));
        for (int idx = part * share + tid; idx < end; idx += 128) {
            const int r = idx / D;
            float m[kMaxClusterParts], l[kMaxClusterParts], a[kMaxClusterParts], M = NEG_INF;
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) {
                    m[x] = ld_cluster_f32(base[x] + 4u * (R * D + r));
                    l[x] = ld_cluster_f32(base[x] + 4u * (R * D + R + r));
                    a[x] = ld_cluster_f32(base[x] + 4u * idx);
                }
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) M = fmaxf(M, m[x]);
            float A = 0.f, L = 0.f;
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) {  // (0 * NaN: a row of NaN stays one)
                    const float f = m[x] == NEG_INF ? 0.f : fast_exp2(m[x] - M);
                    A = fmaf(f, a[x], A);
                    L = fmaf(f, l[x], L);
                }
            store_out(p.out, row_off(r) + idx % D, L == 0.f ? 0.f : A / L, p.out_dtype);
        }
        cluster_sync_relaxed();  // no CTA leaves while others read its shared memory
    }
}

template <int D, int BS, typename T>
cudaError_t launch_kv8_inst(const Kv8Launch& L, cudaStream_t stream) {
    static AttrFlags raised;
    auto kern = kv8_kernel<D, BS, T>;
    cudaError_t e = raise_smem_limit_once(kern, raised);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = L.grid;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = Kv8Cfg<D, BS>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (L.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (L.p.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)L.p.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, L.tmap_k, L.tmap_v, L.p);
}

template <int D>
cudaError_t launch_kv8_for_d(const Kv8Launch& L, cudaStream_t stream) {
    if (L.block_size == 16)
        return L.bf16 ? launch_kv8_inst<D, 16, __nv_bfloat16>(L, stream)
                      : launch_kv8_inst<D, 16, __half>(L, stream);
    return L.bf16 ? launch_kv8_inst<D, 32, __nv_bfloat16>(L, stream)
                  : launch_kv8_inst<D, 32, __half>(L, stream);
}

}  // namespace pa
