// Attention over the 8-bit cache.  A unit is a (sequence, kv head, chunk of up to
// 32 query rows).  The CTAs work in groups, adjacent blocks that walk the same
// tokens for different units of a sequence (a page's kv heads lie side by side:
// read at different times, 128 bytes each, they cost 166 us where read together
// they cost 94).  A group takes an equal run of the flattened (sequence, group of
// units, 32-token step) order whatever the lengths, a few segments each (the
// pieces of a unit that is cut are joined by kv8_join_kernel); or a CTA takes a
// unit whole, or, of few and short units, a partition that a cluster of up to 8
// joins.
//
// The mathematics: with codes k8, v8 and the page's scales sk, sv,
//     s_t = scale * sk (q . k8_t),      out = sum_t 2^(s_t) sv v8_t / sum_t 2^(s_t)
// (s in base-2 units).  The value's scale goes into the weight's exponent,
//     w_t = 2^(s_t + log2 sv - m),  m a reference near the maximum of s_t + log2 sv,
//     acc = sum_t w_t v8_t,         l = sum over pages of (1 / sv) sum_t w_t,
// so that a weight is as large as its token's share of the output can be: a page
// of tiny values keeps its precision where its tokens have all the weight, and
// no page's values are ever multiplied.
//
// The MMAs are warp-level m16n8k16 in fp16, to which e4m3 widens exactly
// (cvt.f16x2.e4m3x2, two codes an instruction); for so few rows a tcgen05 tile
// would be mostly empty, and its operands would go through shared memory a
// second time.  Both products are transposed, tokens and value elements in M,
// query rows in N:
//     S^T [16 tokens x 8 rows] += K [16 x 16] Q^T,   O^T [16 elements x 8 rows] += V^T [16 x 16] P^T
// so that a group of 8 heads or fewer costs half of what 16-row tiles did.
// Nothing is transposed in memory: a lane loads 16 consecutive codes of a token's
// key, and the products' k order, and the output's element order, are permuted
// to what the lanes hold (the queries are loaded in that order).  Values go
// two tokens at a time through a byte permutation, four elements of each to the
// registers that the conversion turns into the A operand; the weights change
// sides by movmatrix.
// Bounds: of few rows DRAM (4 sequences of 131,072 tokens, 8 kv heads of 128, 1.08
// GB: 176 us, 6.1 TB/s; the copies alone 170), behind it the half-rate pipe of the
// conversions and permutations (two cycles each; 33 % busy) and the MMAs (one in
// 2 cycles an SM; 21 % with weights in two parts); of 64 sequences of 1 .. 4096
// tokens (270 MB) 57 us, 4.7 TB/s, 12 us of them starts, cuts and the join.  Of many rows at head_dim 256 the
// latency of a step's chain on the two warps that a scheduler holds: 16 sequences of
// 8K tokens, 64 rows: 51 us, 2.1 a step of 32 tokens.
//
// Weights meet the values as fp16, 2^kHalfLift up (pa_internal.h), in two parts; once
// rounded (by at most 2^-11 of each) where the output is bf16, whose own rounding is
// eight times that.  In one part it is half of the second product: 51 us against 57 for
// 16 sequences of 8K tokens with 64 rows of 256, 56 against 57 for 64 of 1 .. 4096, no
// difference for 4 of 131,072; an fp16 output's error would grow by a tenth (0.00020
// to 0.00022).  Tokens whose w_t lies 2^-32 under the row's largest are lost whole:
// their values add nothing to an output, but their 2^(s_t) may be most of the
// normaliser (a page of zero values has sv = 2^-60).  So l sums the weights as they
// are, in fp32.
// fp32 ends as well, at 2^-126: where a page on the scale 2^60 is met, tokens of one
// on 2^-60 lie there from 2^-6 of its weights down, however many they are.  So pages
// more than 2^64 under the largest scale sum 2^(s_t - m) itself, which loses no token
// above 2^-69 of the row's largest, and where a sum moves to another reference, the
// factor 2^(m' - m) of l is applied as two halves (scale_sum), each inside fp32.
// The queries are brought to fp16 exactly, each row scaled by a power of two to
// below 2^15 (elements 2^-28 and less of the row's largest begin to round).
#pragma once

#include "pa_kv8.cuh"

namespace pa {

// NR: tiles of 8 query rows of a CTA.
template <int D, int BS, int NR>
struct Kv8Cfg {
    static constexpr int NW = 4;                    // warps, each a token stream with a ring of its own
    static constexpr int KSTEPS = D / 16;
    static constexpr int MT = D / 16;               // 16-element tiles of O^T
    static constexpr int ROW = D < 128 ? D : 128;   // bytes of a row of a column block
    static constexpr int BLK = D / ROW;             // column blocks
    static constexpr int STEP = 32;                 // tokens of a step: one page of 32, two of 16
    static constexpr int PP = STEP / BS;
    static constexpr uint32_t PAGE = BS * D;        // bytes of a page's keys of one head
    static constexpr uint32_t TILE = STEP * D;      // and of a step's
    static constexpr bool QSMEM = KSTEPS * NR > 16; // queries' fragments in shared memory, not registers
    // CTAs of an SM: two hold the queries, sums and weights in registers; at head_dim
    // 64 three do (three at 128: the same time, with spills)
    static constexpr int CTAS = D == 64 && NR < 4 ? 3 : 2;
    // stages of a ring: as a CTA's share of shared memory allows
    static constexpr int NS_RAW = (int)((224u / CTAS - 4u) * 1024u / (NW * 2 * TILE));
    static constexpr int NS = NS_RAW > 4 ? 4 : NS_RAW < 1 ? 1 : NS_RAW;
    static constexpr uint32_t RING = NW * NS * 2 * TILE;
    static constexpr int R = NR * 8;
    // the join of the warps, and of a cluster, in the rings' place
    static constexpr uint32_t JOIN = 4u * (NW * R * D + R * D + 2 * NW * R + 4 * R);
    static constexpr uint32_t BAR_OFF = RING > JOIN ? RING : JOIN;
    static constexpr uint32_t RUN_OFF = BAR_OFF + (8 + 4) * NW * NS + 16 - (12 * NW * NS) % 16;
    static constexpr uint32_t QK_OFF = RUN_OFF + 48;  // [R] the queries' factors (beside the fragments)
    static constexpr uint32_t Q_OFF = QK_OFF + (QSMEM ? R * 4u : 0u);
    static constexpr uint32_t SMEM = Q_OFF + (QSMEM ? KSTEPS * NR * 256u : 0u) + kSmemAlignSlack;
    static_assert(SMEM * CTAS <= 227u * 1024u - CTAS * 1024u, "shared memory");
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
__device__ __forceinline__ void sts128_zero(uint32_t a) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}


// Four consecutive outputs v * f in the output's type.
__device__ __forceinline__ void store4(void* out, size_t at, float4 v, float f, int out_dtype) {
    v.x *= f, v.y *= f, v.z *= f, v.w *= f;
    if (out_dtype == PA_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
    else if (out_dtype == PA_F16)
        *reinterpret_cast<uint2*>(static_cast<__half*>(out) + at) =
            make_uint2(Mma<__half>::pack(v.x, v.y), Mma<__half>::pack(v.z, v.w));
    else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
            make_uint2(Mma<__nv_bfloat16>::pack(v.x, v.y), Mma<__nv_bfloat16>::pack(v.z, v.w));
}

// l * 2^d (d <= 0) where 2^d itself may be below fp32's numbers and l far above one;
// f: 2^d, or 0.
__device__ __forceinline__ float scale_sum(float l, float d, float& f) {
    const float h = fast_exp2(0.5f * d);
    f = h * h;
    return l * h * h;
}

// 8 x 8 16-bit values, a row to four lanes, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int D, int BS, int NR, bool HL>
__global__ void __launch_bounds__(128, Kv8Cfg<D, BS, NR>::CTAS)
    kv8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
               const Kv8Params p) {
    using C = Kv8Cfg<D, BS, NR>;
    constexpr int NW = C::NW, NS = C::NS, KSTEPS = C::KSTEPS, MT = C::MT, STEP = C::STEP, PP = C::PP;
    constexpr float NEG_INF = -INFINITY;
    constexpr float kSlack = 8.f;  // log2 units that weights may stand above 2^kHalfLift

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlignSlack - 1)) & ~uintptr_t(kSmemAlignSlack - 1));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    int32_t* on_of = reinterpret_cast<int32_t*>(full + NW * NS);
    uint2* qs = reinterpret_cast<uint2*>(smem + C::Q_OFF);  // [KSTEPS][NR][32]
    float* qks = reinterpret_cast<float*>(smem + C::QK_OFF);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int G = p.group, Hkv = p.num_kv_heads, Q = p.q_len;
    const int gshift = __ffs(G) - 1;  // the group is a power of two
    // start, end, flat position of the present sequence's steps, total, present
    // position; the present sequence
    long long* run = reinterpret_cast<long long*>(smem + C::RUN_OFF);
    int32_t* run_b = reinterpret_cast<int32_t*>(run + 5);

    if (tid == 0) {
        for (int i = 0; i < NW * NS; ++i) mbar_init(smem_u32(full + i), 1);
        mbar_init_fence();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    const int per_seq = Hkv * p.chunks;  // units of a sequence
    auto steps_of = [&](int b) -> int {
        const int t = min(min(max(__ldg(p.context_lens + b), 0), p.max_blocks * BS), p.token_limit);
        return max((t + STEP - 1) / STEP, 1);  // (an empty sequence writes its zeros)
    };
    if (p.balanced && warp == 0) {
        // the CTA's run: [start, end) of all steps, and the sequence that it begins in
        long long w = 0;
        for (int b = lane; b < p.batch; b += 32) w += steps_of(b);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) w += __shfl_xor_sync(kFullMask, w, k);
        w *= p.unit_groups;
        const long long groups = gridDim.x / p.group_size, group = blockIdx.x / p.group_size;
        const long long start = group * w / groups, end = (group + 1) * w / groups;
        int b = 0;
        long long base = 0;
        while (start < end) {
            const int bb = b + lane;
            const long long v = bb < p.batch ? (long long)steps_of(bb) * p.unit_groups : 0;
            long long incl = v;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const long long o = __shfl_up_sync(kFullMask, incl, k);
                if (lane >= k) incl += o;
            }
            const unsigned hit = __ballot_sync(kFullMask, bb < p.batch && base + incl > start);
            if (hit) {
                const int k = __ffs(hit) - 1;
                base += __shfl_sync(kFullMask, incl - v, k);
                b += k;
                break;
            }
            base += __shfl_sync(kFullMask, incl, 31);
            b += 32;
        }
        if (lane == 0) run[0] = run[4] = start, run[1] = end, run[2] = base, run[3] = w, *run_b = b;
    }
    __syncthreads();  // barriers initialised, the run known

    bool aborted = false;
    int done = 0;  // steps of the warp's ring so far

    // Steps [k0, k1) of unit (b, kvh, chunk); `record`: where a piece's (m, l, acc)
    // go, -1 for a whole unit's output, -2 for a cluster's.
    auto segment = [&](int b, int kvh, int chunk, int k0, int k1, long long record) {
    const int qi0 = chunk * p.q_chunk;
    const int R = min(p.q_chunk, Q - qi0) * G;
    const int ctx = max(__ldg(p.context_lens + b), 0);
    const int reach = min(min(ctx, p.max_blocks * BS), p.token_limit);  // tokens of the call
    const int pb = k0 * PP, pe = min(k1 * PP, (reach + BS - 1) / BS);
    auto row_off = [&](int r) -> size_t {
        return (((size_t)b * Q + qi0 + (r >> gshift)) * p.num_heads + kvh * G + (r & (G - 1))) * D;
    };

    // ---- the warp's steps of PP pages: number warp, warp + NW, ... of the
    // segment's; it keeps 32 table entries ahead, one a lane, and the scales of
    // the pages that it consumes ----
    constexpr int WINDOW = 32 / PP;  // steps whose entries the lanes hold
    const int steps = pe > pb ? (pe - pb + PP - 1) / PP : 0;
    const int n_s = steps > warp ? (steps - warp + NW - 1) / NW : 0;
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks;
    auto fetch = [&](int chunk) -> int {
        const int j = pb + (warp + (chunk * WINDOW + lane / PP) * NW) * PP + lane % PP;
        const int e = j < pe ? __ldg(table + j) : -1;
        return e >= 0 && (int64_t)e < p.num_blocks ? e : -1;
    };
    float sk_ahead = 0.f, sv_ahead = 1.f;
    auto fetch_scales = [&](int e) {
        sk_ahead = e >= 0 ? __ldg(p.k_scales + (size_t)e * Hkv + kvh) : 0.f;
        sv_ahead = e >= 0 ? __ldg(p.v_scales + (size_t)e * Hkv + kvh) : 1.f;
    };
    int ent = fetch(0), ent_next = fetch(1);
    // Whole warp: entries of its step i, and (one lane) the copies.
    auto issue = [&](int i) {
        if (i > 0 && i % WINDOW == 0) {
            ent = ent_next;
            ent_next = fetch(i / WINDOW + 1);
            fetch_scales(ent);  // (consumed from step i on, NS steps later)
        }
        int e[PP];
        uint32_t on = 0;
#pragma unroll
        for (int u = 0; u < PP; ++u) {
            e[u] = __shfl_sync(kFullMask, ent, i % WINDOW * PP + u);
            on |= (e[u] >= 0 ? 1u : 0u) << u;
        }
        if (lane == 0) {
            const int sidx = warp * NS + (done + i) % NS;
            const uint32_t bar = smem_u32(full + sidx);
            on_of[sidx] = (int32_t)on;
            if (on) {
                // (several chunks of rows read the same pages)
                const uint64_t policy = p.chunks > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
                mbar_arrive_expect_tx(bar, 2 * C::PAGE * __popc(on));
#pragma unroll
                for (int u = 0; u < PP; ++u) {
                    if (e[u] < 0) continue;
                    const uint32_t dst = smem_u32(smem) + (uint32_t)sidx * 2 * C::TILE + u * BS * C::ROW;
#pragma unroll
                    for (int blk = 0; blk < C::BLK; ++blk) {
                        tma_load_4d(dst + blk * STEP * C::ROW, &tmap_k, blk * C::ROW, kvh, 0, e[u], bar, policy);
                        tma_load_4d(dst + C::TILE + blk * STEP * C::ROW, &tmap_v, blk * C::ROW, kvh, 0, e[u],
                                    bar, policy);
                    }
                }
            } else {
                mbar_arrive(bar);
            }
        }
    };
    // The queries, B operand of S^T: element order of a lane's keys, row g of each
    // tile.  (Loaded ahead of the first pages, behind which they waited 4 us.)  With
    // the fragments in shared memory a warp takes the tiles warp, warp + NW, ...
    constexpr int MINE = C::QSMEM ? (NR + NW - 1) / NW : NR, STRIDE = C::QSMEM ? NW : 1;
    const int j0 = C::QSMEM ? warp : 0;
    uint2 raw[MINE][KSTEPS];
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int r = (j0 + y * STRIDE) * 8 + g;
        const bool real = r < R;  // (other rows: zeros, their results are not used)
        const char* q = static_cast<const char*>(p.q) + row_off(real ? r : 0) * 2;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) {
            const int d = k / (C::ROW / 16) * C::ROW + tig * (C::ROW / 4) + k % (C::ROW / 16) * 4;
            raw[y][k] = real ? __ldg(reinterpret_cast<const uint2*>(q + d * 2)) : make_uint2(0, 0);
        }
    }
    fence_proxy_async_smem();  // the last segment's join used the rings
    for (int i = 0; i < min(n_s, NS); ++i) issue(i);
    fetch_scales(ent);

    // each row scaled by a power of two
    uint2 qf[C::QSMEM ? 1 : KSTEPS][C::QSMEM ? 1 : NR];
    float qk[NR][2];  // of rows 2 tig, + 1: scale * log2(e), and the row's power of two taken out again
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
        const int j = j0 + y * STRIDE;
        auto widen = [&](uint32_t x, float& lo, float& hi) {
            if (p.bf16) Mma<__nv_bfloat16>::unpack(x, lo, hi);
            else Mma<__half>::unpack(x, lo, hi);
        };
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) {
            float a, c, d, e;
            widen(raw[y][k].x, a, c);
            widen(raw[y][k].y, d, e);
            top = fmaxf(top, fmaxf(fmaxf(fabsf(a), fabsf(c)), fmaxf(fabsf(d), fabsf(e))));
        }
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        // 2^14 <= f * top < 2^15 (rows of less than 2^-112: f = 2^126)
        const int ex = max(min(268 - (int)(__float_as_uint(top) >> 23), 253), 1);
        const float f = __uint_as_float((uint32_t)ex << 23);
        const float back = p.qscale * __uint_as_float((uint32_t)(254 - ex) << 23);
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) {
            float a, c, d, e;
            widen(raw[y][k].x, a, c);
            widen(raw[y][k].y, d, e);
            const uint2 v = make_uint2(Mma<__half>::pack(a * f, c * f), Mma<__half>::pack(d * f, e * f));
            if constexpr (C::QSMEM) {
                if (j < NR) qs[(k * NR + j) * 32 + lane] = v;
            } else {
                qf[k][y] = v;
            }
        }
        if constexpr (C::QSMEM) {
            if (j < NR && tig == 0) qks[j * 8 + g] = back;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) qk[y][e] = __shfl_sync(kFullMask, back, (tig * 2 + e) * 4);
        }
    }
    if constexpr (C::QSMEM) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) qk[j][e] = qks[j * 8 + tig * 2 + e];
    }
    // Tokens that a row attends to: its query token's causal limit; the first row's
    // is the least.  (Rows past R see all: their results are not used.)
    const int lim_first = ctx - Q + qi0 + 1, lim_least = min(reach, lim_first);
    auto lim = [&](int r) { return min(reach, lim_first + (r >> gshift)); };

    float m[NR][2], l[NR][2], acc[MT][NR][4];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) m[j][e] = NEG_INF, l[j][e] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;

    float sk = 0.f, sv = 1.f;
    float lv_top = NEG_INF;  // largest log2 sv that the warp has met
    int issued = min(n_s, NS);
    for (int i = 0; i < n_s; ++i) {
        if (i % WINDOW == 0) sk = sk_ahead, sv = sv_ahead;
        const int sidx = warp * NS + (done + i) % NS;
        if (!__all_sync(kFullMask,
                        mbar_wait_bounded(smem_u32(full + sidx), ((done + i) / NS) & 1, p.timeout_ns))) {
            if (lane == 0) record_error(p.err, PA_ERR_TIMEOUT);
            aborted = true;
        }
        float page_sk[PP], page_sv[PP];
#pragma unroll
        for (int u = 0; u < PP; ++u) {
            page_sk[u] = __shfl_sync(kFullMask, sk, i % WINDOW * PP + u);
            page_sv[u] = __shfl_sync(kFullMask, sv, i % WINDOW * PP + u);
        }
        const uint32_t on = on_of[sidx];  // pages of the step that are there
        if (!aborted && on) {
            const int first = (pb + (warp + i * NW) * PP) * BS;
            // tokens of the step before the context's end; those of a page that is not
            // there are masked one by one
            const int nvalid = reach - first;
            const bool whole = nvalid >= STEP && on == (1u << PP) - 1;
            auto held = [&](int t) { return t < nvalid && (PP == 1 || (on >> (t / BS) & 1)); };
            const uint32_t kt = smem_u32(smem) + (uint32_t)sidx * 2 * C::TILE, vt = kt + C::TILE;

            // ---- S^T = K Q^T: tokens g, g + 8 of each 16, rows 2 tig, + 1 ----
            float s[2][NR][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < NR; ++j) s[t][j][0] = s[t][j][1] = s[t][j][2] = s[t][j][3] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                // 16 codes of a token: chunk c & 1 of the lane's pair (rows of 128 bytes), or its only one
                const uint32_t at = kt + (C::ROW == 128 ? (c >> 1) * STEP * 128 : 0);
                const int ch = C::ROW == 128 ? 2 * tig + (c & 1) : tig;
                uint4 v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) v[t] = lds128(at + chunk8<C::ROW>(t * 8 + g, ch));
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int k = c * 4 + x;
                    uint32_t a[2][4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t w = x == 0 ? v[t].x : x == 1 ? v[t].y : x == 2 ? v[t].z : v[t].w;
                        a[t >> 1][t & 1] = decode2((uint16_t)w);
                        a[t >> 1][2 + (t & 1)] = decode2((uint16_t)(w >> 16));
                    }
#pragma unroll
                    for (int j = 0; j < NR; ++j) {
                        uint2 y;
                        if constexpr (C::QSMEM) y = lds64(smem_u32(smem) + C::Q_OFF + ((k * NR + j) * 32 + lane) * 8);
                        else y = qf[k][j];
                        Mma<__half>::mma(s[0][j], a[0], y.x, y.y);
                        Mma<__half>::mma(s[1][j], a[1], y.x, y.y);
                    }
                }
            }

            // ---- exponents s_t + log2 sv; a rescale where one stands 2^8 above the reference ----
            float lv[PP], inv_sv[PP];
#pragma unroll
            for (int u = 0; u < PP; ++u) {
                const float svc = fminf(fmaxf(page_sv[u], kMinScale8), kMaxScale8);
                lv[u] = __log2f(svc);
                inv_sv[u] = __frcp_rn(svc);
            }
            const bool masked = !whole || lim_least - first < STEP;
            float above = NEG_INF;
#pragma unroll
            for (int j = 0; j < NR; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int u = t * 16 / BS;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        s[t][j][c] = fmaf(s[t][j][c], qk[j][c & 1] * page_sk[u], lv[u]);
                }
            if (masked) {
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int at = t * 16 + (c >> 1) * 8 + g;
                            if (first + at >= lim(j * 8 + tig * 2 + (c & 1)) || !held(at)) s[t][j][c] = NEG_INF;
                        }
            }
#pragma unroll
            for (int j = 0; j < NR; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) above = fmaxf(above, s[t][j][c] - m[j][c & 1]);
            if (__any_sync(kFullMask, above > kSlack + kHalfLift)) {
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(s[0][j][e], s[0][j][2 + e]), fmaxf(s[1][j][e], s[1][j][2 + e]));
#pragma unroll
                        for (int x = 4; x <= 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
                        const float to = fmaxf(m[j][e], top - kHalfLift);
                        float f = 1.f;
                        if (to != m[j][e]) l[j][e] = scale_sum(l[j][e], m[j][e] - to, f);
                        m[j][e] = to;
#pragma unroll
                        for (int k = 0; k < MT; ++k) acc[k][j][e] *= f, acc[k][j][2 + e] *= f;
                    }
            }
            if (!whole) {
                // slots without a token hold zeros in the second product: 0 * NaN is not 0
                for (int i = lane; i < STEP * (D / 16); i += 32) {
                    const int at = i / (C::ROW / 16) % STEP, blk = i / (C::ROW / 16) / STEP;
                    if (!held(at))
                        sts128_zero(vt + blk * STEP * C::ROW + at * C::ROW + i % (C::ROW / 16) * 16);
                }
                __syncwarp();
            }
            // ---- weights: P^T, B operand of the second product (a row without a token
            // so far has m = -inf, and weights 2^-inf) ----
            float mr[NR][2];
#pragma unroll
            for (int j = 0; j < NR; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) mr[j][e] = m[j][e] == NEG_INF ? 0.f : m[j][e];
#pragma unroll
            for (int u = 0; u < PP; ++u) {
                lv_top = fmaxf(lv_top, lv[u]);
                if (lv_top - lv[u] > 64.f) {
                    // weights times sv may lie below fp32's numbers: the sum without sv
#pragma unroll
                    for (int t = u * (2 / PP); t < (u + 1) * (2 / PP); ++t)
#pragma unroll
                        for (int j = 0; j < NR; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c) l[j][c & 1] += fast_exp2(s[t][j][c] - mr[j][c & 1] - lv[u]);
                    inv_sv[u] = 0.f;
                }
            }
            uint32_t ph[2][NR][2], pl[HL ? 2 : 1][HL ? NR : 1][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int u = t * 16 / BS;
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = fast_exp2(s[t][j][2 * h] - mr[j][0]);
                        const float e1 = fast_exp2(s[t][j][2 * h + 1] - mr[j][1]);
                        const uint32_t hi = Mma<__half>::pack(e0, e1);
                        ph[t][j][h] = movmatrix_trans(hi);
                        if constexpr (HL) {
                            float h0, h1;
                            Mma<__half>::unpack(hi, h0, h1);
                            pl[t][j][h] = movmatrix_trans(Mma<__half>::pack(e0 - h0, e1 - h1));
                        }
                        // (not the rounded ones: a page whose values are far smaller than
                        // another's has weights that vanish in fp16, not in the softmax)
                        l[j][0] = fmaf(e0, inv_sv[u], l[j][0]);
                        l[j][1] = fmaf(e1, inv_sv[u], l[j][1]);
                    }
            }

            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                constexpr int WORDS = C::ROW / 32;  // of a lane's elements in a block: 16 codes, or 8
#pragma unroll
                for (int blk = 0; blk < C::BLK; ++blk) {
                    uint32_t v[4][WORDS];  // tokens 2 tig, + 1, + 8, + 9 of the 16
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = t * 16 + tig * 2 + (r & 1) + (r >> 1) * 8;
                        if constexpr (WORDS == 4) {
                            const uint4 x = lds128(vt + blk * STEP * 128 + chunk8<C::ROW>(at, g));
                            v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                        } else {
                            const uint2 x = lds64(vt + chunk8<C::ROW>(at, g >> 1) + (g & 1) * 8);
                            v[r][0] = x.x, v[r][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // elements 4 w + 2 h, + 1 of the lane's
                            const uint32_t lo = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
                            const uint32_t a[4] = {decode2((uint16_t)lo), decode2((uint16_t)(lo >> 16)),
                                                   decode2((uint16_t)hi), decode2((uint16_t)(hi >> 16))};
                            const int k = (blk * WORDS + w) * 2 + h;
#pragma unroll
                            for (int j = 0; j < NR; ++j) {
                                Mma<__half>::mma(acc[k][j], a, ph[t][j][0], ph[t][j][1]);
                                if constexpr (HL) Mma<__half>::mma(acc[k][j], a, pl[t][j][0], pl[t][j][1]);
                            }
                        }
                }
            }
        }
        __syncwarp();
        if (i + NS < n_s && !aborted) {  // the stage is free: the warp's step i + NS
            fence_proxy_async_smem();
            issue(i + NS);
            ++issued;
        }
        if (aborted) {
            // copies in flight land before the stages are used again
            if (lane == 0)
                for (int k = i + 1; k < issued; ++k)
                    (void)mbar_wait_bounded(smem_u32(full + warp * NS + (done + k) % NS),
                                            ((done + k) / NS) & 1, p.timeout_ns);
            break;
        }
    }
    done += n_s;

    // ---- join the warps' results in the rings' place ----
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) l[j][e] += __shfl_xor_sync(kFullMask, l[j][e], x);
    float4* macc = reinterpret_cast<float4*>(smem);     // [NW][R][D / 4], a row's vectors permuted:
    // eight lanes that store at once have two g and four rows of the same banks
    auto mix = [](int r) { return C::ROW == 128 ? r >> 1 & 3 : (r >> 1 & 1) | (r & 4); };
    float* cpart = reinterpret_cast<float*>(macc) + NW * R * D;  // cluster: acc [R][D], m [R], l [R]
    float* mm = cpart + R * D + 2 * R;                  // [NW][R], then the warps' factors
    float* ml = mm + NW * R;                            // [NW][R]
    float* tot = ml + NW * R;                           // [R][2] m and l of the row
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = j * 8 + tig * 2 + e;
            if (r >= R) continue;
            constexpr int PER = C::ROW / 8;             // a lane's elements of a block
#pragma unroll
            for (int k = 0; k < MT; k += 2) {
                const int blk = k / (PER / 2), d = blk * C::ROW + g * PER + k % (PER / 2) * 2;
                macc[(warp * R + r) * (D / 4) + ((d / 4) ^ mix(r))] =
                    make_float4(acc[k][j][e], acc[k][j][2 + e], acc[k + 1][j][e], acc[k + 1][j][2 + e]);
            }
            if (g == 0) mm[warp * R + r] = m[j][e], ml[warp * R + r] = l[j][e];
        }
    __syncthreads();
    if (tid < R) {
        float M = NEG_INF, L = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mm[w * R + tid]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float x = mm[w * R + tid];
            float f;
            L += scale_sum(ml[w * R + tid], x == NEG_INF ? x : x - M, f);
            mm[w * R + tid] = f;
        }
        if (record == -2) cpart[R * D + tid] = M, cpart[R * D + R + tid] = L;
        else if (record >= 0)
            *reinterpret_cast<float2*>(p.part_ml + (record * C::R + tid) * 2) = make_float2(M, L);
        tot[tid] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();
    for (int idx = tid; idx < R * (D / 4); idx += 128) {
        const int r = idx / (D / 4);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 v = macc[w * R * (D / 4) + (idx ^ mix(r))];
            const float f = mm[w * R + r];
            a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
        }
        if (record == -2) {
            reinterpret_cast<float4*>(cpart)[idx] = a;
        } else if (record >= 0) {
            reinterpret_cast<float4*>(p.part_acc + record * C::R * D)[idx] = a;
        } else {
            store4(p.out, row_off(r) + idx % (D / 4) * 4, a, tot[r], p.out_dtype);
        }
    }
    if (record == -2) {
        // the cluster's partitions, through distributed shared memory: each CTA
        // finishes a share of the outputs
        cluster_sync_release_acquire();
        const int part = (int)blockIdx.x % p.cluster;
        const uint32_t cp = smem_u32(cpart);
        const int P = p.cluster, share = (R * (D / 4) + P - 1) / P;
        const int end = min((part + 1) * share, R * (D / 4));
        uint32_t base[kMaxClusterParts];
#pragma unroll
        for (int x = 0; x < kMaxClusterParts; ++x) base[x] = map_cluster_rank(cp, (uint32_t)(x < P ? x : 0));
        for (int idx = part * share + tid; idx < end; idx += 128) {
            const int r = idx / (D / 4);
            float m[kMaxClusterParts], l[kMaxClusterParts], M = NEG_INF;
            float4 a[kMaxClusterParts];
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) {
                    m[x] = ld_cluster_f32(base[x] + 4u * (R * D + r));
                    l[x] = ld_cluster_f32(base[x] + 4u * (R * D + R + r));
                    a[x] = ld_cluster_v4f32(base[x] + 16u * idx);
                }
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) M = fmaxf(M, m[x]);
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f;
#pragma unroll
            for (int x = 0; x < kMaxClusterParts; ++x)
                if (x < P) {  // (0 * NaN: a row of NaN stays one)
                    float f;
                    L += scale_sum(l[x], m[x] == NEG_INF ? NEG_INF : m[x] - M, f);
                    A.x = fmaf(f, a[x].x, A.x), A.y = fmaf(f, a[x].y, A.y);
                    A.z = fmaf(f, a[x].z, A.z), A.w = fmaf(f, a[x].w, A.w);
                }
            store4(p.out, row_off(r) + idx % (D / 4) * 4, A, L == 0.f ? 0.f : 1.f / L, p.out_dtype);
        }
        cluster_sync_relaxed();  // no CTA leaves while others read its shared memory
    }
    };

    // ---- the CTA's segments: those of its run, or its unit's one (the walk's state
    // stays in shared memory: in registers it spilled) ----
    if (p.balanced && run[0] >= run[1]) return;
    for (;;) {
        int b, x, k0, k1;
        long long record = -1;
        if (p.balanced) {
            b = *run_b;
            const long long base = run[2], at = run[4];
            const int n = steps_of(b);
            const int xg = (int)((at - base) / n), member = (int)blockIdx.x % p.group_size;
            x = xg * p.group_size + member;
            k0 = (int)(at - base - (long long)xg * n);
            k1 = (int)min((long long)n, k0 + (run[1] - at));
            if (k0 > 0 || k1 < n) record = blockIdx.x * 2ll + (at == run[0] ? 0 : 1);
            if (k0 == 0 && tid == 0 && x < per_seq) {
                // where the join finds the unit's pieces: group g has the steps from
                // floor(g total / groups) on
                const long long first = base + (long long)xg * n, groups = gridDim.x / p.group_size;
                PieceDesc d;
                d.first_group = (int)blockIdx.x / p.group_size;
                d.last_group = (int)(((first + n) * groups - 1) / run[3]);
                d.first_record = first == run[0] ? 0 : 1;
                d.member = member;
                d.total = run[3];
                p.part_desc[(size_t)b * per_seq + x] = d;
            }
        } else {
            const long long u = blockIdx.x / p.cluster;
            const int part = (int)blockIdx.x % p.cluster;
            b = (int)(u / per_seq);
            x = (int)(u % per_seq);
            const int n = steps_of(b);
            k0 = min(part * p.part_steps, n);
            k1 = p.cluster > 1 ? min(k0 + p.part_steps, n) : n;
            if (p.cluster > 1) record = -2;
        }
        if (x < per_seq && !aborted) segment(b, x / p.chunks, x % p.chunks, k0, k1, record);
        if (!p.balanced) return;
        // the rings are free again; after a timeout the walk goes on without its
        // segments, so that the join finds every unit's descriptor
        aborted = __syncthreads_or(aborted);
        if (tid == 0) {
            run[4] += k1 - k0;
            const long long whole = (long long)steps_of(b) * p.unit_groups;
            if (run[4] - run[2] >= whole) run[2] += whole, *run_b = b + 1;
        }
        __syncthreads();
        if (run[4] >= run[1]) return;
    }
}

// Joins the pieces of cut units: with each piece's (m, l, acc),
//     out = sum 2^(m - M) acc / sum 2^(m - M) l.
// A thread takes four elements of a row; SHARES threads share the pieces (eight
// where a few units lie in seven runs and more, else one).  Bound by the latency of
// its steps: the unit's descriptor, then statistics and sums.
constexpr int kKv8JoinThreads = 256;

template <int D, int RT, int SHARES>
__global__ void __launch_bounds__(kKv8JoinThreads) kv8_join_kernel(const Kv8Params p, int groups) {
    constexpr int PER = kKv8JoinThreads / SHARES, LANES = D / 4, AHEAD = 4;
    __shared__ float sums[SHARES][6][PER];
    grid_dependency_wait();
    grid_launch_dependents();
    const PieceDesc d = p.part_desc[blockIdx.x];
    if (d.first_group == d.last_group) return;  // whole: written already
    const int u = blockIdx.x, chunk = u % p.chunks, kvh = u / p.chunks % p.num_kv_heads;
    const int b = u / (p.chunks * p.num_kv_heads), qi0 = chunk * p.q_chunk;
    const int R = min(p.q_chunk, p.q_len - qi0) * p.group;
    const int share = threadIdx.x / PER, at = blockIdx.y * PER + threadIdx.x % PER;
    const int r = at / LANES, col = at % LANES * 4;
    const int pieces = r < R ? d.last_group - d.first_group + 1 : 0;
    float M = -INFINITY, L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int x0 = share; x0 < pieces; x0 += SHARES * AHEAD) {
        float2 ml[AHEAD];
        float4 y[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int x = x0 + k * SHARES;
            const long long g = d.first_group + x;
            ml[k] = make_float2(-INFINITY, 0.f);
            y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            // (a group without steps has no record)
            if (x < pieces && g * d.total / groups != (g + 1) * d.total / groups) {
                const long long row =
                    ((g * p.group_size + d.member) * 2 + (x == 0 ? d.first_record : 0)) * RT + r;
                ml[k] = *reinterpret_cast<const float2*>(p.part_ml + row * 2);
                y[k] = *reinterpret_cast<const float4*>(p.part_acc + row * D + col);
            }
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) m = fmaxf(m, ml[k].x);
        float f;
        L = scale_sum(L, M == -INFINITY ? M : M - m, f);
        M = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] *= f;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            float w;  // (0 * NaN: a row of NaN stays one)
            L += scale_sum(ml[k].y, ml[k].x == -INFINITY ? ml[k].x : ml[k].x - m, w);
            a[0] = fmaf(w, y[k].x, a[0]), a[1] = fmaf(w, y[k].y, a[1]);
            a[2] = fmaf(w, y[k].z, a[2]), a[3] = fmaf(w, y[k].w, a[3]);
        }
    }
    if constexpr (SHARES > 1) {
        const int t = threadIdx.x % PER;
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[share][i][t] = a[i];
        sums[share][4][t] = M;
        sums[share][5][t] = L;
        __syncthreads();
        if (share != 0) return;
#pragma unroll
        for (int k = 1; k < SHARES; ++k) M = fmaxf(M, sums[k][4][t]);
        L = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = 0.f;
#pragma unroll
        for (int k = 0; k < SHARES; ++k) {
            const float m = sums[k][4][t];
            float w;
            L += scale_sum(sums[k][5][t], m == -INFINITY ? m : m - M, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = fmaf(w, sums[k][i][t], a[i]);
        }
    }
    if (r >= R) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t o = (((size_t)b * p.q_len + qi0 + r / p.group) * p.num_heads + kvh * p.group + r % p.group) * D + col;
    store4(p.out, o, make_float4(a[0], a[1], a[2], a[3]), inv, p.out_dtype);
}

template <int D, int BS, int NR, bool HL>
cudaError_t launch_kv8_inst(const Kv8Launch& L, cudaStream_t stream) {
    static AttrFlags raised;
    auto kern = kv8_kernel<D, BS, NR, HL>;
    cudaError_t e = raise_smem_limit_once(kern, raised);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = L.grid;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = Kv8Cfg<D, BS, NR>::SMEM;
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

template <int D, int NR>
cudaError_t launch_kv8_join(const Kv8Launch& L, cudaStream_t stream) {
    const int groups = (int)L.grid.x / L.p.group_size;
    const bool shared = (long long)L.units * 6 < L.grid.x;  // seven pieces and more to a unit
    const int per = kKv8JoinThreads / (shared ? 8 : 1), rows = L.p.q_chunk * L.p.group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.units, (unsigned)((rows * (D / 4) + per - 1) / per));
    cfg.blockDim = dim3(kKv8JoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return shared ? cudaLaunchKernelEx(&cfg, kv8_join_kernel<D, NR * 8, 8>, L.p, groups)
                  : cudaLaunchKernelEx(&cfg, kv8_join_kernel<D, NR * 8, 1>, L.p, groups);
}

template <int D, int NR>
cudaError_t launch_kv8_for(const Kv8Launch& L, cudaStream_t stream) {
    const bool two = L.p.out_dtype != PA_BF16;
    const cudaError_t e =
        L.block_size == 16
            ? (two ? launch_kv8_inst<D, 16, NR, true>(L, stream) : launch_kv8_inst<D, 16, NR, false>(L, stream))
            : (two ? launch_kv8_inst<D, 32, NR, true>(L, stream) : launch_kv8_inst<D, 32, NR, false>(L, stream));
    return e != cudaSuccess || !L.p.balanced ? e : launch_kv8_join<D, NR>(L, stream);
}

// Resident CTAs per SM of an instantiation (pages of 16 and 32 alike).
template <int D, int NR>
constexpr int kv8_ctas = Kv8Cfg<D, 16, NR>::CTAS;

}  // namespace pa
