// Attention over the latent cache on the Blackwell tensor cores (tcgen05).
//
// The mathematics: with c_t the vector of token t (latent part of R elements,
// positional part of 64) and q_r a query row (query token, head),
//     out_r = sum_t 2^(s_rt - m_r) c_t[:R] / sum_t 2^(s_rt - m_r),  s_rt = scale log2(e) q_r . c_t.
// All heads share the tokens, so that one read of a token serves every row.
//
// Both products are formed transposed, tokens and value elements in the MMAs' M
// and query rows in their N:
//     S^T [64 tokens x N] = C [64 x (R + 64)] Q^T,      M = 64
//     O^T [R x N]        += C[:, :R]^T [R x 64] P^T,    M = 128, R / 128 of them
// (P^T of bf16 weights as [64 x 2N], their high and low parts side by side)
// so that the tile of tokens that TMA has put into shared memory is the A
// operand of both (K-major for the first, M-major for the second), 16, 32 or
// 64 rows cost what they are instead of a tile of 128, and O^T of 64 rows takes
// 256 columns of tensor memory where O would take all 512 (R = 512).
//
// A CTA (one to an SM) takes a run of the flattened (sequence, group of row tiles,
// 64-token tile) order, the same number of tiles as every other CTA whatever the
// lengths: a run is a few segments of one sequence each.  A segment that is a
// sequence whole writes its output; of one that is cut the pieces' (m, l, O) go to
// the workspace and join_latent_kernel joins them.  The CTAs of a group (adjacent
// blocks) walk the same tokens for different row tiles, the second reader from L2.
// Roles:
//   warp 0      copies: Q of a segment, and the tiles in rings of slots: pairs of
//               64-element column blocks (16 KB) and the positional block (8 KB);
//               a slot is loaded again as soon as its own MMAs are done
//   warp 1      issues S^T of a tile as its slots land, a tile ahead
//   warp 2      issues O^T += C^T P^T as P lands in shared memory
//   warp 3      owns tensor memory
//   warps 4-11  softmax, a warpgroup to half of the rows: a thread has two tokens and
//               N / 8 rows; P^T to shared memory, rescales of O^T, the output
// The running maxima move only where a score is 2^8 above them: a tile then costs
// one vote of the warpgroup, no reduction over tokens.  The normalisers are
// summed a thread's tokens at a time and joined at the segment's end.
//
// Weights meet the values in 16 bits, the MMA's operands having one type.  fp16's 11
// bits (at most 2^-11 off, as an fp16 output) are held once, the normaliser summing
// the rounded ones.  bf16's 8 bits would put 2^-8 of a weight on a bf16 output's own
// 2^-8 (16 heads, 64 ragged sequences: 0.0013 off where the output's rounding is
// 0.0011), so those are held in two parts, 16 bits: the low parts are N more columns
// of the same MMAs, summed at the end.  Without and with them (4 x 65,536 tokens): 16
// heads 63.3 and 63.4 us, 32 65.5 and 66.5; 128 heads at latent_dim 256 72.4 and
// 73.7, at 128 57.5 and 61.5.  At latent_dim 512 with 64 rows tensor memory has no 256
// columns more, and low parts by MMAs of their own into the same ones took 132 us
// where one part takes 103, the error staying at 0.0017 (the output's rounding):
// there bf16 weights are rounded once.
//
// Bounds (latent_dim 512; isolated MMAs: M = 64, N = 64 30 cycles, N = 16 22;
// M = 128 44 and 36).  With 64 rows shared memory's 128 bytes a cycle: a tile's S^T
// reads 147 KB of it and O^T 98, its load writes 72, 2480 cycles in all; a tile takes 2950.
// 4 sequences of 65,536 tokens, 128 heads (302 MB, 73 GFLOP): 102 us, 715
// TFLOP/s; 32 of 4001 .. 4096 with two query tokens: 111 us.  With 16 rows DRAM: 64
// sequences of 1 .. 8192 tokens, 16 heads (304 MB): 68 us, 4.5 TB/s, 5.4 between the
// first tile (4 us, when all SMs start at once) and the pieces' ends (5 us with the join).
#pragma once

#include <type_traits>

#include "pa_device.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kLatentTile = 64;      // tokens of a tile
constexpr int kLatentThreads = 384;
constexpr int kLatentP = 64;         // positional elements

template <int R, int N, bool BF>
struct LatentCfg {
    static constexpr int MB = R / 128;                         // value blocks of a tile
    static constexpr int PARTS = BF && (R < 512 || N < 64) ? 2 : 1;  // of a weight
    static constexpr int ON = N * PARTS;                       // columns of P^T and of a value block of O^T
    static constexpr uint32_t Q_BYTES = N * (R + kLatentP) * 2u;
    static constexpr int PBUF = (R == 512 && N == 64) ? 1 : 2;  // P^T buffers
    static constexpr uint32_t P_BLOCK = kLatentTile * 128u;    // 64 columns
    static constexpr uint32_t P_BYTES = (ON + 63) / 64 * P_BLOCK;
    static constexpr uint32_t PAIR = 2u * kLatentTile * 128u, ROPE = kLatentTile * 128u;
    static constexpr uint32_t BUDGET = 229376u;                // leaves 2 KB for barriers and statistics
    // as many tiles' worth of slots as fit, whole pairs
    static constexpr uint32_t TILE = MB * PAIR + ROPE;
    static constexpr uint32_t FREE = BUDGET - Q_BYTES - PBUF * P_BYTES;
    static constexpr int NR = FREE / TILE > 6 ? 6 : FREE / TILE;                 // positional slots
    static constexpr int NP_RAW = (FREE - NR * ROPE) / PAIR;
    static constexpr int NP = NP_RAW > 12 ? 12 : NP_RAW;       // pair slots
    static constexpr uint32_t P_OFF = Q_BYTES;
    static constexpr uint32_t ROPE_OFF = P_OFF + PBUF * P_BYTES;
    static constexpr uint32_t PAIR_OFF = ROPE_OFF + NR * ROPE;
    static constexpr uint32_t STAT_OFF = PAIR_OFF + NP * PAIR;  // wmax [4][N], fac [N], lim [N]
    static constexpr uint32_t LIVE_OFF = STAT_OFF + 6 * N * 4;  // [16] 64-bit masks
    static constexpr uint32_t BAR_OFF = LIVE_OFF + 16 * 8;
    static constexpr int BARS = 2 * NP + 2 * NR + 15;
    static constexpr uint32_t MISC_OFF = BAR_OFF + BARS * 8;    // tmem address, abort flag, run
    static constexpr uint32_t SMEM = MISC_OFF + 64 + kSmemAlignSlack;
    static_assert(SMEM <= 227u * 1024u, "shared memory");
    static_assert(NP >= 2 * MB && NR >= 2, "two tiles in flight");
    static constexpr uint32_t COLS_RAW = 2 * N + MB * ON;
    static constexpr uint32_t COLS = COLS_RAW <= 64 ? 64 : COLS_RAW <= 128 ? 128 : COLS_RAW <= 256 ? 256 : 512;
};

namespace tc {

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// mma_ss with the descriptors as words.
__device__ __forceinline__ void mma_parts(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Lanes base .. base + 15 of the warp's quarter, 8 J consecutive columns: register
// 4 j + 2 h + e of lane l holds lane base + l / 4 + 8 h, column 8 j + 2 (l % 4) + e.
template <int J>
__device__ __forceinline__ void ld_16x256b(uint32_t taddr, float* r);
template <>
__device__ __forceinline__ void ld_16x256b<1>(uint32_t taddr, float* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
                 : "r"(taddr)
                 : "memory");
}
template <>
__device__ __forceinline__ void ld_16x256b<2>(uint32_t taddr, float* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
                   "=f"(r[7])
                 : "r"(taddr)
                 : "memory");
}
template <>
__device__ __forceinline__ void ld_16x256b<4>(uint32_t taddr, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ld_32x32b_x8(uint32_t taddr, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
                   "=f"(r[7])
                 : "r"(taddr)
                 : "memory");
}

}  // namespace tc

// Has phase `parity` of an mbarrier completed?  (Looks once, does not wait.)
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// Brings `bytes` (a multiple of 16) to L2 ahead of their load.
__device__ __forceinline__ void l2_prefetch(const void* at, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(at)), "r"(bytes)
                 : "memory");
}

// 2-D tiled TMA load; completion is signalled on `bar` as transaction bytes.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// A softmax warpgroup's barrier (id 1 or 2), and whether any of its threads votes yes.
__device__ __forceinline__ void group_sync(int id) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_any(int id, bool vote) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)vote), "r"(id) : "memory");
    return r != 0;
}

// Eight rows' values of the lane's element (f: their factors) become eight
// consecutive elements of row `lane % 8`, packed: three exchanges among eight lanes.
template <typename T>
__device__ __forceinline__ uint4 transpose8(const float (&v)[8], int lane) {
    uint32_t a[4], b[2][2];
    const bool o1 = lane & 1, o2 = lane & 2, o4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows 2 i + (lane & 1), elements lane & ~1 and the next
        const float got = __shfl_xor_sync(kFullMask, o1 ? v[2 * i] : v[2 * i + 1], 1);
        a[i] = o1 ? Mma<T>::pack(got, v[2 * i + 1]) : Mma<T>::pack(v[2 * i], got);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // rows 4 i + (lane & 3), four elements
        const uint32_t got = __shfl_xor_sync(kFullMask, o2 ? a[2 * i] : a[2 * i + 1], 2);
        b[i][0] = o2 ? got : a[2 * i];
        b[i][1] = o2 ? a[2 * i + 1] : got;
    }
    const uint32_t g0 = __shfl_xor_sync(kFullMask, o4 ? b[0][0] : b[1][0], 4);
    const uint32_t g1 = __shfl_xor_sync(kFullMask, o4 ? b[0][1] : b[1][1], 4);
    return o4 ? make_uint4(g0, g1, b[1][0], b[1][1]) : make_uint4(b[0][0], b[0][1], g0, g1);
}

// Tiles of a sequence: those of its attended tokens, one (with none) for an
// empty one, whose output is zeros.
__device__ __forceinline__ int latent_reach(const LatentParams& p, int b) {
    return min(min(max(__ldg(p.context_lens + b), 0), p.max_blocks * p.block_size), p.token_limit);
}
__device__ __forceinline__ int latent_tiles(const LatentParams& p, int b) {
    return max((latent_reach(p, b) + kLatentTile - 1) / kLatentTile, 1);
}

// One CTA's part of the work: tiles [k0, k1) of row tile rt of sequence b, of n.
struct LatentSeg {
    int b, rt, k0, k1, n;
    long long first;  // flat position of the (sequence, row tile group)'s tile 0
};

template <int R, int N, typename T>
__global__ void __launch_bounds__(kLatentThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_q,
                  const LatentParams p) {
    constexpr bool kBF = std::is_same<T, __nv_bfloat16>::value;
    using C = LatentCfg<R, N, kBF>;
    constexpr int MB = C::MB, NP = C::NP, NR = C::NR, PBUF = C::PBUF, ON = C::ON, PARTS = C::PARTS;
    constexpr float NEG_INF = -INFINITY;
    constexpr float kSlack = 8.f, kLift = kBF ? 0.f : kHalfLift;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlignSlack - 1)) & ~uintptr_t(kSmemAlignSlack - 1));
    const uint32_t sbase = smem_u32(smem);
    float* wmax = reinterpret_cast<float*>(smem + C::STAT_OFF);  // [4][N]
    float* fac = wmax + 4 * N;                                   // [N]
    int32_t* lim = reinterpret_cast<int32_t*>(fac + N);          // [N]
    uint64_t* live = reinterpret_cast<uint64_t*>(smem + C::LIVE_OFF);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t *pair_full = bar, *pair_free = pair_full + NP, *rope_full = pair_free + NP,
             *rope_free = rope_full + NR, *s_full = rope_free + NR, *s_free = s_full + 2,
             *p_full = s_free + 2, *pv_done = p_full + 2, *q_full = pv_done + 2, *q_free = q_full + 1,
             *o_free = q_free + 1, *final_s = o_free + 1, *final_o = final_s + 1,
             *live_full = final_o + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    // start, end, flat position of the first sequence's tiles, total
    long long* run = reinterpret_cast<long long*>(smem + C::MISC_OFF + 8);
    int32_t* run_b = reinterpret_cast<int32_t*>(run + 4);  // the first sequence; 1: no run, units in turn

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int BS = p.block_size, rows = p.q_len * p.num_heads;
    const int member = (int)blockIdx.x % p.group_size, group = (int)blockIdx.x / p.group_size;

    if (tid == 0) {
        for (int i = 0; i < NP; ++i) mbar_init(smem_u32(pair_full + i), 1), mbar_init(smem_u32(pair_free + i), 1);
        for (int i = 0; i < NR; ++i) mbar_init(smem_u32(rope_full + i), 1), mbar_init(smem_u32(rope_free + i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(s_full + i), 1);
            mbar_init(smem_u32(s_free + i), 8);  // a lane of each softmax warp
            mbar_init(smem_u32(p_full + i), 8);
            mbar_init(smem_u32(pv_done + i), 1);
            mbar_init(smem_u32(live_full + i), 1);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_free), 1);
        mbar_init(smem_u32(o_free), 8);
        mbar_init(smem_u32(final_s), 1);
        mbar_init(smem_u32(final_o), 1);
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tmap_c);
        prefetch_tensormap(&tmap_q);
    }
    if (warp == 3) {
        tc::tmem_alloc(smem_u32(tmem_slot), C::COLS);
        tc::tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the CTA's run [start, end) of the flat order (sequence, group of row
    // tiles, tile), where it begins ----
    if (warp == 0) {
        if (p.balanced) {
            long long w = 0;
            int most = 0;
            for (int b = lane; b < p.batch; b += 32) {
                const int n = latent_tiles(p, b);
                w += n;
                most = max(most, n);
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) {
                w += __shfl_xor_sync(kFullMask, w, m);
                most = max(most, __shfl_xor_sync(kFullMask, most, m));
            }
            w *= p.row_groups;
            const long long groups = gridDim.x / p.group_size, units = (long long)p.batch * p.row_groups;
            // Sequences of about one length, about as many as groups: each whole to a
            // group in turn, where that is at most a cut's own cost longer (its
            // partial results and the join, measured in tiles).
            constexpr int kCut = N == 64 ? 12 : 4;
            const bool in_turn = (units + groups - 1) / groups * most * groups <= w + kCut * groups;
            const long long start = group * w / groups, end = (group + 1) * w / groups;
            int b = 0;
            long long base = 0;
            while (start < end) {
                const int bb = b + lane;
                const long long v = bb < p.batch ? (long long)latent_tiles(p, bb) * p.row_groups : 0;
                long long incl = v;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const long long o = __shfl_up_sync(kFullMask, incl, m);
                    if (lane >= m) incl += o;
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
            if (lane == 0) run[0] = start, run[1] = end, run[2] = base, run[3] = w, run_b[0] = b, run_b[1] = in_turn;
        } else if (lane == 0) {
            run_b[1] = 1;  // a group to each (sequence, row tile group)
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const long long run_start = run[0], run_end = run[1];

    // f(segment, its number): the CTA's segments in order, until f returns false.
    // Every role walks them alike.
    const bool in_turn = run_b[1] != 0;
    auto for_segments = [&](auto&& f) {
        const long long groups = gridDim.x / p.group_size, units = (long long)p.batch * p.row_groups;
        int b = run_b[0], s = 0;
        long long base = run[2], at = in_turn ? group : run_start;
        while (at < (in_turn ? units : run_end)) {
            LatentSeg g;
            int x;
            if (in_turn) {
                g.b = (int)(at / p.row_groups);
                x = (int)(at % p.row_groups);
                g.n = g.k1 = latent_tiles(p, g.b);
                g.k0 = 0;
                g.first = 0;
                at += groups;
            } else {
                g.b = b;
                g.n = latent_tiles(p, b);
                x = (int)((at - base) / g.n);
                g.k0 = (int)(at - base - (long long)x * g.n);
                g.k1 = (int)min((long long)g.n, g.k0 + (run_end - at));
                g.first = base + (long long)x * g.n;
                at += g.k1 - g.k0;
                if (at - base >= (long long)g.n * p.row_groups) base += (long long)g.n * p.row_groups, ++b;
            }
            g.rt = x * p.group_size + member;
            if (g.rt * N >= rows) continue;  // (a group's row tiles past the last)
            if (!f(g, s++)) return;
        }
    };
    auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        const bool ok = mbar_wait_bounded(smem_u32(b), parity, p.timeout_ns);
        if (!ok) {
            record_error(p.err, PA_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        return ok;
    };
    // a value that is the same in every lane, in a uniform register
    auto uniform = [](uint32_t x) -> uint32_t { return __shfl_sync(kFullMask, x, 0); };
    constexpr int kType = kBF ? 1 : 0;
    // high words of the operands' descriptors (8-row groups 1024 bytes apart, version 1,
    // 128-byte swizzle); a low word is the address / 16 and, M- / N-major, the distance
    // of the 64-element blocks above it
    constexpr uint32_t kDesc = (1024u >> 4) | (1u << 14) | ((uint32_t)tc::kSwizzle128B << 29);

    if (warp == 0) {
        // ================= copies =================
        const int PG = kLatentTile / BS;  // pages of a tile
        int tile = 0, pairs = 0, segs = 0;
        for_segments([&](const LatentSeg& g, int s) {
            const int32_t* row = p.block_tables + (size_t)g.b * p.max_blocks;
            const int npages = (latent_reach(p, g.b) + BS - 1) / BS;
            // lane l < PG: the entry of page l of the tile, one tile ahead
            auto fetch = [&](int k) -> int {
                return lane < PG ? page_phys(row, k * PG + lane, npages, p.num_blocks) : -1;
            };
            int next = fetch(g.k0), ahead = fetch(g.k0 + 1);
            // (a later segment's queries behind its first tile, whose slots are free earlier)
            auto load_q = [&]() -> bool {
                if (s > 0 && !__all_sync(kFullMask, wait(q_free, (s - 1) & 1))) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_u32(q_full), C::Q_BYTES);
                    for (int c = 0; c < (R + kLatentP) / 64; ++c)
                        tma_load_2d(sbase + c * N * 128, &tmap_q, c * 64, g.b * rows + g.rt * N, smem_u32(q_full));
                }
                segs = s + 1;
                return true;
            };
            if (s == 0 && !load_q()) return false;
            const uint64_t policy = p.group_size > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
            for (int k = g.k0; k < g.k1 && !*abort_flag; ++k, ++tile) {
                const int phys = next;
                next = ahead;
                if (k + 2 < g.k1) ahead = fetch(k + 2);
                // the next tile's pages to L2, each in one piece: their slots are free
                // late, and the loads by column block read 128 bytes a row
                if (member == 0 && k + 1 < g.k1 && next >= 0)
                    l2_prefetch(static_cast<const T*>(p.cache) + (size_t)next * BS * (R + kLatentP),
                                (uint32_t)BS * (R + kLatentP) * 2u);
                const unsigned on = __ballot_sync(kFullMask, phys >= 0);
                // one slot: `blocks` column blocks from element `col` on
                auto load = [&](uint64_t* full, uint32_t dst, int col, int blocks) {
                    if (lane == 0) {
                        if (on) mbar_arrive_expect_tx(smem_u32(full), (uint32_t)__popc(on) * BS * 128u * blocks);
                        else mbar_arrive(smem_u32(full));
                    }
                    __syncwarp();
                    if (phys >= 0)
                        for (int c = 0; c < blocks; ++c)
                            tma_load_4d(dst + c * C::ROPE + lane * BS * 128, &tmap_c, col + c * 64, 0, phys, 0,
                                        smem_u32(full), policy);
                };
                const int rs = tile % NR;
                if (tile >= NR && !__all_sync(kFullMask, wait(rope_free + rs, (tile / NR - 1) & 1))) return false;
                if (lane == 0) {
                    // the tile's tokens that a page holds
                    uint64_t m = 0;
                    for (int l = 0; l < PG; ++l)
                        if (on >> l & 1) m |= (BS == 64 ? ~0ull : (1ull << BS) - 1) << (l * BS);
                    live[tile & 15] = m;
                }
                load(rope_full + rs, sbase + C::ROPE_OFF + rs * C::ROPE, R, 1);
                for (int m = 0; m < MB; ++m, ++pairs) {
                    const int ps = pairs % NP;
                    if (pairs >= NP && !__all_sync(kFullMask, wait(pair_free + ps, (pairs / NP - 1) & 1)))
                        return false;
                    load(pair_full + ps, sbase + C::PAIR_OFF + ps * C::PAIR, m * 128, 2);
                }
                if (s > 0 && k == g.k0 && !load_q()) return false;
            }
            return !*abort_flag;
        });
        if (*abort_flag && lane == 0) {
            // copies in flight land before the CTA ends
            for (int k = max(0, pairs - NP); k < pairs; ++k)
                (void)mbar_wait_bounded(smem_u32(pair_full + k % NP), (k / NP) & 1, p.timeout_ns);
            for (int k = max(0, tile - NR); k <= tile; ++k)
                (void)mbar_wait_bounded(smem_u32(rope_full + k % NR), (k / NR) & 1, p.timeout_ns);
            if (segs) (void)mbar_wait_bounded(smem_u32(q_full), (segs - 1) & 1, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= S^T = C Q^T =================
        // (the whole warp walks, so that descriptors stay in uniform registers;
        // one lane issues: with one lane walking, an MMA took 94 cycles to issue)
        constexpr uint32_t idesc = tc::idesc_f16(kType, false, 64, N);
        const uint32_t qbase = uniform(sbase >> 4);
        const int watch = lane < 2 + MB ? lane : 0;
        const bool one = tc::elect_one();
        int tile = 0, pairs = 0;
        for_segments([&](const LatentSeg& g, int s) {
            if (!__all_sync(kFullMask, wait(q_full, s & 1))) return false;
            for (int k = g.k0; k < g.k1; ++k, ++tile) {
                // operand addresses / 16, the same in every lane
                const int rs = tile % NR;
                const uint32_t rope = uniform((sbase + C::ROPE_OFF + rs * C::ROPE) >> 4);
                uint32_t at[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    at[m] = uniform((sbase + C::PAIR_OFF + (pairs + m) % NP * C::PAIR) >> 4);
                const uint32_t d = uniform(tmem + (tile & 1) * N);
                // lane 0 watches the score buffer, lane 1 the positional slot, lane 2 + m
                // pair m: a tile whose slots have all landed costs one look
                const int mine = (pairs + watch - 2) % NP;
                const uint32_t bar_at = smem_u32(watch == 0   ? s_free + (tile & 1)
                                                 : watch == 1 ? rope_full + rs
                                                              : pair_full + mine);
                const uint32_t parity = watch == 0   ? (tile / 2 - 1) & 1
                                        : watch == 1 ? (tile / NR) & 1
                                                     : ((pairs + watch - 2) / NP) & 1;
                uint32_t ready = 0;
                auto need = [&](uint32_t bits) -> bool {
                    if ((ready & bits) == bits) return true;
                    uint64_t start = 0;
                    for (uint32_t it = 1;; ++it) {
                        ready = __ballot_sync(kFullMask, (watch == 0 && tile < 2) || mbar_test_wait(bar_at, parity));
                        if ((ready & bits) == bits) break;
                        if ((it & 255u) == 0) {
                            const uint64_t now = global_timer_ns();
                            if (!start) start = now;
                            if (__any_sync(kFullMask, *abort_flag || now - start > p.timeout_ns)) {
                                record_error(p.err, PA_ERR_TIMEOUT);
                                *abort_flag = 1;
                                return false;
                            }
                        }
                    }
                    __syncwarp();
                    tc::fence_after_sync();
                    return true;
                };
                if (!need(3)) return false;
                auto block = [&](uint32_t a, int c, bool first) {  // 64 elements
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma_parts(d, a + kk * 2 + (1u << 16), kDesc, qbase + c * N * 8 + kk * 2 + (1u << 16),
                                      kDesc, idesc, !(first && kk == 0));
                };
                if (one) {
                    block(rope, R / 64, true);
                    mbar_arrive(smem_u32(live_full + (tile & 1)));  // hands the tile's mask on
                }
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    if (!need(4u << m)) return false;
                    if (one) {
                        block(at[m], 2 * m, false);
                        block(at[m] + (C::ROPE >> 4), 2 * m + 1, false);
                    }
                }
                pairs += MB;
                if (one) {
                    tc::commit(smem_u32(rope_free + rs));
                    tc::commit(smem_u32(s_full + (tile & 1)));
                }
                __syncwarp();
            }
            if (one) tc::commit(smem_u32(q_free));
            __syncwarp();
            return true;
        });
        if (one) {
            tc::commit(smem_u32(final_s));
            (void)mbar_wait_bounded(smem_u32(final_s), 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ================= O^T += C^T P^T =================
        // A and B both M- / N-major: elements and rows contiguous, tokens the rows of 128 bytes
        constexpr uint32_t idesc = tc::idesc_f16(kType, true, 128, ON) | (1u << 15);
        const uint32_t otmem = uniform(tmem + 2 * N);
        const bool one = tc::elect_one();
        int tile = 0, pairs = 0;
        for_segments([&](const LatentSeg& g, int s) {
            // the last segment's output is read
            if (s > 0 && !__all_sync(kFullMask, wait(o_free, (s - 1) & 1))) return false;
            for (int k = g.k0; k < g.k1; ++k, ++tile) {
                const int pb = tile % PBUF;
                const uint32_t pt = uniform((sbase + C::P_OFF + pb * C::P_BYTES) >> 4);
                uint32_t at[MB], freed[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int ps = (pairs + m) % NP;
                    at[m] = uniform((sbase + C::PAIR_OFF + ps * C::PAIR) >> 4);
                    freed[m] = uniform(smem_u32(pair_free + ps));
                }
                pairs += MB;
                if (!__all_sync(kFullMask, !*abort_flag && wait(p_full + pb, (tile / PBUF) & 1))) return false;
                tc::fence_after_sync();
                const bool first = k == g.k0;
                if (one) {
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 16 tokens
                            tc::mma_parts(otmem + m * ON, at[m] + kk * 128 + (C::ROPE >> 4 << 16), kDesc,
                                          pt + kk * 128 + (C::P_BLOCK >> 4 << 16), kDesc, idesc,
                                          !(first && kk == 0));
                        tc::commit(freed[m]);
                    }
                }
                if (one) tc::commit(smem_u32(pv_done + (tile & 1)));
                __syncwarp();
            }
            return true;
        });
        if (one) {
            tc::commit(smem_u32(final_o));
            (void)mbar_wait_bounded(smem_u32(final_o), 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ================= softmax =================
        constexpr int NC = N / 2, J = NC / 8;  // rows of a warpgroup, in groups of 8: a thread has two of each
        const int wg = (warp - 4) >> 2, w = warp & 3, id = 1 + wg;
        const int quarter = w << 21;           // lanes 32 w on; tokens 16 w on in lanes 32 w .. + 15
        const int tg = lane >> 2, tq = lane & 3, cb = wg * NC;
        int tile = 0, pairs = 0;
        for_segments([&](const LatentSeg& g, int s) {
            const int ctx = max(__ldg(p.context_lens + g.b), 0), reach = latent_reach(p, g.b);
            const int r0 = g.rt * N;
            group_sync(id);  // the last segment's statistics are read
            for (int c = cb + w * 32 + lane; c < cb + NC; c += 128)
                lim[c] = r0 + c < rows ? min(reach, ctx - p.q_len + (r0 + c) / p.num_heads + 1) : reach;
            const int least = min(reach, ctx - p.q_len + r0 / p.num_heads + 1);
            float ref[2 * J], sum[2 * J];      // reference exponents and normalisers of the thread's rows
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) ref[i] = NEG_INF, sum[i] = 0.f;
            for (int k = g.k0; k < g.k1; ++k, ++tile, pairs += MB) {
                const int t0 = k * kLatentTile;
                wait(s_full + (tile & 1), (tile / 2) & 1);
                wait(live_full + (tile & 1), (tile / 2) & 1);
                tc::fence_after_sync();
                float x[4 * J];
                tc::ld_16x256b<J>(tmem + quarter + (tile & 1) * N + cb, x);
                uint64_t valid = live[tile & 15];
                const bool aborted = *abort_flag;
                if (reach - t0 < kLatentTile) valid &= reach > t0 ? (1ull << (reach - t0)) - 1 : 0ull;
                const bool masked = valid != ~0ull || least < t0 + kLatentTile;
                tc::wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(s_free + (tile & 1)));
#pragma unroll
                for (int i = 0; i < 4 * J; ++i) x[i] *= p.qscale;
                if (masked) {
                    if (k == g.k0) group_sync(id);  // lim
#pragma unroll
                    for (int i = 0; i < 4 * J; ++i) {
                        const int t = w * 16 + tg + (i & 2) * 4, c = cb + (i >> 2) * 8 + tq * 2 + (i & 1);
                        if (!(valid >> t & 1) || t0 + t >= lim[c]) x[i] = NEG_INF;
                    }
                }
                float above = NEG_INF;
#pragma unroll
                for (int i = 0; i < 4 * J; ++i) above = fmaxf(above, x[i] - ref[(i >> 2) * 2 + (i & 1)]);
                // (an abort anywhere brings all of the warpgroup to the second vote)
                if (group_any(id, above > kSlack + kLift || aborted)) {
                    if (group_any(id, *abort_flag)) return false;
                    // some row's maximum has risen: the tile's maxima, new references
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        float v = fmaxf(x[(i >> 1) * 4 + (i & 1)], x[(i >> 1) * 4 + 2 + (i & 1)]);
                        v = fmaxf(v, __shfl_xor_sync(kFullMask, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(kFullMask, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(kFullMask, v, 16));
                        if (tg == 0) wmax[w * N + cb + (i >> 1) * 8 + tq * 2 + (i & 1)] = v;
                    }
                    group_sync(id);
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        const int c = cb + (i >> 1) * 8 + tq * 2 + (i & 1);
                        const float v = fmaxf(fmaxf(wmax[c], wmax[N + c]), fmaxf(wmax[2 * N + c], wmax[3 * N + c]));
                        const float to = fmaxf(ref[i], v - kLift);
                        const float f = to == ref[i] ? 1.f : fast_exp2(ref[i] - to);
                        if (w == 0 && tg == 0) fac[c] = f;
                        ref[i] = to;
                        sum[i] *= f;
                    }
                    if (k > g.k0) wait(pv_done + ((tile - 1) & 1), ((tile - 1) / 2) & 1);
                    group_sync(id);
                    if (k > g.k0) {
                        // O^T (elements in lanes, rows in columns) on the new references
                        tc::fence_after_sync();
                        for (int c0 = 0; c0 < MB * PARTS * NC; c0 += 8) {
                            const uint32_t at = tmem + quarter + (2 + c0 / NC) * N + cb + c0 % NC;
                            float o[8];
                            tc::ld_32x32b_x8(at, o);
                            tc::wait_ld();
                            uint32_t u[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(o[i] * fac[cb + c0 % NC + i]);
                            tc::st_32x32b_x8(at, u);
                        }
                        tc::wait_st();
                    }
                }
                // ---- weights, in 16 bits as they meet the values: rounded once, or in two parts ----
                uint32_t pk[2 * J], pl[PARTS == 2 ? 2 * J : 1];
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    // i: group i / 2, token tg or tg + 8; two neighbouring rows
                    const int a = (i >> 1) * 4 + (i & 1) * 2, r = (i >> 1) * 2;
                    float e0 = fast_exp2(x[a] - ref[r]), e1 = fast_exp2(x[a + 1] - ref[r + 1]);
                    if (masked) {  // (rows without a token so far: -inf less -inf)
                        if (x[a] == NEG_INF) e0 = 0.f;
                        if (x[a + 1] == NEG_INF) e1 = 0.f;
                    }
                    pk[i] = Mma<T>::pack(e0, e1);
                    float h0, h1;
                    Mma<T>::unpack(pk[i], h0, h1);
                    if constexpr (PARTS == 2) pl[i] = Mma<T>::pack(e0 - h0, e1 - h1);
                    else e0 = h0, e1 = h1;  // (the normaliser sums the rounded ones)
                    sum[r] += e0;
                    sum[r + 1] += e1;
                }
                // the buffer's last reader, O^T of PBUF tiles ago, is done
                if (tile >= PBUF) wait(pv_done + ((tile - PBUF) & 1), ((tile - PBUF) / 2) & 1);
                const uint32_t pt = sbase + C::P_OFF + (tile % PBUF) * C::P_BYTES;
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    const int t = w * 16 + tg + (i & 1) * 8;
                    const uint32_t at = pt + t * 128 + ((((cb >> 3) + (i >> 1)) ^ (t & 7)) << 4) + tq * 4;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pk[i]) : "memory");
                    if constexpr (PARTS == 2) {  // columns N on
                        const uint32_t lo = N == 64 ? at + C::P_BLOCK
                                                    : pt + t * 128 + (((((N + cb) >> 3) + (i >> 1)) ^ (t & 7)) << 4) + tq * 4;
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(lo), "r"(pl[i]) : "memory");
                    }
                }
                if (valid != ~0ull) {
                    // tokens without a page, or past the context: their rows must be
                    // finite for the product with weights of 0
                    for (int i = tid - 128; i < kLatentTile * 8 * 2 * MB; i += 256) {
                        const int t = (i >> 3) % kLatentTile, blk = (i >> 3) / kLatentTile;
                        if (!(valid >> t & 1))
                            *reinterpret_cast<uint4*>(smem + C::PAIR_OFF + ((pairs + blk / 2) % NP) * C::PAIR +
                                                      (blk & 1) * C::ROPE + t * 128 + (i & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + tile % PBUF));
            }
            // ---- the segment's output ----
            group_sync(id);
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                float v = sum[i];
                v += __shfl_xor_sync(kFullMask, v, 4);
                v += __shfl_xor_sync(kFullMask, v, 8);
                v += __shfl_xor_sync(kFullMask, v, 16);
                const int c = cb + (i >> 1) * 8 + tq * 2 + (i & 1);
                if (tg == 0) wmax[w * N + c] = v;
                if (w == 0 && tg == 0) fac[c] = ref[i];
            }
            wait(pv_done + ((tile - 1) & 1), ((tile - 1) / 2) & 1);
            if (group_any(id, *abort_flag)) return false;
            tc::fence_after_sync();
            const bool whole = g.k0 == 0 && g.k1 == g.n;
            const size_t rec = (size_t)blockIdx.x * 2 + (g.first + g.k0 == run_start ? 0 : 1);
            const int count = min(N, rows - r0);
            auto total = [&](int c) { return (wmax[c] + wmax[N + c]) + (wmax[2 * N + c] + wmax[3 * N + c]); };
            if (!whole)
                for (int c = cb + w * 32 + lane; c < cb + NC; c += 128)
                    *reinterpret_cast<float2*>(p.part_ml + (rec * N + c) * 2) = make_float2(fac[c], total(c));
            group_sync(id);
            for (int c = cb + w * 32 + lane; c < cb + NC; c += 128) {
                const float l = total(c);
                fac[c] = l == 0.f ? 0.f : 1.f / l;
            }
            group_sync(id);
            for (int m = 0; m < MB; ++m) {
#pragma unroll
                for (int c0 = 0; c0 < NC; c0 += 8) {
                    float o[8];
                    const uint32_t from = tmem + quarter + 2 * N + m * ON + cb + c0;
                    tc::ld_32x32b_x8(from, o);
                    if constexpr (PARTS == 2) {
                        float lo[8];
                        tc::ld_32x32b_x8(from + N, lo);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] += lo[i];
                    } else {
                        tc::wait_ld();
                    }
                    const int d = m * 128 + w * 32 + lane, c = cb + c0;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] *= fac[c + i];
                        const uint4 v = transpose8<T>(o, lane);
                        const int r = c + (lane & 7);
                        if (r < count)
                            *reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                                      ((size_t)g.b * rows + r0 + r) * R + (d & ~7)) = v;
                    } else {  // [element][row]: whole sectors a lane
                        st_global_v8(p.part_acc + (rec * R + d) * N + c, o);
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(o_free));
            return true;
        });
    }
    // ---- where the join finds the pieces of a (sequence, row tile): said by the
    // CTA that has its first tile ----
    if (p.balanced && warp == 3 && lane == 0) {
        const long long groups = gridDim.x / p.group_size, total = run[3];
        for_segments([&](const LatentSeg& g, int) {
            if (g.k0 == 0) {
                // group x has the tiles from floor(x total / groups) on
                PieceDesc d;
                d.first_group = group;
                d.last_group = in_turn ? group : (int)(((g.first + g.n) * groups - 1) / total);
                d.first_record = g.first == run_start ? 0 : 1;
                d.member = member;
                d.total = total;
                p.part_desc[(size_t)g.b * p.row_tiles + g.rt] = d;
            }
            return true;
        });
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, C::COLS);
}

// Joins the pieces of cut (sequence, row tile)s: with each piece's (m, l, O),
// out = sum 2^(m - M) O / sum 2^(m - M) l.  A thread takes a row and eight
// elements; neighbouring threads have neighbouring rows, as a piece's records lie
// ([element][row]).  SHARES threads share the pieces: one where many units keep
// the GPU busy (a piece or two each), eight where a few long sequences lie in up to
// a piece an SM.  Bound by the latency of its steps (descriptor, statistics and
// sums): rows one after the other in a CTA took 72 us for 8192 rows of two pieces.
constexpr int kLatentJoinThreads = 256;

template <int R, int N, typename T, int SHARES>
__global__ void __launch_bounds__(kLatentJoinThreads) join_latent_kernel(const LatentParams p, int groups) {
    constexpr int PER = kLatentJoinThreads / SHARES, AHEAD = 4;
    __shared__ float sums[SHARES > 1 ? SHARES : 1][10][PER];
    grid_dependency_wait();
    grid_launch_dependents();
    const PieceDesc d = p.part_desc[blockIdx.x];
    if (d.first_group == d.last_group) return;  // whole: written already
    const int b = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
    const int rows = p.q_len * p.num_heads;
    const int share = threadIdx.x / PER, at = blockIdx.y * PER + threadIdx.x % PER;
    const int c = at % N, e0 = at / N * 8;      // (R / 8 * N is a multiple of PER)
    const int pieces = d.last_group - d.first_group + 1;
    float M = -INFINITY, L = 0.f, a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
    for (int x0 = share; x0 < pieces; x0 += SHARES * AHEAD) {
        float2 ml[AHEAD];
        float y[AHEAD][8];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int x = x0 + k * SHARES;
            const long long g = d.first_group + x;
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[k][i] = 0.f;
            // (a group without tiles has no record)
            if (x < pieces && g * d.total / groups != (g + 1) * d.total / groups) {
                const long long rec = (g * p.group_size + d.member) * 2 + (x == 0 ? d.first_record : 0);
                ml[k] = *reinterpret_cast<const float2*>(p.part_ml + (rec * N + c) * 2);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[k][i] = p.part_acc[(rec * R + e0 + i) * N + c];
            }
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) m = fmaxf(m, ml[k].x);
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - m);
        M = m;
        L *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= f;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const float w = ml[k].x == -INFINITY ? 0.f : fast_exp2(ml[k].x - m);
            L = fmaf(w, ml[k].y, L);            // (0 * NaN: a row of NaN stays one)
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = fmaf(w, y[k][i], a[i]);
        }
    }
    if constexpr (SHARES > 1) {
        const int t = threadIdx.x % PER;
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[share][i][t] = a[i];
        sums[share][8][t] = M;
        sums[share][9][t] = L;
        __syncthreads();
        if (share != 0) return;
#pragma unroll
        for (int k = 1; k < SHARES; ++k) M = fmaxf(M, sums[k][8][t]);
        L = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = 0.f;
#pragma unroll
        for (int k = 0; k < SHARES; ++k) {
            const float m = sums[k][8][t], w = m == -INFINITY ? 0.f : fast_exp2(m - M);
            L = fmaf(w, sums[k][9][t], L);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = fmaf(w, sums[k][i][t], a[i]);
        }
    }
    if (rt * N + c >= rows) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + ((size_t)b * rows + rt * N + c) * R + e0) =
        make_uint4(Mma<T>::pack(a[0] * inv, a[1] * inv), Mma<T>::pack(a[2] * inv, a[3] * inv),
                   Mma<T>::pack(a[4] * inv, a[5] * inv), Mma<T>::pack(a[6] * inv, a[7] * inv));
}

template <int R, int N, typename T>
cudaError_t launch_latent_inst(const LatentLaunch& L, cudaStream_t stream) {
    static AttrFlags raised;
    auto kern = latent_kernel<R, N, T>;
    cudaError_t e = raise_smem_limit_once(kern, raised);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.ctas);
    cfg.blockDim = dim3(kLatentThreads);
    cfg.dynamicSmemBytes = LatentCfg<R, N, std::is_same<T, __nv_bfloat16>::value>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, L.tmap_c, L.tmap_q, L.p);
    if (e != cudaSuccess || !L.join) return e;
    const int units = L.p.batch * L.p.row_tiles, groups = L.ctas / L.p.group_size;
    const bool shared = (long long)units * 6 < L.ctas;  // seven pieces and more to a unit
    const int per = kLatentJoinThreads / (shared ? 8 : 1);
    cfg.gridDim = dim3((unsigned)units, (unsigned)((R / 8 * N + per - 1) / per));
    cfg.blockDim = dim3(kLatentJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return shared ? cudaLaunchKernelEx(&cfg, join_latent_kernel<R, N, T, 8>, L.p, groups)
                  : cudaLaunchKernelEx(&cfg, join_latent_kernel<R, N, T, 1>, L.p, groups);
}

template <int R>
cudaError_t launch_latent_for_r(const LatentLaunch& L, cudaStream_t stream) {
    switch (L.row_tile) {
        case 16:
            return L.bf16 ? launch_latent_inst<R, 16, __nv_bfloat16>(L, stream)
                          : launch_latent_inst<R, 16, __half>(L, stream);
        case 32:
            return L.bf16 ? launch_latent_inst<R, 32, __nv_bfloat16>(L, stream)
                          : launch_latent_inst<R, 32, __half>(L, stream);
        default:
            return L.bf16 ? launch_latent_inst<R, 64, __nv_bfloat16>(L, stream)
                          : launch_latent_inst<R, 64, __half>(L, stream);
    }
}

}  // namespace pa
