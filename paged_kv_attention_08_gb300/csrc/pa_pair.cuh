// Paged attention of two 128-row tiles side by side on the Blackwell tensor
// cores, for units of more than 128 query rows (query token x head of the
// group) at head_dim 64 and 128: the rows of sequences that share a prefix.
//
// The mathematics is that of the tile kernel (pa_tile.cuh): per row a running
// maximum m (base-2 units), normaliser l and O; S = Q K^T, P = 2^(S - m), O += P V.
// That kernel has one tile to a CTA and two S buffers, and its period is the
// chain of a block -- S, softmax, P V, the hand-offs between them.  Here a CTA has
// two tiles that share each K and V block, each with an O, an S buffer, a softmax
// warpgroup (a whole row to a thread: no exchange) and an MMA-issuing warp of its
// own.  While one tile is in its softmax the other's MMAs run, and a block is
// copied once for 256 rows.
//
// Warps: 0 copies K, and clears the V rows that P weights with 0; 1 and 2 issue
// the MMAs of tiles 0 and 1 (2 owns tensor memory); 3 copies Q and V; 4-7 and
// 8-11 are the tiles' softmax warpgroups.  P is handed over in pieces of 32
// tokens, so that P V runs beside the rest of the softmax; S of the next block
// follows once P V has read P, which lies over S.
//
// Bound: no one unit.  A block of two tiles takes 5300 cycles, of which the MMAs
// (bf16: 48 of 64 cycles) are 58 % and the exponentials (16 a cycle) 39 %; the
// rest is a tile's own chain.  512 rows of 8 kv heads of 128 on a prefix of 65,536
// (152 SMs, with the join): bf16 183 us, 752 TFLOP/s, fp16 146 us, 940 (a tile to a CTA:
// 197 and 154).  Also measured, bf16: P in two pieces 192; both tiles in step 186;
// each waiting for the other's first piece 240; one issuer for both, taking
// whichever is ready, 251; two threads to a row 190.
#pragma once

#include <type_traits>

#include "pa_device.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr float kPairRescaleSlack = 8.0f;  // log2 units: P may reach 2^8 before a rescale

// bf16's P goes in two parts of 8 bits each; fp16's in one, 2^kHalfLift higher
// (pa_internal.h), with the normaliser summed from the weights as rounded, so
// that the result is a mean of V's rows.
// Partials only: a prefix's and the sequences' own are joined by another launch.
template <int D, int BS, typename KV>
__global__ void __launch_bounds__(kTileThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ CUtensorMap tmap_q, const AttnParams p) {
    constexpr int BN = kPairBlock, BH = BN / 2;
    constexpr int BP = 32, NP = BN / BP;  // tokens of a piece of P, pieces of a block
    constexpr int NPB = BN / BS;  // pages of a block
    constexpr int DBLK = D / 64, KSTEPS = D / 16;
    constexpr int NK = pair_k_stages(D), NV = pair_v_stages(D);
    constexpr bool kSplitP = std::is_same<KV, __nv_bfloat16>::value;
    constexpr uint32_t TILE = 2u * BN * D, QTILE = 2u * kTileRows * D;  // bytes
    constexpr uint32_t O_COL = 0, S_COL = 2 * D;  // tensor memory: O of tile t at t D, S at S_COL + t BN
    static_assert(S_COL + 2 * BN <= 512, "tensor memory");
    constexpr float NEG_INF = -INFINITY;
    constexpr float kLift = kSplitP ? 0.f : kHalfLift;  // m: the row maximum less this

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlignSlack - 1)) &
        ~uintptr_t(kSmemAlignSlack - 1));
    uint8_t* const k_ring = smem + 2 * QTILE;
    uint8_t* const v_ring = k_ring + NK * TILE;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(v_ring + NV * TILE);
    uint64_t* k_empty = k_full + NK;
    uint64_t* v_full = k_empty + NK;
    uint64_t* v_clear = v_full + NV;  // the stage's rows of no weight hold zeros
    uint64_t* v_empty = v_clear + NV;
    uint64_t* s_full = v_empty + NV;  // [2] per tile
    uint64_t* p_full = s_full + 2;    // [2][NP] per tile and piece
    uint64_t* pv_done = p_full + 2 * NP;  // [2]
    uint64_t* q_full = pv_done + 2;
    uint64_t* turn = q_full + 1;      // tile 1's S has been issued
    uint64_t* final_bar = turn + 1;
    int32_t* k_live = reinterpret_cast<int32_t*>(final_bar + 1);  // [NK] the block holds a page
    int32_t* v_live = k_live + NK;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_live + NV);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group, gshift = __ffs(G) - 1, Q = p.q_len, Hkv = p.num_kv_heads, U = p.unit_rows;
    const int part = blockIdx.x, kvh = (int)blockIdx.y % Hkv, b = blockIdx.z;
    const int row0 = ((int)blockIdx.y / Hkv) * (2 * kTileRows);  // the CTA's first row of the unit
    const int ntile = U - row0 > kTileRows ? 2 : 1;
    grid_dependency_wait();
    grid_launch_dependents();

    const int reach = reachable_tokens(p.context_lens, b, p.max_blocks, BS);
    const int T = p.token_limit ? min(reach, p.token_limit) : reach;
    const int pb = part * p.part_pages, pe = min(pb + p.part_pages, (T + BS - 1) / BS);
    const int32_t* table_row = p.block_tables + (size_t)b * p.max_blocks;
    if (pe <= pb) return;  // no page of the sequence: the join reads nothing of such a partition
    const int nblk = (pe - pb + NPB - 1) / NPB;
    const int tend = min(T, pe * BS);  // the partition's tokens end here

    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_u32(k_full + i), 1);
            mbar_init(smem_u32(k_empty + i), ntile);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_u32(v_full + i), 1);
            mbar_init(smem_u32(v_clear + i), 1);
            mbar_init(smem_u32(v_empty + i), ntile);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(s_full + i), 1);
            for (int j = 0; j < NP; ++j) mbar_init(smem_u32(p_full + i * NP + j), 4);
            mbar_init(smem_u32(pv_done + i), 1);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(turn), 1);
        mbar_init(smem_u32(final_bar), ntile);
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        prefetch_tensormap(&tmap_q);
    }
    if (warp == 2) {
        tc::tmem_alloc(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();  // barriers initialised, tensor memory allocated
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = mbar_wait_bounded(smem_u32(bar), parity, p.timeout_ns);
        if (!ok) {
            record_error(p.err, PA_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        return ok;
    };
    // lane q < NPB: the block of page q of KV block k, or -1
    auto page_of = [&](int k) -> int {
        const int j = pb + k * NPB + lane;
        const int e = (lane < NPB && j < pe && k < nblk) ? __ldg(table_row + j) : -1;
        return e >= 0 && (int64_t)e < p.num_blocks ? e : -1;
    };

    if (warp == 0 || warp == 3) {
        // ---- copies: one lane per page of a block ----
        const bool is_k = warp == 0;
        const int NS = is_k ? NK : NV;
        uint64_t* full = is_k ? k_full : v_full;
        uint64_t* empty = is_k ? k_empty : v_empty;
        int32_t* live_of = is_k ? k_live : v_live;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        const uint32_t ring = smem_u32(is_k ? k_ring : v_ring);
        // (pages that other CTAs read too stay at the default priority)
        const uint64_t policy =
            U > 2 * kTileRows ? l2_policy_evict_normal() : l2_policy_evict_first();
        int issued = 0;
        bool q_issued = false;
        if (!is_k && lane == 0) {
            // the tiles' rows, G heads x 128 / G query tokens each; rows past the
            // unit's hold other queries or the fill value, and are masked
            mbar_arrive_expect_tx(smem_u32(q_full), (uint32_t)ntile * QTILE);
            for (int t = 0; t < ntile; ++t)
#pragma unroll
                for (int blk = 0; blk < DBLK; ++blk)
                    tma_load_3d(smem_u32(smem) + t * QTILE + blk * (kTileRows * 128), &tmap_q, blk * 64,
                                kvh * G, b * Q + ((row0 + t * kTileRows) >> gshift), smem_u32(q_full));
            q_issued = true;
        }
        // V rows that P weights with 0 (of pages that are not there, and past
        // the last token) are cleared once the stage's copies have landed: 0 x
        // NaN would reach O
        auto clear_v = [&](int k) -> bool {
            const int st = k % NV, phys = page_of(k);
            // (both issuers have seen the signal of the stage's last use)
            if (k >= NV && !__all_sync(kFullMask, wait(v_empty + st, (k / NV - 1) & 1))) return false;
            const unsigned live = __ballot_sync(kFullMask, phys >= 0);
            const int tb = (pb + k * NPB) * BS;
            if (live != (1u << NPB) - 1u || tb + BN > tend) {
                if (!__all_sync(kFullMask, wait(v_full + st, (k / NV) & 1))) return false;
                if (live) {  // (without a page there is no P V)
                    uint8_t* vt = v_ring + st * TILE;
                    for (int row = 0; row < BN; ++row) {
                        if (((live >> (row / BS)) & 1u) && tb + row < tend) continue;
                        if (lane < DBLK * 8)
                            *reinterpret_cast<uint4*>(vt + (lane >> 3) * (BN * 128) + row * 128 +
                                                      (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (lane == 0) mbar_arrive(smem_u32(v_clear + st));
            return true;
        };
        int phys = page_of(0);
        for (int k = 0; k < nblk && !*abort_flag; ++k) {
            const int st = k % NS, round = k / NS;
            const int next = page_of(k + 1);
            bool ok = true;
            if (round > 0) ok = __all_sync(kFullMask, wait(empty + st, (round - 1) & 1));
            if (!ok) break;
            const unsigned live = __ballot_sync(kFullMask, phys >= 0);
            const uint32_t bar = smem_u32(full + st);
            if (lane == 0) {
                live_of[st] = live != 0;
                if (live) mbar_arrive_expect_tx(bar, (uint32_t)__popc(live) * 2u * BS * D);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (phys >= 0) {
                const uint32_t dst = ring + (uint32_t)st * TILE + (uint32_t)lane * BS * 128;
#pragma unroll
                for (int blk = 0; blk < DBLK; ++blk)
                    tma_load_4d(dst + blk * BN * 128, map, blk * 64, kvh, 0, phys, bar, policy);
            }
            issued = k + 1;
            phys = next;
            if (is_k && k > 0 && !clear_v(k - 1)) break;
        }
        if (is_k && issued == nblk && !*abort_flag) (void)clear_v(nblk - 1);
        if (*abort_flag && lane == 0) {
            // copies still in flight land before the CTA may exit
            for (int k = issued > NS ? issued - NS : 0; k < issued; ++k)
                (void)mbar_wait_bounded(smem_u32(full + k % NS), (k / NS) & 1, p.timeout_ns);
            if (q_issued) (void)mbar_wait_bounded(smem_u32(q_full), 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp < 3) {
        // ---- MMAs of tile t (one lane) ----
        const int t = warp - 1;
        if (lane == 0 && t < ntile) {
            constexpr int kType = kSplitP ? 1 : 0;
            constexpr uint32_t id_s = tc::idesc_f16(kType, false, kTileRows, BN);
            constexpr uint32_t id_o = tc::idesc_f16(kType, true, kTileRows, D);
            const uint32_t s_col = tmem + S_COL + t * BN, o_col = tmem + O_COL + t * D;
            // (an address is below 2^18, so a descriptor of base + offset is the
            // base's plus offset >> 4)
            const uint64_t qd = tc::smem_desc(smem_u32(smem) + t * QTILE, 16, 1024, tc::kSwizzle128B);
            auto issue_s = [&](int k) -> bool {
                const int st = k % NK;
                if (!wait(k_full + st, (k / NK) & 1)) return false;
                // tile 1 starts a block once tile 0 has written a piece of its P: in step,
                // both would be in their softmax and then both at their MMAs
                if (ntile > 1) {
                    if (t == 1 ? !wait(p_full, k & 1) : (k > 0 && !wait(turn, (k - 1) & 1))) return false;
                }
                // S goes over the previous block's P
                if (k > 0 && !wait(pv_done + t, (k - 1) & 1)) return false;
                tc::fence_after_sync();
                if (k_live[st]) {
                    const uint64_t kd =
                        tc::smem_desc(smem_u32(k_ring) + st * TILE, 16, 1024, tc::kSwizzle128B);
#pragma unroll
                    for (int ks = 0; ks < KSTEPS; ++ks) {
                        const uint32_t off = (ks >> 2) * (BN * 128) + (ks & 3) * 32;
                        tc::mma_ss(s_col, qd + (off >> 4), kd + (off >> 4), id_s, ks > 0);
                    }
                }
                tc::commit(smem_u32(s_full + t));
                tc::commit(smem_u32(k_empty + st));
                if (t == 1) mbar_arrive(smem_u32(turn));
                return true;
            };
            bool started = false;  // O holds a sum
            bool ok = wait(q_full, 0) && issue_s(0);
            for (int k = 0; k < nblk && ok && !*abort_flag; ++k) {
                const int st = k % NV;
                ok = wait(v_full + st, (k / NV) & 1) && wait(v_clear + st, (k / NV) & 1);
                if (!ok) break;
                const bool live = v_live[st] != 0;
                // V: MN-major, 64-column blocks BN * 128 bytes apart, 8-row groups 1024
                const uint64_t vd0 =
                    tc::smem_desc(smem_u32(v_ring) + st * TILE, BN * 128, 1024, tc::kSwizzle128B);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    if (!(ok = wait(p_full + t * NP + i, k & 1))) break;
                    tc::fence_after_sync();
                    if (!live) continue;
                    const uint32_t ph = s_col + i * BP;  // hi; lo BP / 2 columns on
#pragma unroll
                    for (int kk = 0; kk < BP / 16; ++kk) {
                        const uint64_t vd = vd0 + (uint64_t)(((i * (BP / 16) + kk) * 16 * 128) >> 4);
                        tc::mma_ts(o_col, ph + kk * 8, vd, id_o, (started || i + kk > 0) ? 1u : 0u);
                        if (kSplitP) tc::mma_ts(o_col, ph + BP / 2 + kk * 8, vd, id_o, 1u);
                    }
                }
                if (!ok) break;
                started = started || live;
                tc::commit(smem_u32(pv_done + t));
                tc::commit(smem_u32(v_empty + st));
                if (k + 1 < nblk) ok = issue_s(k + 1);
            }
            // every MMA issued has completed before tensor memory is released
            tc::commit(smem_u32(final_bar));
            (void)mbar_wait_bounded(smem_u32(final_bar), 0, p.timeout_ns);
        }
        __syncwarp();
    } else if ((warp - 4) >> 2 < ntile) {
        // ---- softmax: a row to a thread ----
        const int t = (warp - 4) >> 2, w4 = warp & 3;
        const int u = row0 + t * kTileRows + w4 * 32 + lane;
        const bool dead = u - lane >= U;  // all of the warp's rows lie past the unit's
        const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
        const uint32_t sb = lane_base + S_COL + t * BN, ob = lane_base + O_COL + t * D;
        const float qscale = p.qscale;
        const int ctx = max(__ldg(p.context_lens + b), 0);
        // tokens below lim: the row's causal limit, the table's reach, the partition's end
        const int lim =
            u >= U ? 0
                   : min(tend, p.own_lens ? prefix_limit(reach, b, u >> gshift, Q, p.own_q, p.own_lens)
                                          : ctx - Q + (u >> gshift) + 1);
        float m = NEG_INF, l = 0.f;
        unsigned bits_next = __ballot_sync(kFullMask, page_of(0) >= 0);
        int k = 0;
        for (; k < nblk && !*abort_flag; ++k) {
            const unsigned bits = bits_next;
            bits_next = __ballot_sync(kFullMask, page_of(k + 1) >= 0);
            if (!__all_sync(kFullMask, wait(s_full + t, k & 1))) break;
            tc::fence_after_sync();
            const bool work = bits != 0 && !dead;  // (the same in the whole warp)
            const int t0 = (pb + k * NPB) * BS;
            const bool open = __all_sync(kFullMask, bits == (1u << NPB) - 1u && t0 + BN <= lim);
            float sc[BH];
            // scores of half h, masked
            auto load = [&](int h) {
                uint32_t x[BH / 32][32];
#pragma unroll
                for (int i = 0; i < BH / 32; ++i) tc::ld_32x32b_x32(sb + h * BH + i * 32, x[i]);
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < BH; ++c) sc[c] = __uint_as_float(x[c / 32][c % 32]);
                if (!open) {
#pragma unroll
                    for (int c = 0; c < BH; ++c) {
                        const bool pl = (bits >> ((h * BH + c) / BS)) & 1u;
                        sc[c] = (pl && t0 + h * BH + c < lim) ? sc[c] : NEG_INF;
                    }
                }
            };
            float me = 0.f;
            if (work) {
                float mx = NEG_INF;
                load(1);
#pragma unroll
                for (int c = 0; c < BH; c += 2) mx = fmax3(mx, sc[c], sc[c + 1]);
                load(0);
#pragma unroll
                for (int c = 0; c < BH; c += 2) mx = fmax3(mx, sc[c], sc[c + 1]);
                const float ms = mx * qscale;
                const bool need = ms > m + (kPairRescaleSlack + kLift);
                float alpha = 1.f;
                if (need) {
                    const float base = ms - kLift;
                    alpha = m == NEG_INF ? 1.f : fast_exp2(m - base);
                    l *= alpha;
                    m = base;
                }
                // (S is issued after the previous block's P V has completed: O is at rest)
                if (__any_sync(kFullMask, need && alpha != 1.f)) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t x[16];
                        tc::ld_32x32b_x16(ob + c0, x);
                        tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            x[c] = __float_as_uint(__uint_as_float(x[c]) * alpha);
                        tc::st_32x32b_x16(ob + c0, x);
                    }
                }
                me = m == NEG_INF ? 0.f : m;
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (work) {
                    if (i == NP / 2) load(1);
                    // P = 2^(s scale log2 e - m) over the piece's S: hi, then lo
#pragma unroll
                    for (int c0 = 0; c0 < BP; c0 += 16) {
                        const int at = (i * BP + c0) % BH;
                        uint32_t ph[8], pl[8];
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float x0 = fast_exp2(fmaf(sc[at + c], qscale, -me));
                            const float x1 = fast_exp2(fmaf(sc[at + c + 1], qscale, -me));
                            const uint32_t hi = Mma<KV>::pack(x0, x1);
                            ph[c / 2] = hi;
                            if constexpr (kSplitP) {
                                float h0, h1;
                                Mma<KV>::unpack(hi, h0, h1);
                                l += x0 + x1;
                                pl[c / 2] = Mma<KV>::pack(x0 - h0, x1 - h1);
                            } else {
                                l = Mma<KV>::add2(hi, l);  // the weights that the MMA uses
                            }
                        }
                        tc::st_32x32b_x8(sb + i * BP + c0 / 2, ph);
                        if (kSplitP) tc::st_32x32b_x8(sb + i * BP + BP / 2 + c0 / 2, pl);
                    }
                    tc::wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + t * NP + i));
            }
        }
        // ---- the partial (m, l, O) ----
        bool have = __all_sync(kFullMask, k == nblk && !*abort_flag);
        if (have) have = __all_sync(kFullMask, wait(pv_done + t, (nblk - 1) & 1));
        tc::fence_after_sync();
        if (have && !dead) {
            const bool live = u < U;
            const size_t row = (((size_t)b * Hkv + kvh) * p.num_parts + part) * U + u;
            if (live) {
                p.part_ml[row * 2] = l > 0.f ? m : NEG_INF;
                p.part_ml[row * 2 + 1] = l;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t x[16];
                float v[16];
                tc::ld_32x32b_x16(ob + c0, x);
                tc::wait_ld();
                if (!live) continue;
                // (an O that no P V wrote holds garbage)
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = l > 0.f ? __uint_as_float(x[c]) : 0.f;
                float* dst = p.part_acc + row * D + c0;
                if ((reinterpret_cast<uintptr_t>(p.part_acc) & 31) == 0) {  // whole sectors
                    st_global_v8(dst, v);
                    st_global_v8(dst + 8, v + 8);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; c += 4)
                        *reinterpret_cast<float4*>(dst + c) =
                            make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                }
            }
        }
    }

    // ---- release tensor memory once every role is done with it ----
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, int BS, typename KV>
cudaError_t launch_pair_inst(const AttnLaunch& L, cudaStream_t stream) {
    auto kern = pair_kernel<D, BS, KV>;
    static AttrFlags smem_limit;
    cudaError_t e = raise_smem_limit_once(kern, smem_limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = L.grid;
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = L.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, L.tmap_k, L.tmap_v, L.tmap_q, L.p);
}

template <int D>
cudaError_t launch_pair_for_d(const AttnLaunch& L, cudaStream_t stream) {
    const bool bs16 = L.block_size == 16;
    if (L.kv_dtype == PA_BF16)
        return bs16 ? launch_pair_inst<D, 16, __nv_bfloat16>(L, stream)
                    : launch_pair_inst<D, 32, __nv_bfloat16>(L, stream);
    return bs16 ? launch_pair_inst<D, 16, __half>(L, stream) : launch_pair_inst<D, 32, __half>(L, stream);
}

}  // namespace pa
