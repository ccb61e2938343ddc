// Accumulated attention weights for many query rows per kv head, on the
// Blackwell tensor cores (tcgen05).
//
// What it computes is weights[b, kvh, t] += sum_r 2^(s_rt - lse_r) (pa_weights.cu),
// for the rows of a several-token step: more than 16 per kv head.
//
// The scores are formed transposed, tokens in the 128 lanes of an MMA's
// result and query rows in its columns: a thread then owns a token, walks the
// columns with the rows' statistics broadcast from shared memory, and its sum
// never leaves a register.  A CTA keeps its tokens' keys in shared memory (256
// tokens; 128 at head_dim 256) and streams the query rows past them in chunks:
//   - warp 0 copies the keys (one lane per page, as the attention kernels do)
//     and each chunk of query rows (one box of 64 columns x the chunk's rows
//     per column block) by TMA;
//   - warp 1 (one lane) issues K Q^T, one MMA chain per 128 tokens and chunk;
//   - warp 3 fetches the chunk's statistics and causal limits;
//   - each further warpgroup reads one 128-token tile's scores from tensor
//     memory and sums the exponentials.
// Bound: the exponentials (16 a cycle and SM: a CTA's 256 x 128 scores take 2048
// cycles of the special-function units, its MMAs 1024), and the start of a CTA
// (2.5 us to its first scores), which is much for the 2 chunks that 256 rows are.
// Two CTAs share an SM, so that one's loads and waits hide behind the other's
// exponentials.  Two sequences of 8001 tokens, 8 kv heads of 128, 256 rows: 22 us
// cold (76 us for the same sums on warp-level MMAs with the query rows staged
// 64 at a time).  Every wait is bounded, as in the attention kernels.
#include <type_traits>

#include "pa_device.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

template <int D>
struct WTile {
    static constexpr int NT = D == 256 ? 1 : 2;      // 128-token tiles of a CTA
    static constexpr int NC = D == 256 ? 64 : 128;   // query rows of a chunk
    static constexpr int THREADS = 128 + 128 * NT;
    static constexpr uint32_t K_BYTES = 128u * D * 2u;  // one token tile
    static constexpr uint32_t Q_BYTES = NC * D * 2u;
    static constexpr uint32_t Q_OFF = NT * K_BYTES;
    static constexpr uint32_t LS_OFF = Q_OFF + Q_BYTES;     // [2][NC] -lse
    static constexpr uint32_t LIM_OFF = LS_OFF + 2 * NC * 4;  // [2][NC] attended tokens
    static constexpr uint32_t BAR_OFF = LIM_OFF + 2 * NC * 4;
    static constexpr uint32_t END = BAR_OFF + 16 * 8 + 16;
    // at least 100 KB, so that no more CTAs are resident than tensor memory holds
    static constexpr uint32_t SMEM = (END > 100u * 1024u ? END : 100u * 1024u) + kSmemAlignSlack;
    static constexpr uint32_t COLS = NT * NC;  // tensor-memory columns: 256, or 64
};

template <int D, int BS, typename KV>
__global__ void __launch_bounds__(WTile<D>::THREADS, 2)
    weights_tile_kernel(const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_q, const WeightParams p) {
    using W = WTile<D>;
    constexpr int NT = W::NT, NC = W::NC, DBLK = D / 64, KSTEPS = D / 16;
    constexpr int PAGES = NT * 128 / BS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlignSlack - 1)) &
        ~uintptr_t(kSmemAlignSlack - 1));
    float* ls = reinterpret_cast<float*>(smem + W::LS_OFF);
    int32_t* lim = reinterpret_cast<int32_t*>(smem + W::LIM_OFF);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + W::BAR_OFF);
    uint64_t* q_full = k_full + 1;
    uint64_t* q_empty = q_full + 1;
    uint64_t* st_full = q_empty + 1;   // [2] statistics buffer filled
    uint64_t* st_empty = st_full + 2;  // [2] and used
    uint64_t* s_full = st_empty + 2;   // [NT] scores of a tile in tensor memory
    uint64_t* s_empty = s_full + 2;    // [NT] and read
    uint64_t* final_bar = s_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + W::BAR_OFF + 16 * 8);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.group, gshift = __ffs(G) - 1, rows = p.q_len * G;
    grid_dependency_wait();
    grid_launch_dependents();
    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, BS);
    const int t0 = blockIdx.x * (NT * 128);
    if (t0 >= T) return;
    const int npages = (T + BS - 1) / BS;
    const int32_t* table_row = p.block_tables + (size_t)b * p.max_blocks;
    const int chunks = (rows + NC - 1) / NC;

    if (tid == 0) {
        mbar_init(smem_u32(k_full), 1);
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(st_full + i), 32);
            mbar_init(smem_u32(st_empty + i), 128 * NT);
            mbar_init(smem_u32(s_full + i), 1);
            mbar_init(smem_u32(s_empty + i), 128);
        }
        mbar_init(smem_u32(final_bar), 1);
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_q);
    }
    if (warp == 2) {
        tc::tmem_alloc(smem_u32(tmem_slot), W::COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
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

    if (warp == 0) {
        // ---- copies: the keys, then every chunk of query rows ----
        const int phys =
            lane < PAGES ? page_phys(table_row, t0 / BS + lane, npages, p.num_blocks) : -1;
        const unsigned live = __ballot_sync(kFullMask, phys >= 0);
        if (lane == 0) {
            if (live) mbar_arrive_expect_tx(smem_u32(k_full), (uint32_t)__popc(live) * 2u * BS * D);
            else mbar_arrive(smem_u32(k_full));
        }
        __syncwarp();
        if (phys >= 0) {
            const int row = lane * BS;
            const uint32_t dst = smem_u32(smem) + (row >> 7) * W::K_BYTES + (row & 127) * 128;
            const uint64_t policy = l2_policy_evict_first();
#pragma unroll
            for (int blk = 0; blk < DBLK; ++blk)
                tma_load_4d(dst + blk * 128 * 128, &tmap_k, blk * 64, kvh, 0, phys, smem_u32(k_full),
                            policy);
        }
        int issued = 0;
        if (lane == 0) {
            for (int c = 0; c < chunks && !*abort_flag; ++c) {
                if (c > 0 && !wait(q_empty, (c - 1) & 1)) break;
                mbar_arrive_expect_tx(smem_u32(q_full), W::Q_BYTES);
#pragma unroll
                for (int blk = 0; blk < DBLK; ++blk)
                    tma_load_3d(smem_u32(smem) + W::Q_OFF + blk * NC * 128, &tmap_q, blk * 64,
                                kvh * G, b * p.q_len + (c * NC >> gshift), smem_u32(q_full));
                issued = c + 1;
            }
            // no copy is in flight when the CTA ends
            (void)mbar_wait_bounded(smem_u32(k_full), 0, p.timeout_ns);
            if (issued > 0)
                (void)mbar_wait_bounded(smem_u32(q_full), (issued - 1) & 1, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMAs ----
        if (lane == 0) {
            constexpr int kType = std::is_same<KV, __nv_bfloat16>::value ? 1 : 0;
            constexpr uint32_t idesc = tc::idesc_f16(kType, false, 128, NC);
            bool ok = wait(k_full, 0);
            for (int c = 0; c < chunks && ok && !*abort_flag; ++c) {
                ok = wait(q_full, c & 1);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (c > 0 && !(ok = wait(s_empty + i, (c - 1) & 1))) break;
                    tc::fence_after_sync();
                    const uint32_t kb = smem_u32(smem) + i * W::K_BYTES;
                    const uint32_t qb = smem_u32(smem) + W::Q_OFF;
#pragma unroll
                    for (int ks = 0; ks < KSTEPS; ++ks)
                        tc::mma_ss(tmem + i * NC,
                                   tc::smem_desc(kb + (ks >> 2) * (128 * 128) + (ks & 3) * 32, 16, 1024,
                                                 tc::kSwizzle128B),
                                   tc::smem_desc(qb + (ks >> 2) * (NC * 128) + (ks & 3) * 32, 16, 1024,
                                                 tc::kSwizzle128B),
                                   idesc, ks > 0);
                    tc::commit(smem_u32(s_full + i));
                }
                if (ok) tc::commit(smem_u32(q_empty));
            }
            // every MMA issued has completed before tensor memory is released
            tc::commit(smem_u32(final_bar));
            (void)mbar_wait_bounded(smem_u32(final_bar), 0, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---- the rows' statistics ----
        const int ctx = max(__ldg(p.context_lens + b), 0);
        const int end = min(T, p.token_limit);
        for (int c = 0; c < chunks && !*abort_flag; ++c) {
            if (c >= 2 && !__all_sync(kFullMask, wait(st_empty + (c & 1), ((c - 2) >> 1) & 1))) break;
            for (int i = lane; i < NC; i += 32) {
                const int u = c * NC + i;
                // (rows past the last hold other queries or zeros: they see no token)
                ls[(c & 1) * NC + i] =
                    u < rows ? -p.lse[((size_t)b * p.q_len + (u >> gshift)) * p.num_heads + kvh * G +
                                      (u & (G - 1))]
                             : 0.f;
                lim[(c & 1) * NC + i] = u < rows ? min(end, ctx - p.q_len + (u >> gshift) + 1) : 0;
            }
            mbar_arrive(smem_u32(st_full + (c & 1)));
        }
    } else if (warp >= 4) {
        // ---- one token per thread ----
        const int tile = (warp - 4) >> 2, w4 = warp & 3;
        const int t = t0 + tile * 128 + w4 * 32 + lane;
        const uint32_t sb = tmem + ((uint32_t)(w4 * 32) << 16) + tile * NC;
        const float qscale = p.qscale;
        const int warp_end = t0 + tile * 128 + w4 * 32 + 32;  // past the warp's last token
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        int c = 0;
        for (; c < chunks && !*abort_flag; ++c) {
            const bool ok = wait(st_full + (c & 1), (c >> 1) & 1) && wait(s_full + tile, c & 1);
            if (!__all_sync(kFullMask, ok)) break;
            tc::fence_after_sync();
            const float* l = ls + (c & 1) * NC;
            const int32_t* e = lim + (c & 1) * NC;
            // limits rise with the row: the first row's holds for all of a full chunk
            const bool open = c * NC + NC <= rows && warp_end <= e[0];
#pragma unroll 1
            for (int c0 = 0; c0 < NC; c0 += 32) {
                uint32_t x[32];
                tc::ld_32x32b_x32(sb + c0, x);
                tc::wait_ld();
                if (open) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(l + c0 + i);
                        sum[0] += fast_exp2(fmaf(__uint_as_float(x[i]), qscale, m.x));
                        sum[1] += fast_exp2(fmaf(__uint_as_float(x[i + 1]), qscale, m.y));
                        sum[2] += fast_exp2(fmaf(__uint_as_float(x[i + 2]), qscale, m.z));
                        sum[3] += fast_exp2(fmaf(__uint_as_float(x[i + 3]), qscale, m.w));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float v = fast_exp2(fmaf(__uint_as_float(x[i]), qscale, l[c0 + i]));
                        sum[i & 3] += t < e[c0 + i] ? v : 0.f;
                    }
                }
            }
            tc::fence_before_sync();
            mbar_arrive(smem_u32(s_empty + tile));
            mbar_arrive(smem_u32(st_empty + (c & 1)));
        }
        if (c == chunks && t < T) {
            const bool held = page_phys(table_row, t / BS, npages, p.num_blocks) >= 0;
            const size_t at = ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * BS + t;
            p.weights_out[at] =
                p.weights_in[at] + (held ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f);
        }
    }

    if (blockIdx.x == gridDim.x - 1) {  // tokens past those attended to: nothing to add
        const size_t unit = ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * BS;
        for (int t = gridDim.x * (NT * 128) + tid; t < T; t += W::THREADS)
            p.weights_out[unit + t] = p.weights_in[unit + t];
    }

    // ---- release tensor memory once every role is done with it ----
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, W::COLS);
    }
}

template <int D, int BS, typename KV>
cudaError_t launch_inst(const WeightParams& p, const CUtensorMap& k, const CUtensorMap& q, bool pdl,
                        cudaStream_t stream) {
    using W = WTile<D>;
    auto kern = weights_tile_kernel<D, BS, KV>;
    static AttrFlags smem_limit;
    cudaError_t e = raise_smem_limit_once(kern, smem_limit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.token_limit + W::NT * 128 - 1) / (W::NT * 128)),
                       (unsigned)p.num_kv_heads, (unsigned)p.batch);
    cfg.blockDim = dim3(W::THREADS);
    cfg.dynamicSmemBytes = W::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, k, q, p);
}

template <int D>
cudaError_t launch_d(const WeightParams& p, int kv_dtype, const CUtensorMap& k, const CUtensorMap& q,
                     bool pdl, cudaStream_t stream) {
    const bool bf = kv_dtype == PA_BF16;
    if (p.block_size == 16)
        return bf ? launch_inst<D, 16, __nv_bfloat16>(p, k, q, pdl, stream)
                  : launch_inst<D, 16, __half>(p, k, q, pdl, stream);
    return bf ? launch_inst<D, 32, __nv_bfloat16>(p, k, q, pdl, stream)
              : launch_inst<D, 32, __half>(p, k, q, pdl, stream);
}

}  // namespace

int weights_tile_chunk(int head_dim) { return head_dim == 256 ? WTile<256>::NC : WTile<128>::NC; }

cudaError_t launch_weights_tile(const WeightParams& p, int head_dim, int kv_dtype,
                                const CUtensorMap& k, const CUtensorMap& q, bool pdl,
                                cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_d<64>(p, kv_dtype, k, q, pdl, stream);
        case 128: return launch_d<128>(p, kv_dtype, k, q, pdl, stream);
        default: return launch_d<256>(p, kv_dtype, k, q, pdl, stream);
    }
}

}  // namespace pa
