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
// Four sequences of 65,000 to 131,072 tokens, 8 kv heads of 128, cut to 8192 each:
// 81 us to other pages (selection 27, copy 48 at 5.6 TB/s), 144 us in place, 0.6 ms
// with a copy of the table.
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kSelThreads = 512;
constexpr int kMaxSelCluster = 8;
constexpr int kBins = 2048;           // digits of 11, 11 and 10 bits; four per thread
constexpr int kSelShare = 4096;       // tokens a CTA takes before a row gets a larger cluster
constexpr int kMaxCached = 38 * 1024; // tokens whose keys fit in a CTA's shared memory

// Keys of tokens that the selection does not weigh.
constexpr uint32_t kKeyAlways = 0xffffffffu;  // kept whatever the weight
constexpr uint32_t kKeyAbsent = 0u;           // of a masked page: never kept
// In a kept token's position, between the selection and the copy: the new table
// names a page of the old one at its own place.
constexpr int32_t kMarked = INT32_MIN;

// Integers that order as the weights do: NaN below every number, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 1u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Exclusive sum over the CTA of one number per thread; *total gets the sum.
// One barrier: `scratch` holds a number per warp and is not used again.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* scratch, uint32_t* total) {
    constexpr int W = kSelThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t y = __shfl_up_sync(kFullMask, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    uint32_t s = lane < W ? scratch[lane] : 0;
    const uint32_t own = s;
#pragma unroll
    for (int m = 1; m < W; m <<= 1) {
        const uint32_t y = __shfl_up_sync(kFullMask, s, m);
        if (lane >= m) s += y;
    }
    *total = __shfl_sync(kFullMask, s, W - 1);
    return x - v + __shfl_sync(kFullMask, s - own, warp);
}

// Stores and adds to the same place in another CTA's shared memory.
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_add(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Word of cached quad q: four words in 36 are skipped, so that threads that
// each walk a run of eight quads meet in no bank.
__device__ __forceinline__ int quad_word(int q) { return q * 4 + (q >> 3) * 4; }

// One cluster of up to 8 CTAs per (kv head, sequence), each with a run of the
// row's tokens, handled in quads (which lie in one page).  A CTA turns its
// weights into keys once and keeps them in shared memory (CACHED; a row too
// long for that is read again where its keys are needed).  The threshold, the
// want-th largest key among the tokens that are not kept anyway, is found by
// digits of 11, 11 and 10 bits:
//   - each CTA counts its keys' first digits (four copies of the bins, a lane
//     takes copy lane % 4: weights meet in few bins) and adds its non-empty
//     bins to those of every CTA of the cluster through distributed shared
//     memory; all of them then know the threshold's first digit;
//   - the keys with that digit, a few in a hundred as a rule, are sent to
//     every CTA, each of which finds the other two digits by itself;
//   - where they are too many for that (ties), the CTAs count and add up the
//     other digits as they did the first.
// Then each thread marks what it keeps of its own run of quads in a bit mask;
// one scan over the CTA, and the counts of the CTAs before it, tell it where
// to write them.
//
// What bounds it: the latency of its steps (a cluster barrier 1 to 2 us with
// the skew of its CTAs), not the 17 MB that 32 rows of 128K weights are.  The
// 32 rows of up to 131,072 tokens take 27 us; one CTA to a row, reading the row
// from global memory in four passes of 8 bits, took 460 us, and a cluster
// whose CTAs read each other's whole bins 37 us.
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) uint32_t hist[kBins * 4];  // this CTA's counts; later the candidates' keys
    __shared__ __align__(16) uint32_t sums[kBins];      // the cluster's counts
    __shared__ uint32_t scratch[6][kSelThreads / 32];
    __shared__ uint32_t chosen[3][2];  // of each pass: the threshold's digit, tokens still wanted of it
    // every CTA's tokens held, and of them those kept whatever their weight;
    // those above the threshold (the latter included), and those equal to it;
    // those that share the threshold's first digit
    __shared__ uint32_t shares[kMaxSelCluster][5];
    __shared__ uint32_t counted[2];
    __shared__ int32_t mark;  // kMarked or 0
    const int tid = threadIdx.x, lane = tid & 31;
    const int C = (int)p.cluster, rank = (int)blockIdx.x % C;
    const int kvh = (int)blockIdx.x / C, b = blockIdx.y;
    const uint4 zeros = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kBins; i += kSelThreads) reinterpret_cast<uint4*>(hist)[i] = zeros;
    reinterpret_cast<uint4*>(sums)[tid] = zeros;
    if (tid < 2) counted[tid] = 0;
    if (tid == 0) mark = 0;
    // (the others' adds may come from here on: every CTA waits for this before its first)
    if (C > 1) cluster_arrive_release();
    else __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    const int T = reachable_tokens(p.context_lens, b, p.max_blocks, p.block_size);
    const float* w = p.weights + ((size_t)b * p.num_kv_heads + kvh) * p.max_blocks * p.block_size;
    int32_t* kept = p.kept + ((size_t)b * p.num_kv_heads + kvh) * p.budget;
    const int32_t* row = p.block_tables + (size_t)b * p.max_blocks;
    // does the new table name a page of the old one at its own place (a copy of it)?
    bool same = false;
    if (!p.in_place) {
        const int32_t* new_row = p.new_block_tables + (size_t)b * p.new_max_blocks;
        const int pages = min((p.budget + p.block_size - 1) / p.block_size, p.max_blocks);
        for (int i = tid; i < pages; i += kSelThreads) {
            const int e = __ldg(new_row + i);
            same |= e >= 0 && e == __ldg(row + i);
        }
    }
    const int npages = (T + p.block_size - 1) / p.block_size;
    const int bshift = __ffs(p.block_size) - 1;
    const int recent = T - p.recent;
    const bool wide = (reinterpret_cast<uintptr_t>(p.weights) & 15) == 0;
    // quads [q0, q0 + nq) of the row
    const int quads = (T + 3) / 4, per = (quads + C - 1) / C;
    const int q0 = min(rank * per, quads), nq = min(per, quads - q0);

    // a quad's page, and its weights (inside the row: its width is a multiple of 16)
    auto quad_held = [&](int q) { return page_phys(row, (q * 4) >> bshift, npages, p.num_blocks) >= 0; };
    auto quad_load = [&](int q) {
        const float* v = w + (size_t)q * 4;
        return wide ? *reinterpret_cast<const float4*>(v) : make_float4(v[0], v[1], v[2], v[3]);
    };
    auto quad_keys = [&](int q, bool held, const float4& x) {
        if (!held) return make_uint4(0, 0, 0, 0);
        uint4 k = make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
        const int t = q * 4;
        if (t < p.sink || t + 3 >= recent) {  // at the row's ends: token by token
            auto end = [&](int u, uint32_t v) {
                return u >= T ? kKeyAbsent : (u < p.sink || u >= recent ? kKeyAlways : v);
            };
            k = make_uint4(end(t, k.x), end(t + 1, k.y), end(t + 2, k.z), end(t + 3, k.w));
        }
        return k;
    };
    // keys of the CTA's quad i
    auto keys_at = [&](int i) {
        if constexpr (CACHED) return *reinterpret_cast<const uint4*>(keys + quad_word(i));
        const bool held = quad_held(q0 + i);
        return quad_keys(q0 + i, held, held ? quad_load(q0 + i) : make_float4(0.f, 0.f, 0.f, 0.f));
    };
    auto cluster_barrier = [&]() {
        if (C > 1) cluster_sync_release_acquire();
        else __syncthreads();
    };
    // the same number to every CTA of the cluster, before a cluster barrier
    auto tell = [&](int which, uint32_t v) {
        for (int r = 0; r < C; ++r)
            st_cluster_u32(map_cluster_rank(smem_u32(&shares[rank][which]), r), v);
    };

    // the keys, and the first pass's counts: eight quads in flight (the
    // weights of a masked page are loaded like the others, and not used)
    uint32_t held = 0, must = 0;
    uint32_t* const copy = hist + (lane & 3);
    auto count_first = [&](uint32_t k) {
        if (k == kKeyAlways) ++must;
        else if (k != kKeyAbsent) {
            ++held;
            atomicAdd(&copy[(k >> 21) * 4], 1u);
        }
    };
    if (C > 1) cluster_wait_acquire();  // (also a barrier of the CTA: hist is zero)
    if (same) mark = kMarked;
    for (int base = tid; base < nq; base += kSelThreads * 8) {
        float4 x[8];
        bool ok[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int q = base + u * kSelThreads;
            x[u] = q < nq ? quad_load(q0 + q) : make_float4(0.f, 0.f, 0.f, 0.f);
            ok[u] = q < nq && quad_held(q0 + q);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int q = base + u * kSelThreads;
            if (q >= nq) continue;
            const uint4 k = quad_keys(q0 + q, ok[u], x[u]);
            if constexpr (CACHED) *reinterpret_cast<uint4*>(keys + quad_word(q)) = k;
            const int t = (q0 + q) * 4;
            if (ok[u] && t >= p.sink && t + 3 < recent) {  // four tokens to weigh
                held += 4;
                atomicAdd(&copy[(k.x >> 21) * 4], 1u);
                atomicAdd(&copy[(k.y >> 21) * 4], 1u);
                atomicAdd(&copy[(k.z >> 21) * 4], 1u);
                atomicAdd(&copy[(k.w >> 21) * 4], 1u);
            } else {
                count_first(k.x);
                count_first(k.y);
                count_first(k.z);
                count_first(k.w);
            }
        }
    }
    held = __reduce_add_sync(kFullMask, held);
    must = __reduce_add_sync(kFullMask, must);
    if (lane == 0) {
        atomicAdd(&counted[0], held + must);
        atomicAdd(&counted[1], must);
    }

    // a thread's run of quads: a power of two up to eight, then whole eights
    int run = 1;
    while (run < 8 && run * kSelThreads < nq) run *= 2;
    if (run == 8) run = ((nq + kSelThreads - 1) / kSelThreads + 7) / 8 * 8;
    const int i0 = min(tid * run, nq), i1 = min(i0 + run, nq);

    uint32_t prefix = 0, mask = 0, want = 0, n = 0;
    int steps = 0;
    // the digit of the want-th largest key among those counted: thread tid has
    // the counts of bins 4 tid .. 4 tid + 3
    auto find_digit = [&](const uint4& c, int shift, uint32_t digit) {
        uint32_t total;
        const uint32_t before = block_exclusive(c.x + c.y + c.z + c.w, scratch[steps], &total);
        if (tid == 0 && want == 0) {  // nothing is wanted: above every key
            chosen[steps][0] = digit;
            chosen[steps][1] = 0;
        }
        const uint32_t below = total - want;  // candidates left out
        if (want > 0 && below >= before && below < before + c.x + c.y + c.z + c.w) {
            const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
            uint32_t s = before;
            int d = 0;
            while (d < 3 && below >= s + cs[d]) s += cs[d++];
            chosen[steps][0] = (uint32_t)(4 * tid + d);
            chosen[steps][1] = s + cs[d] - below;
        }
        __syncthreads();
        prefix |= chosen[steps][0] << shift;
        mask |= digit << shift;
        want = chosen[steps][1];
        ++steps;
    };
    // this CTA's counts of this thread's bins, the non-empty ones to every CTA
    auto send_counts = [&](const uint4& c) {
        if ((c.x | c.y | c.z | c.w) == 0) return;
        for (int r = 0; r < C; ++r) {
            const uint32_t at = map_cluster_rank(smem_u32(&sums[4 * tid]), r);
            if (c.x) red_cluster_add(at, c.x);
            if (c.y) red_cluster_add(at + 4, c.y);
            if (c.z) red_cluster_add(at + 8, c.z);
            if (c.w) red_cluster_add(at + 12, c.w);
        }
    };
    uint4* const my_sums = reinterpret_cast<uint4*>(sums) + tid;

    __syncthreads();  // this CTA's counts are complete
    uint4 c;
    {
        const uint4* h = reinterpret_cast<const uint4*>(hist) + 4 * tid;
        const uint4 h0 = h[0], h1 = h[1], h2 = h[2], h3 = h[3];
        c = make_uint4(h0.x + h0.y + h0.z + h0.w, h1.x + h1.y + h1.z + h1.w,
                       h2.x + h2.y + h2.z + h2.w, h3.x + h3.y + h3.z + h3.w);
    }
    if (C > 1) send_counts(c);
    if (tid < 2) tell(tid, counted[tid]);
    cluster_barrier();
    if (C > 1) c = *my_sums;
    uint32_t valid = 0, fixed = 0;
    for (int r = 0; r < C; ++r) {
        valid += shares[r][0];
        fixed += shares[r][1];
    }
    n = min(valid, (uint32_t)p.budget);
    want = n - fixed;
    const bool all = valid <= (uint32_t)p.budget;  // (the same in every CTA of the cluster)
    if (!all) {
        find_digit(c, 21, 2047u);
        *my_sums = zeros;
        auto each_key = [&](auto&& fn) {  // of this thread's run
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const uint4 k = keys_at(i);
                fn(k.x);
                fn(k.y);
                fn(k.z);
                fn(k.w);
            }
        };
        auto candidate = [&](uint32_t k) {
            return (k & mask) == prefix && k != kKeyAbsent && k != kKeyAlways;
        };
        // the keys with the threshold's first digit, into this CTA's part of the list
        // (a row of one CTA counts its keys again instead)
        const uint32_t room = kBins * 4 / C;
        bool fits = C > 1;
        if (C > 1) {
            uint32_t* const mine = hist + rank * room;
            uint32_t count = 0;
            each_key([&](uint32_t k) { count += candidate(k); });
            uint32_t sent;
            uint32_t at = block_exclusive(count, scratch[4], &sent);
            if (count > 0 && sent <= room)
                each_key([&](uint32_t k) {
                    if (candidate(k)) mine[at++] = k;
                });
            if (tid == 0) tell(4, sent);
            __syncthreads();
            if (sent <= room)
                for (int r = 0; r < C; ++r) {
                    if (r == rank) continue;
                    const uint32_t to = map_cluster_rank(smem_u32(mine), r);
                    for (uint32_t i = tid; i < sent; i += kSelThreads) st_cluster_u32(to + 4u * i, mine[i]);
                }
            cluster_barrier();
            for (int r = 0; r < C; ++r) fits = fits && shares[r][4] <= room;
        }
        for (int step = 0; step < 2; ++step) {
            const int shift = step == 0 ? 10 : 0;
            const uint32_t digit = step == 0 ? 2047u : 1023u;
            if (fits) {
                // (an equal share of the threads to each CTA's part)
                const int r = tid / (kSelThreads / C);
                const uint32_t len = shares[r][4];
                for (uint32_t i = tid % (kSelThreads / C); i < len; i += kSelThreads / C) {
                    const uint32_t k = hist[r * room + i];
                    if (candidate(k)) atomicAdd(&sums[(k >> shift) & digit], 1u);
                }
                __syncthreads();
                c = *my_sums;
                *my_sums = zeros;
                find_digit(c, shift, digit);  // (its barriers order the zeros before the next counts)
            } else {
                // (the list is not used: its first words hold this CTA's counts)
                reinterpret_cast<uint4*>(hist)[tid] = zeros;
                __syncthreads();
                each_key([&](uint32_t k) {
                    if (candidate(k)) atomicAdd(&hist[(k >> shift) & digit], 1u);
                });
                __syncthreads();
                c = reinterpret_cast<const uint4*>(hist)[tid];
                if (C > 1) {
                    send_counts(c);
                    cluster_barrier();
                    c = *my_sums;
                    *my_sums = zeros;
                    cluster_barrier();  // zero before the next step's counts arrive
                }
                find_digit(c, shift, digit);
            }
        }
    }

    // what this thread surely keeps of its run, and what equals the threshold,
    // of which the row keeps its lowest `want`: a bit for each token of eight quads
    // (with `all` the prefix is 0 = absent: every other key is above it)
    auto masks = [&](int i, uint32_t& s, uint32_t& e) {
        s = e = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint4 k = i + u < i1 ? keys_at(i + u) : make_uint4(0, 0, 0, 0);
            s |= ((uint32_t)(k.x > prefix) | (uint32_t)(k.y > prefix) << 1 |
                  (uint32_t)(k.z > prefix) << 2 | (uint32_t)(k.w > prefix) << 3) << (4 * u);
            e |= ((uint32_t)(k.x == prefix) | (uint32_t)(k.y == prefix) << 1 |
                  (uint32_t)(k.z == prefix) << 2 | (uint32_t)(k.w == prefix) << 3) << (4 * u);
        }
        // (with nothing wanted the threshold is the key of the tokens always kept)
        if (prefix == kKeyAlways) s = e;
        if (prefix == kKeyAbsent || prefix == kKeyAlways) e = 0;
    };
    uint32_t sure = 0, equal = 0, s0 = 0, e0 = 0;
    for (int i = i0; i < i1; i += 8) {
        uint32_t s, e;
        masks(i, s, e);
        if (i == i0) {
            s0 = s;
            e0 = e;
        }
        sure += __popc(s);
        equal += __popc(e);
    }
    uint32_t sures, equals;
    if constexpr (CACHED) {  // both below 2^16: one scan
        static_assert(kMaxCached < 65536, "packed counts");
        const uint32_t at = block_exclusive(sure | equal << 16, scratch[3], &sures);
        sure = at & 0xffffu;
        equal = at >> 16;
        equals = sures >> 16;
        sures &= 0xffffu;
    } else {
        sure = block_exclusive(sure, scratch[3], &sures);
        equal = block_exclusive(equal, scratch[5], &equals);
    }
    if (tid < 2) tell(2 + tid, tid == 0 ? sures : equals);
    cluster_barrier();  // (the last access to another CTA's memory is before it)
    uint32_t begin = 0, left = want;  // where this CTA's list begins; equal tokens still wanted
    for (int r = 0; r < rank; ++r) {
        const uint32_t eq = min(left, shares[r][3]);
        begin += shares[r][2] + eq;
        left -= eq;
    }
    uint32_t j = begin + sure;  // plus the kept ones of the equal tokens before
    const int32_t marks = mark;
    for (int i = i0; i < i1; i += 8) {
        uint32_t s = s0, e = e0;
        if (i > i0) masks(i, s, e);
        const int t = (q0 + i) * 4;
        for (uint32_t any = s | e; any; any &= any - 1) {
            const int u = __ffs(any) - 1;
            if ((s >> u) & 1u) {
                kept[j + min(equal, left)] = (t + u) | marks;
                ++j;
            } else {
                if (equal < left) kept[j + equal] = (t + u) | marks;
                ++equal;
            }
        }
    }
    if (rank == 0) {
        for (int i = (int)n + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
        if (kvh == 0 && tid == 0) p.new_lens[b] = (int32_t)n;
    }
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

// One CTA per (64 tokens of the new row, kv head, sequence): 32 KB of keys and
// values, eight 16-byte vectors of a thread on their way at a time.
//
// Where the selection found an entry that stands at the same place in both
// tables (kept tokens carry kMarked), row j may be written over old token j,
// which another CTA may have to read.  Then the first CTA moves all of the kv
// head's rows in order: they come from old tokens kept[j] >= j, so that no row
// comes from where an earlier one went.  The others only take the marks off.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p) {
    __shared__ long long src[kCopyRows], dst[kCopyRows];
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int j0 = blockIdx.x * kCopyRows;
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t unit = (size_t)b * p.num_kv_heads + kvh;
    const int vecs = p.head_dim / 8;
    const int32_t* old_row = p.block_tables + (size_t)b * p.max_blocks;
    const int32_t* new_row = p.new_block_tables + (size_t)b * p.new_max_blocks;
    // (volatile: a CTA that moves all rows reads entries while theirs take the marks off)
    volatile int32_t* kept = p.kept + unit * p.budget;
    // the old token that row j is, and where both of them lie (-1: nowhere)
    auto place = [&](int j, bool& marked) {
        int t = j < p.budget ? kept[j] : -1;
        marked = t < -1;
        if (marked) t &= ~kMarked;
        long long s = -1, d = -1;
        if (t >= 0) {
            s = slot_of(old_row, t, p.block_size, p.max_blocks, p.num_blocks);
            d = slot_of(new_row, j, p.block_size, p.new_max_blocks, p.num_blocks);
        }
        src[tid] = s;
        dst[tid] = d;
        return t;
    };
    bool marked = false;
    if (tid < kCopyRows) {
        const int j = j0 + tid, t = place(j, marked);
        if (marked) kept[j] = t;
        const size_t width = (size_t)p.max_blocks * p.block_size;
        const size_t new_width = (size_t)p.new_max_blocks * p.block_size;
        if ((size_t)j < new_width)
            p.new_weights[unit * new_width + j] = t >= 0 ? p.weights[unit * width + t] : 0.f;
    }
    const bool in_order = __syncthreads_or(marked);
    if (in_order && blockIdx.x > 0) return;
    const long long row = (long long)p.num_kv_heads * vecs;
    // eight vectors of a thread in flight at a time
    const int vshift = __ffs(vecs) - 1;  // (8, 16 or 32 vectors a head)
    for (int next = kCopyRows;; next += kCopyRows) {
        for (int i0 = tid; i0 < kCopyRows * 2 * vecs; i0 += kCopyThreads * 8) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kCopyThreads, r = i >> (vshift + 1), c = i & (2 * vecs - 1);
                if (r >= kCopyRows || src[r] < 0 || dst[r] < 0) continue;
                const uint4* cache = static_cast<const uint4*>(c < vecs ? p.k_cache : p.v_cache);
                v[k] = cache[src[r] * row + kvh * vecs + (c & (vecs - 1))];
            }
            if (in_order) __syncthreads();  // (as many turns in every thread)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kCopyThreads, r = i >> (vshift + 1), c = i & (2 * vecs - 1);
                if (r >= kCopyRows || src[r] < 0 || dst[r] < 0) continue;
                uint4* cache = static_cast<uint4*>(c < vecs ? p.k_cache : p.v_cache);
                cache[dst[r] * row + kvh * vecs + (c & (vecs - 1))] = v[k];
            }
        }
        if (!in_order || next >= p.budget) return;
        __syncthreads();  // these rows' places have been used
        if (tid < kCopyRows) (void)place(next + tid, marked);  // (its own CTA takes a mark off)
        __syncthreads();
    }
}

constexpr int kPackThreads = 512;
constexpr int kPackRows = kPackThreads / 8;          // rows of 64 columns moved by one step
constexpr int kPackSteps = 8;
constexpr int kPackChunk = kPackRows * kPackSteps;   // rows that are read before the first is written
constexpr int kPackSegment = 8192;                   // rows whose places are in shared memory at a time
constexpr uint32_t kPackSmem = kPackSegment * 8 + kPackSegment / 16 * 4;

// In place: token j of the new row comes from slot kept[j] >= j of the same
// row, so a chunk of rows may be written once all of it has been read, and
// no later chunk reads what it writes.  One CTA per (64 columns of the keys
// or of the values, kv head, sequence) takes the chunks in order, the next
// chunk's rows on their way while it writes this one's; columns do not meet,
// so the CTAs need no order among them.  One more CTA packs the weights.
//
// Bound: the latency of a chunk (64 KB a CTA in flight), with few CTAs: 4
// sequences, 8 kv heads and head_dim 128 are 128 of them.  The rows' places
// are found for a segment at once: looked up chunk by chunk, 256 rows at a
// time and none ahead, four sequences of 65,000 to 131,072 tokens cut to 8192
// took 412 us.
__global__ void __launch_bounds__(kPackThreads, 1) evict_pack_kernel(const EvictParams p) {
    extern __shared__ long long src[];  // [segment] slot that a row comes from, -1: it stays
    int32_t* page = reinterpret_cast<int32_t*>(src + kPackSegment);  // block of each new page, or -1
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int slices = p.head_dim / 64;
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t unit = (size_t)b * p.num_kv_heads + kvh;
    const int32_t* kept = p.kept + unit * p.budget;
    const int n = p.new_lens[b];
    if ((int)blockIdx.x == 2 * slices) {
        // the weights, and zeros behind them
        const float* w = p.weights + unit * p.max_blocks * p.block_size;
        const int new_width = p.new_max_blocks * p.block_size;
        float* nw = p.new_weights + unit * new_width;
        for (int j0 = 0; j0 < n; j0 += kPackThreads * kPackSteps) {
            float x[kPackSteps];
#pragma unroll
            for (int k = 0; k < kPackSteps; ++k) {
                const int j = j0 + k * kPackThreads + tid;
                if (j < n) x[k] = w[kept[j]];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kPackSteps; ++k) {
                const int j = j0 + k * kPackThreads + tid;
                if (j < n) nw[j] = x[k];
            }
        }
        for (int j = n + tid; j < new_width; j += kPackThreads) nw[j] = 0.f;
        return;
    }
    uint4* cache = static_cast<uint4*>((int)blockIdx.x < slices ? p.k_cache : p.v_cache);
    const int32_t* old_row = p.block_tables + (size_t)b * p.max_blocks;
    const int32_t* new_row = p.new_block_tables + (size_t)b * p.new_max_blocks;
    const long long row = (long long)p.num_kv_heads * (p.head_dim / 8);
    const int col = kvh * (p.head_dim / 8) + (int)(blockIdx.x % slices) * 8 + (tid & 7);
    const int bshift = __ffs(p.block_size) - 1;
    for (int seg = 0; seg < n; seg += kPackSegment) {
        const int count = min(n - seg, kPackSegment);
        __syncthreads();  // the previous segment's places have been used
        for (int i = tid; i < (count + p.block_size - 1) >> bshift; i += kPackThreads)
            page[i] = page_phys(new_row, (seg >> bshift) + i, p.new_max_blocks, p.num_blocks);
        for (int i0 = tid; i0 < count; i0 += kPackThreads * 4) {
            int t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kPackThreads;
                t[k] = i < count ? kept[seg + i] : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kPackThreads;
                if (i < count) src[i] = slot_of(old_row, t[k], p.block_size, p.max_blocks, p.num_blocks);
            }
        }
        __syncthreads();
        auto to_of = [&](int i) -> long long {  // slot of the segment's row i, -1: it is not moved
            if (i >= count || src[i] < 0) return -1;
            const int e = page[i >> bshift];
            const long long d = (long long)e * p.block_size + (i & (p.block_size - 1));
            return e < 0 || d == src[i] ? -1 : d;
        };
        uint4 v[2][kPackSteps];
        auto read = [&](int i0, uint4 (&x)[kPackSteps]) {
#pragma unroll
            for (int k = 0; k < kPackSteps; ++k) {
                const int i = i0 + k * kPackRows + (tid >> 3);
                if (to_of(i) >= 0) x[k] = cache[src[i] * row + col];
            }
        };
        auto write = [&](int i0, const uint4 (&x)[kPackSteps]) {
#pragma unroll
            for (int k = 0; k < kPackSteps; ++k) {
                const int i = i0 + k * kPackRows + (tid >> 3);
                const long long d = to_of(i);
                if (d >= 0) cache[d * row + col] = x[k];
            }
        };
        read(0, v[0]);
        for (int i0 = 0; i0 < count; i0 += 2 * kPackChunk) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = i0 + h * kPackChunk;
                if (i >= count) break;  // (the same in every thread)
                read(i + kPackChunk, v[1 - h]);
                __syncthreads();  // the chunk has been read
                write(i, v[h]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict(EvictParams p, bool in_place, bool pdl, cudaStream_t stream) {
    p.in_place = in_place ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    const int64_t width = (int64_t)p.max_blocks * p.block_size;
    int cluster = 1;
    while (cluster < kMaxSelCluster && cluster * (int64_t)kSelShare < width) cluster *= 2;
    p.cluster = cluster;
    const int64_t per = (width / 4 + cluster - 1) / cluster * 4;  // tokens of a CTA at most
    const bool cached = per <= kMaxCached;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    cfg.gridDim = dim3((unsigned)(p.num_kv_heads * cluster), (unsigned)p.batch);
    cfg.blockDim = dim3(kSelThreads);
    cudaError_t e;
    if (cached) {
        static AttrFlags smem_limit;
        e = raise_smem_limit_once(evict_select_kernel<true>, smem_limit);
        if (e != cudaSuccess) return e;
        cfg.dynamicSmemBytes = (size_t)(per + (per / 32 + 1) * 4) * sizeof(uint32_t);
        e = cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, p);
    } else {
        e = cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, p);
    }
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = pdl ? 1 : 0;
    if (in_place) {
        static AttrFlags smem_limit;
        e = raise_smem_limit_once(evict_pack_kernel, smem_limit);
        if (e != cudaSuccess) return e;
        cfg.dynamicSmemBytes = kPackSmem;
        cfg.gridDim = dim3((unsigned)(2 * p.head_dim / 64 + 1), (unsigned)p.num_kv_heads, (unsigned)p.batch);
        cfg.blockDim = dim3(kPackThreads);
        return cudaLaunchKernelEx(&cfg, evict_pack_kernel, p);
    }
    // (the new pages hold at least the budget)
    const int new_width = p.new_max_blocks * p.block_size;
    cfg.gridDim = dim3((unsigned)((new_width + kCopyRows - 1) / kCopyRows), (unsigned)p.num_kv_heads,
                       (unsigned)p.batch);
    cfg.blockDim = dim3(kCopyThreads);
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
}

}  // namespace pa
