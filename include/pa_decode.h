/*
 * pa_decode.h -- C ABI of the GB300 (sm_103a) paged-attention decode library
 * (libpa_decode.so).
 *
 * The operation.  One decode step: every sequence b of a batch has one query
 * token q[b, h, :] per query head h; it attends over the keys and values of
 * its context_lens[b] cached tokens, which live in a pool of fixed-size
 * physical blocks reached through a per-sequence block table:
 *
 *   out[b, h, :] = sum_t softmax_t(scale * q[b, h, :] . K_t) * V_t
 *   K_t = k_cache[block_tables[b][t / block_size], t % block_size, kvh, :]
 *   kvh = h / (num_heads / num_kv_heads)       (grouped-query heads)
 *
 * Sources: MiniVLLM docs "Decoding Benchmark" (sections "What paged attention
 * decode does" and "Block table lookup mechanics"); "benchmark_decoding.py"
 * (reference_output: the float32 definition; setup_test_data: the layouts;
 * the Triton (new) kernel: head grouping and masking of -1 entries);
 * flash-decoding-bench "design.md" (Flash-Decoding: split the KV sequence into
 * chunks processed in parallel, each producing a local max, sum and weighted
 * value sum, then reduce the partials into the output).
 *
 * Layouts (all row-major, contiguous, device memory owned by the caller):
 *   q            [batch, num_heads, head_dim]                      kv_dtype
 *   k_cache      [num_blocks, block_size, num_kv_heads, head_dim]  kv_dtype
 *   v_cache      same shape and dtype as k_cache
 *   block_tables [batch, max_blocks_per_seq]                       int32, -1 = unallocated
 *   context_lens [batch]                                           int32
 *   out          [batch, num_heads, head_dim]                      out_dtype
 *
 * Semantics at the edges (the pages are silent or disagree; this library and
 * its tests take these readings):
 *   - tokens t >= max_blocks_per_seq * block_size are unreachable and ignored;
 *     a negative context length counts as 0;
 *   - a table entry inside the used range that is -1 or outside
 *     [0, num_blocks) excludes its tokens from the softmax (never read);
 *   - a sequence with no attended token gets an all-zero output row.
 *
 * Arithmetic: scores, the online softmax (running max m and normaliser l) and
 * the value accumulation are fp32; K/V/q are fp16 or bf16.  On the way into the
 * product with V a weight is held in two 16-bit parts, on the tile kernel (below)
 * fp16's in one, rounded to 11 bits.  fp16 weights under 2^-25 of the row's
 * largest count as 0 there, in pa_decode_shared_prefix and pa_decode_accumulate
 * those under 2^-32.  `scale` must be
 * finite and > 0 (PA_ERR_INVALID_ARG otherwise).
 *
 * Calls.  All entry points validate on the host and either launch work on
 * `stream` (a cudaStream_t; NULL = the legacy default stream) and return
 * PA_OK immediately, or return an error status and launch nothing.  A
 * PA_ERR_CUDA status means the launch itself failed.  The library allocates no
 * device memory.  Entry points may be called from several host threads; the
 * shared state is a per-device cache of the SM count, of the device error
 * word's address and of which cluster sizes fit, per-thread caches of tensor
 * maps, streams of the library's own (pa_decode_shared_prefix), and the two test
 * switches of pa_set_switch.  No call reads the
 * environment (the tuning variables are read once, when the library loads).
 *
 * Supported shapes: head_dim in {64, 128, 256}; block_size in {16, 32};
 * num_heads / num_kv_heads in {1, 2, 4, 8, 16}; kv_dtype fp16 or bf16; out_dtype
 * fp32 or equal to kv_dtype; every pointer 16-byte aligned.  Anything else
 * returns PA_ERR_UNSUPPORTED (or PA_ERR_INVALID_ARG for inconsistent values).
 */
#ifndef PA_DECODE_H
#define PA_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1, /* null pointer, inconsistent or negative sizes */
    PA_ERR_UNSUPPORTED = 2, /* a shape or dtype this library has no kernel for */
    PA_ERR_WORKSPACE = 3,   /* split-KV workspace missing, misaligned or too small */
    PA_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
    PA_ERR_TIMEOUT = 5      /* a kernel gave up waiting on its own copy pipeline */
} pa_status;

typedef enum pa_dtype { PA_F16 = 0, PA_BF16 = 1, PA_F32 = 2 } pa_dtype;

/* partition_tokens value requesting the balanced split: one CTA per SM, each
 * taking an equal share of all (sequence, kv head, page) triples in order,
 * pieces of a (sequence, kv head) that straddle CTAs combined afterwards.
 * Needs batch <= 512 (otherwise the automatic choice is used). */
#define PA_PARTITION_BALANCED (-1)

typedef struct pa_shape {
    int32_t batch;              /* B >= 0 (B = 0 launches nothing) */
    int32_t num_heads;          /* H, query heads */
    int32_t num_kv_heads;       /* Hkv, H % Hkv == 0 */
    int32_t head_dim;           /* D */
    int32_t block_size;         /* tokens per physical block */
    int32_t max_blocks_per_seq; /* columns of block_tables */
    int64_t num_blocks;         /* physical blocks in the pool, < 2^31 */
    int32_t kv_dtype;           /* pa_dtype of q, k_cache, v_cache: PA_F16 or PA_BF16 */
    int32_t out_dtype;          /* pa_dtype of out: PA_F32 or kv_dtype */
} pa_shape;

/*
 * Single-pass decode ("benchmark_decoding.py", reference_output and the
 * Triton (new) kernel; MiniVLLM docs "Decoding Benchmark", "Why CUDA chunk
 * processing matters"): one CTA per (sequence, kv head) walks all of that
 * sequence's pages, one block-table read per page, with an fp32 online
 * softmax, and writes out[b, h, :] for the head group.
 * Arguments: device pointers as laid out above; `scale` multiplies q.K
 * (1/sqrt(head_dim) in the pages' set-up); `stream` is a cudaStream_t.
 */
pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens,
                    const pa_shape* shape, float scale, void* stream);

/*
 * Bytes of device workspace pa_decode_splitkv needs for this shape, longest
 * context `max_context_len` and partition size `partition_tokens` (tokens per
 * split, a multiple of block_size; 0 = choose automatically for the current
 * device; PA_PARTITION_BALANCED = the balanced split).  Returns 0 for invalid
 * arguments and when no workspace is needed (one partition, or partitions
 * reduced inside a thread-block cluster: see pa_decode_splitkv).  The answer
 * is for the current device, as the call plans with its SM count (which picks
 * the CTA shape and with it whether a cluster split fits); an explicit
 * partition size may be queried without a device, and is then sized as for
 * one SM.  A size that does not fit in a size_t is reported as SIZE_MAX, which
 * no workspace satisfies (the call is then refused with PA_ERR_WORKSPACE).
 */
size_t pa_workspace_size(const pa_shape* shape, int32_t max_context_len,
                         int32_t partition_tokens);

/*
 * Partition size (tokens) the automatic choice picks for `num_sms`
 * multiprocessors: a multiple of block_size (a result >= max_context_len
 * means "no split"), or PA_PARTITION_BALANCED when it picks the balanced
 * split; 0 for invalid arguments.  A function of its arguments, exported so
 * that the choice can be checked without a GPU, with one exception: which
 * cluster sizes fit on the device at once is asked of the current device
 * when there is one (cached per device); without a device, clusters of up to
 * 8 CTAs are assumed to fit.  Launches nothing.
 * The rules are this library's own, fitted to GB300 timings: the
 * flash-decoding-bench design notes only say that the chunk size is picked
 * from the KV length.
 */
int32_t pa_choose_partition_tokens(const pa_shape* shape, int32_t max_context_len,
                                   int32_t num_sms);

/*
 * Flash-Decoding split-KV decode (flash-decoding-bench "design.md": the KV
 * cache is split into chunks, one thread block each, each computing its local
 * max, sum and weighted value sum, followed by a reduction of the partials).
 * Each (sequence, kv head) is cut into partitions of `partition_tokens` tokens
 * (or, with PA_PARTITION_BALANCED, the flattened pages of all of them are cut
 * into one equal share per SM, and a piece that straddles two shares leaves
 * a partial record for the combine kernel);
 * one CTA per partition computes fp32 partials (m, l, acc[head_dim]) for each
 * query head of the group.  The partitions of a (sequence, kv head) are
 * launched as one thread-block cluster and reduced through distributed
 * shared memory inside the same kernel (no workspace needed) when there are
 * at most 8 of them (up to 16 for the automatic choice) and the device can
 * hold every cluster of the call at once; otherwise they write their
 * partials to `workspace` and a second kernel combines them with a
 * log-sum-exp reduction into out.  pa_workspace_size reports which.  `max_context_len` must be >= every context_lens[b] that
 * should be attended in full (tokens beyond it are dropped; no device->host
 * read is made); `partition_tokens` = 0 chooses the split automatically, and a
 * choice of one partition runs the single pass.  `workspace` (device, 16-byte
 * aligned) must hold at least pa_workspace_size(shape, max_context_len,
 * partition_tokens) bytes (may be NULL when that is 0); it is scratch owned by
 * the caller and may be reused once the stream has passed this call.
 * Kernel choice: groups of 16 query heads at head_dim 256 run on the tcgen05
 * tile kernel described at pa_decode_multi (its own split, from the device's
 * resident clusters); every other shape on the warp-level kernel, whose split
 * pa_choose_partition_tokens reports.  PA_PARTITION_BALANCED always runs the
 * warp-level kernel.
 */
pa_status pa_decode_splitkv(void* out, const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens,
                            const pa_shape* shape, float scale, int32_t max_context_len,
                            int32_t partition_tokens, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * Several query tokens per sequence in one call: the decode step of
 * speculative decoding's verification, or a short chunk of new tokens (the
 * pages define only the one-token decode; this is its causal extension, the
 * q_len > 1 attention that the flash-decoding-bench design notes contrast
 * with the q_len = 1 decode).  Layouts:
 *   q    [batch, q_len, num_heads, head_dim]  kv_dtype
 *   out  [batch, q_len, num_heads, head_dim]  out_dtype
 * context_lens[b] counts the q_len new tokens, whose keys and values are
 * already in the cache at positions T - q_len .. T - 1 (T = context_lens[b]).
 * Query token i sits at position T - q_len + i and attends to the tokens
 * t <= T - q_len + i that the table reaches, with the same masking as
 * pa_decode; a query token with no such token gets zeros.  With q_len = 1
 * this is pa_decode_splitkv.
 *
 * Rows.  A (sequence, kv head) has q_len * group rows, one per (query token,
 * head) pair.  Up to 16 rows (except exactly 16 at head_dim 256) the
 * warp-level kernel serves them: its MMA tile's 16 rows hold the pairs, one
 * CTA per floor(16 / group) query tokens of a kv head and partition.  Beyond
 * that the tcgen05 tile kernel serves them: 384-thread CTAs of 128 rows (one
 * per ceil(q_len * group / 128) tiles of a kv head and partition) with
 * Q K^T and P V on the tensor cores (operands staged by TMA in shared memory,
 * S and O accumulated in tensor memory), the online softmax on two
 * warpgroups, and its partitions sized from the device's resident clusters.
 * Either way every CTA of a (sequence, kv head) reads that sequence's pages
 * again, and num_kv_heads times the CTA count per kv head must be <= 65535
 * (else PA_ERR_UNSUPPORTED).  Partitions, workspace and max_context_len as in
 * pa_decode_splitkv; PA_PARTITION_BALANCED is honoured only when
 * q_len * group <= 16 (otherwise the automatic choice is used).  The
 * workspace must hold pa_workspace_size_multi(shape, q_len, ...) bytes.
 * pa_plan_info reports the kernel and split a call will use.
 */
pa_status pa_decode_multi(void* out, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens,
                          const pa_shape* shape, int32_t q_len, float scale,
                          int32_t max_context_len, int32_t partition_tokens, void* workspace,
                          size_t workspace_bytes, void* stream);

/* How a split-KV call (pa_decode_splitkv / pa_decode_multi) with these
 * arguments runs on the current device; filled by pa_plan_info. */
typedef struct pa_plan_desc {
    int32_t kernel;           /* 0: warp-level m16n8k16 kernel; 1: tcgen05 tile kernel */
    int32_t partitions;       /* partitions per (sequence, kv head[, query chunk / tile]) */
    int32_t partition_tokens; /* tokens per partition (the longest context for one) */
    int32_t reduce;           /* 0: none (one pass); 1: cluster (distributed shared
                                 memory); 2: workspace + combine kernel; 3: balanced split */
    int32_t ctas;             /* CTAs of the attention kernel */
    int32_t threads;          /* threads per CTA */
} pa_plan_desc;

/* Describes, without launching anything, the plan a split-KV call with these
 * arguments would use on the current device (no counterpart in the pages: a
 * diagnostic of this library's own choices).  Automatic and balanced choices
 * need the device, as the calls do; an explicit partition size may be
 * queried without one (planned as for one SM).  Returns PA_ERR_INVALID_ARG /
 * PA_ERR_UNSUPPORTED like the calls, else PA_OK. */
pa_status pa_plan_info(const pa_shape* shape, int32_t q_len, int32_t max_context_len,
                       int32_t partition_tokens, pa_plan_desc* desc);

/* Workspace bytes of pa_decode_multi (0 for invalid arguments or when none is
 * needed); pa_workspace_size(shape, ...) is this with q_len = 1. */
size_t pa_workspace_size_multi(const pa_shape* shape, int32_t q_len, int32_t max_context_len,
                               int32_t partition_tokens);

/*
 * Append of each sequence's new token to the paged cache, the step that
 * precedes attention in every decode iteration (MiniVLLM docs "Decoding
 * Benchmark", "What paged attention decode does": the cache is a pool of
 * blocks allocated on demand, token t of sequence b in block
 * block_tables[b][t / block_size] at slot t % block_size).  For each b with
 * 0 <= positions[b] < max_blocks_per_seq * block_size and a table entry in
 * [0, num_blocks): k_cache[entry][positions[b] % block_size][:][:] =
 * k_new[b][:][:], and likewise v_cache from v_new.  Other sequences (padding:
 * a negative position; a masked entry) write nothing.  k_new, v_new:
 * [batch, num_kv_heads, head_dim] in kv_dtype, 16-byte aligned; positions:
 * [batch] int32.  Launched with programmatic stream serialization, so a
 * decode call queued right after it overlaps its launch and still sees every
 * write.  Bit-exact (a copy).
 */
pa_status pa_append_kv(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                       const int32_t* block_tables, const int32_t* positions,
                       const pa_shape* shape, void* stream);

/* Rotary embedding of pa_rope_append_kv.  Strides are in elements between the
 * tokens of the flattened [batch * q_len] order (a token's heads are
 * contiguous), so that q, k_new and v_new may be views of one fused
 * projection's output; each at least a token's row and a multiple of 8. */
typedef struct pa_rope {
    int32_t rotary_dim;   /* R: leading elements of a head that turn, a multiple of 16, <= head_dim */
    int32_t num_axes;     /* position axes (1 for text; time, height, width for video), >= 1 */
    int32_t interleaved;  /* 0: pair j is elements (j, j + R/2); 1: (2j, 2j + 1) */
    int32_t reserved;     /* 0 */
    int64_t q_stride, q_out_stride, k_stride, v_stride;
} pa_rope;

/*
 * Rotary positions with one or several axes for the new tokens, and their
 * append to the cache: the step between a layer's projections and
 * pa_decode_splitkv / pa_decode_multi.  For token i of sequence b, pair j of
 * every query and key head turns by the angle
 *   a = rotary_positions[axes[j]][b][i] * f_j,
 *   (x, y) -> (x cos a - y sin a, x sin a + y cos a);
 * elements from rotary_dim on, and the values, pass through.  The turned
 * query goes to q_out; the turned key and the value go to cache position
 * context_lens[b] - q_len + i of sequence b (context_lens counts the q_len new
 * tokens, as in pa_decode_multi).  Rotary positions and cache positions are
 * apart: an image's patches share a time, and eviction moves tokens to lower
 * slots.  A token at a negative position (padding) or past the table, or whose
 * table entry is masked, is turned into q_out and writes nothing to the cache.
 *   q, q_out          [batch, q_len, num_heads, head_dim]     kv_dtype (q_out may be q,
 *                     with its stride; else none of its rows meets one of q, k_new,
 *                     v_new or the caches: PA_ERR_INVALID_ARG where they do, or
 *                     where arrays of different strides share a range)
 *   k_new, v_new      [batch, q_len, num_kv_heads, head_dim]  kv_dtype
 *   rotary_positions  [num_axes, batch, q_len]  int32, any value
 *   phases            [rotary_dim / 2]  int64: f_j / (2 pi) * 2^64, modulo 2^64
 *   axes              [rotary_dim / 2]  int32; a pair whose axis is outside
 *                     [0, num_axes) does not turn
 * Angles are formed modulo one turn in 64-bit integers, so that a far position
 * is as exact as a near one; sine, cosine and the products are fp32, and each
 * result is rounded once to kv_dtype.  shape->out_dtype is checked and not
 * used.  Two tokens of a call must not share a cache slot.
 */
pa_status pa_rope_append_kv(void* q_out, void* k_cache, void* v_cache, const void* q,
                            const void* k_new, const void* v_new, const int32_t* rotary_positions,
                            const int64_t* phases, const int32_t* axes,
                            const int32_t* block_tables, const int32_t* context_lens,
                            const pa_shape* shape, int32_t q_len, const pa_rope* rope,
                            void* stream);

/*
 * Attention of sequences that share a prefix, whose pages are read once for
 * all of them.  The batch's sequences fall into num_prefixes groups of equal
 * size n = batch / num_prefixes, in order: sequence b has prefix b / n.  The
 * softmax of a sequence's query tokens runs over its prefix's tokens and its
 * own as over one sequence, prefix_lens[b / n] + context_lens[b] tokens long:
 *   prefix_tables  [num_prefixes, max_prefix_blocks]  int32: the prefixes' pages
 *   prefix_lens    [num_prefixes]  int32: any length; the last page may be partial
 *   block_tables, context_lens: the sequences' own pages and lengths, which
 *                  count the q_len query tokens (as in pa_decode_multi); own
 *                  tokens start at slot 0 of the first own page
 *   q, out         [batch, q_len, num_heads, head_dim]
 * Query token i of sequence b attends to the whole prefix and to its own
 * tokens t <= context_lens[b] - q_len + i; where a sequence is shorter than
 * q_len its first query tokens stand for the prefix's last tokens and see no
 * further than they would.  Masked entries, lengths past a table's reach and
 * rows with no token as in pa_decode.
 * Where little is to be read, each sequence reads its prefix's pages before its
 * own, in one launch.  Otherwise
 * the query rows of a prefix's sequences (n * q_len * group per kv head) go
 * through the prefix's pages together, on the kernel that pa_decode_multi
 * takes for as many rows; the sequences' own pages as in pa_decode_multi; a
 * third launch joins the two by their softmax statistics.  The first two run
 * beside each other, the second on a stream of the library's own that starts
 * from `stream` and that `stream` waits for before the third (under capture: a
 * branch of the caller's graph).  max_prefix_len and
 * max_context_len bound the lengths: whatever the plan, prefix tokens past the
 * former's last page are left out, and a sequence's own tokens past the latter's.
 * The workspace must hold pa_workspace_size_shared_prefix(...) bytes (device, 16-byte
 * aligned, free again once the stream has passed the call).
 */
pa_status pa_decode_shared_prefix(void* out, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* prefix_tables,
                                  const int32_t* prefix_lens, const int32_t* block_tables,
                                  const int32_t* context_lens, const pa_shape* shape,
                                  int32_t num_prefixes, int32_t max_prefix_blocks, int32_t q_len,
                                  float scale, int32_t max_prefix_len, int32_t max_context_len,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of pa_decode_shared_prefix on the current device (0 where it
 * needs none, for invalid arguments or without a device; SIZE_MAX when no size_t holds it). */
size_t pa_workspace_size_shared_prefix(const pa_shape* shape, int32_t num_prefixes,
                                       int32_t max_prefix_blocks, int32_t q_len,
                                       int32_t max_prefix_len, int32_t max_context_len);

/*
 * pa_decode_multi (q_len = 1: pa_decode_splitkv) that also adds every cached
 * token's attention weight to a running sum per kv head, from which
 * pa_evict_kv chooses:
 *   weights_out[b][kvh][t] = weights_in[b][kvh][t]
 *                            + sum over the group's heads h and query tokens i of p[b][i][h][t]
 * for t < min(context_lens[b], table reach), p the softmax weights of the
 * call's attention (0 for tokens that a row does not attend to); entries from
 * there on are not written.
 *   weights_in, weights_out  [batch, num_kv_heads, max_blocks_per_seq * block_size]
 *                            fp32; may be the same array, else apart
 * Tokens past max_context_len's last page are left out of the attention and keep
 * their weights; the tables reach at most 2^30 tokens (PA_ERR_UNSUPPORTED).
 * Weights are fp32; each is summed over the rows by one thread in a fixed order,
 * so that equal calls give equal bits.  The other arguments are those
 * of pa_decode_multi with an automatic split; the workspace must hold
 * pa_workspace_size_accumulate(...) bytes.
 */
pa_status pa_decode_accumulate(void* out, float* weights_out, const float* weights_in,
                               const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               const pa_shape* shape, int32_t q_len, float scale,
                               int32_t max_context_len, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Workspace bytes of pa_decode_accumulate on the current device (0 for
 * invalid arguments or without a device; SIZE_MAX when no size_t holds it). */
size_t pa_workspace_size_accumulate(const pa_shape* shape, int32_t q_len, int32_t max_context_len);

/*
 * Eviction from the cache by accumulated attention weight (the weights that
 * pa_decode_accumulate keeps).  Every kv head of a sequence keeps at most
 * `budget` of its min(context_lens[b], table reach) tokens: the first `sink`
 * and the last `recent` ones, and of the others those of the largest weights,
 * equal weights by the lowest index (NaN ranks below every number); tokens of
 * masked pages are never kept.  Kept token number j, in the tokens' order, of
 * each kv head moves to cache position j of new_block_tables[b]; the kv heads
 * choose apart, and all keep the same number, which goes to new_lens[b].
 *   weights           [batch, num_kv_heads, max_blocks_per_seq * block_size]      fp32
 *   new_weights       [batch, num_kv_heads, new_max_blocks_per_seq * block_size]  fp32:
 *                     the kept tokens' weights, zeros from new_lens[b] on
 *   new_block_tables  [batch, new_max_blocks_per_seq]  int32
 *   new_lens          [batch]  int32
 *   kept              [batch, num_kv_heads, budget]  int32: the kept tokens'
 *                     former positions, ascending, -1 from new_lens[b] on
 * new_block_tables (and new_weights) may be block_tables (and weights)
 * themselves: the tokens then move down within their own pages, which no
 * other sequence may share.  Otherwise an entry of new_block_tables is the
 * block of the same entry of block_tables (a copy of the table, or of its first
 * columns: the tokens move down there too, more slowly), or a block that is not
 * among any sequence's old ones; old blocks that are not among the new ones stay
 * as they were.  A kept token whose new entry
 * is masked is not stored.  new_weights, new_lens and kept lie apart from each
 * other and from the inputs.  budget >= sink + recent, and
 * new_max_blocks_per_seq * block_size >= budget; both tables reach at most 2^30
 * tokens (PA_ERR_UNSUPPORTED).  The num_heads and out_dtype
 * of the shape are checked and not used.
 */
pa_status pa_evict_kv(void* k_cache, void* v_cache, const float* weights,
                      const int32_t* block_tables, const int32_t* context_lens,
                      const int32_t* new_block_tables, float* new_weights, int32_t* new_lens,
                      int32_t* kept, const pa_shape* shape, int32_t new_max_blocks_per_seq,
                      int32_t budget, int32_t sink, int32_t recent, void* stream);

/*
 * The 8-bit cache: keys and values as e4m3 floats with an fp32 scale for each
 * page and kv head, half the bytes of the 16-bit cache.
 *   k_cache, v_cache    [num_blocks, block_size, num_kv_heads, head_dim]  e4m3 codes (1 byte)
 *   k_scales, v_scales  [num_blocks, num_kv_heads]  fp32
 * A cached key is k_scales[block][kvh] * code, and a value likewise.
 *
 * pa_rope_append_kv8 is pa_rope_append_kv into that cache: queries and keys turn
 * in the same way, and the turned keys and the values (in fp32, rounded once)
 * become codes.  For each page that the call's tokens fall into, and each kv
 * head, with amax the largest finite magnitude among the call's tokens of the
 * page,
 *   s_new = the smallest power of two with amax <= 448 s_new, in [2^-60, 2^60],
 *   s     = s_new where the page's slot 0 is among the call's tokens,
 *           else max(s_old, s_new), s_old the scale that the page has;
 * codes are x / s rounded to nearest even; where s > s_old the page's slots before the
 * call's tokens are rounded anew, as code * s_old / s (for powers of two
 * exact but below 2^-6).  Slots behind the call's tokens stay as they are.
 * Infinities and magnitudes past 448 * 2^60 become NaN, NaN stays NaN.  A page
 * that takes tokens belongs to one sequence of the call, at one place of its table.
 * shape->kv_dtype is the dtype of q, q_out, k_new and v_new; the other
 * arguments, the strides of `rope` and what q_out may lie over are as for
 * pa_rope_append_kv, and q_out lies apart from the scales too.
 */
pa_status pa_rope_append_kv8(void* q_out, void* k_cache, void* v_cache, float* k_scales,
                             float* v_scales, const void* q, const void* k_new, const void* v_new,
                             const int32_t* rotary_positions, const int64_t* phases,
                             const int32_t* axes, const int32_t* block_tables,
                             const int32_t* context_lens, const pa_shape* shape, int32_t q_len,
                             const pa_rope* rope, void* stream);

/*
 * pa_decode_multi (q_len = 1: pa_decode_splitkv) over the 8-bit cache, with the
 * same masking and an automatic split.  Codes are widened exactly; the scores,
 * the softmax and the sums are fp32, the normaliser of every attended token's
 * softmax weight as it is.  On the way into the product with the values a token
 * counts with its softmax weight times its page's v_scale: that product is held in
 * two fp16 parts, rounded once to fp16 (by at most 2^-11 of it) where out is bf16, and
 * one under 2^-32 of the row's largest adds nothing to the output.  A NaN or infinity in a cached value or scale that one
 * row attends to may reach its sequence's other rows.  Scales are finite and positive, whoever wrote them;
 * v_scales outside [2^-60, 2^60] count as the nearer limit.  Scales of pages
 * that hold no attended token are not used.  shape->kv_dtype is
 * the dtype of q, shape->out_dtype fp32 or that.  Tokens past
 * max_context_len's last page are left out whatever the plan.  out lies apart from the
 * other arguments (PA_ERR_INVALID_ARG).  The workspace must hold
 * pa_workspace_size_kv8(...) bytes (device, 16-byte aligned, free again once
 * the stream has passed the call).
 */
pa_status pa_decode_kv8(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const float* k_scales, const float* v_scales, const int32_t* block_tables,
                        const int32_t* context_lens, const pa_shape* shape, int32_t q_len,
                        float scale, int32_t max_context_len, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Workspace bytes of pa_decode_kv8 on the current device (0 where it needs none,
 * for invalid arguments or without a device): enough for every batch up to
 * shape->batch and every announced length up to max_context_len, the rest the same. */
size_t pa_workspace_size_kv8(const pa_shape* shape, int32_t q_len, int32_t max_context_len);

/*
 * The latent cache: one vector a token for all heads, whose first latent_dim
 * elements are both the key's first part and the value, followed by the key's
 * positional part of rope_dim elements.
 *   cache  [num_blocks, block_size, latent_dim + rope_dim]  dtype
 * latent_dim in {128, 256, 512}, rope_dim 64, block_size in {16, 32, 64}, any
 * num_heads up to 65535.
 */
typedef struct pa_latent_shape {
    int32_t batch;              /* B >= 0 (B = 0 launches nothing) */
    int32_t num_heads;          /* H >= 1 */
    int32_t latent_dim;
    int32_t rope_dim;
    int32_t block_size;
    int32_t max_blocks_per_seq; /* columns of block_tables */
    int64_t num_blocks;         /* < 2^31 */
    int32_t dtype;              /* PA_F16 or PA_BF16: q, out, cache, new vectors, norm weight */
    int32_t reserved;           /* 0 (else PA_ERR_INVALID_ARG) */
} pa_latent_shape;

/* Norm and rotary embedding of pa_rope_append_latent.  Strides in elements,
 * multiples of 8: between the tokens of the flattened [batch * q_len] order and
 * between the heads of a token (>= rope_dim; a token's stride spans its heads). */
typedef struct pa_latent_rope {
    int32_t interleaved;  /* 0: pair j is elements (j, j + 32); 1: (2j, 2j + 1) */
    float eps;            /* >= 0, finite */
    int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
    int64_t new_stride;   /* >= latent_dim + rope_dim */
} pa_latent_rope;

/*
 * Append to the latent cache.  The latent part x of each new token becomes
 *   y = x / sqrt(mean(x^2) + eps) * norm_weight
 * (fp32, rounded once; norm_weight NULL: x as it is), its positional part and
 * that of every query head turn by the angle rotary_positions[b][i] * f_j per
 * pair, as in pa_rope_append_kv; the token's vector goes to cache position
 * context_lens[b] - q_len + i of sequence b (tokens without a slot store nothing)
 * and the turned queries to q_out.
 *   q, q_out          [batch, q_len, num_heads, rope_dim]   views with strides; q_out may be q
 *                     (same strides); else their rows lie apart from each other, from
 *                     latent_new's and from the cache: PA_ERR_INVALID_ARG where rows
 *                     meet, or where arrays of different token strides share a range
 *   latent_new        [batch, q_len, latent_dim + rope_dim]
 *   norm_weight       [latent_dim]
 *   rotary_positions  [batch, q_len]  int32, any value
 *   phases            [rope_dim / 2]  int64, as for pa_rope_append_kv
 */
pa_status pa_rope_append_latent(void* q_out, void* cache, const void* q, const void* latent_new,
                                const void* norm_weight, const int32_t* rotary_positions,
                                const int64_t* phases, const int32_t* block_tables,
                                const int32_t* context_lens, const pa_latent_shape* shape,
                                int32_t q_len, const pa_latent_rope* rope, void* stream);

/*
 * Attention over the latent cache (the absorbed form: the up-projections of
 * keys and values are applied to the query before and to the output after):
 *   out[b, i, h, :] = sum_t softmax_t(scale * q[b, i, h, :] . c_t) * c_t[: latent_dim]
 * over the tokens t <= context_lens[b] - q_len + i that the table reaches,
 * with the masking of pa_decode_multi.
 *   q    [batch, q_len, num_heads, latent_dim + rope_dim]
 *   out  [batch, q_len, num_heads, latent_dim], apart from the other arguments
 * Scores, softmax and sums are fp32.  On the way into the product with the values a
 * weight is held in two bf16 parts, in a bf16 cache of latent_dim 512 with more than
 * 32 rows (q_len * num_heads) in one, rounded to 8 bits, in an fp16 cache in one,
 * rounded to 11 bits (those under 2^-32 of the row's largest count as 0); the
 * normaliser sums weights in one part as rounded.  A NaN or infinity in a
 * cached vector that one row attends to may reach its sequence's other rows.
 * Tokens past max_context_len's last page are left out.  The workspace must
 * hold pa_workspace_size_latent(...) bytes.
 */
pa_status pa_decode_latent(void* out, const void* q, const void* cache,
                           const int32_t* block_tables, const int32_t* context_lens,
                           const pa_latent_shape* shape, int32_t q_len, float scale,
                           int32_t max_context_len, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Workspace bytes of pa_decode_latent on the current device (0 where it needs
 * none, for invalid arguments or without a device): enough for every batch up to
 * shape->batch and every announced length up to max_context_len, the rest the same. */
size_t pa_workspace_size_latent(const pa_latent_shape* shape, int32_t q_len,
                                int32_t max_context_len);

/*
 * Test export of the page walk (MiniVLLM docs "Decoding Benchmark", "Block
 * table lookup mechanics"): out_phys[b][j] (device, int32, [batch,
 * max_blocks_per_seq]) = the physical block the decode kernels read for
 * logical page j of sequence b, or -1 where that page holds no attended token
 * (beyond the context, or a masked entry).  Uses the kernels' own page-walk
 * code.
 */
pa_status pa_resolve_blocks(int32_t* out_phys, const int32_t* block_tables,
                            const int32_t* context_lens, const pa_shape* shape, void* stream);

/*
 * Reads and clears the current device's error word, which a kernel sets when
 * a bounded wait on its own copy pipeline runs out (it then abandons the
 * work and returns instead of hanging).  Synchronises `stream`.  *code is 0
 * or the pa_status the kernel recorded.
 */
pa_status pa_device_error(int32_t* code, void* stream);

/*
 * pa_decode_splitkv without a caller-supplied workspace, for callers that
 * cannot allocate device memory: for instance code that runs inside a host
 * application which hands it only fixed input/output buffers and forbids
 * further allocation, or a latency-critical loop that must not pay for
 * cudaMalloc's device-wide synchronisation.  (The pages have no counterpart;
 * this is a convenience of this library.)
 *
 * The split-KV partials go to a fixed scratch array inside the library, 16 MiB
 * of device memory on every GPU that loads it, held until the process exits.
 * A call whose partials need more than that -- batch * num_heads * partitions
 * * (head_dim + 2) * 4 bytes, plus alignment -- returns PA_ERR_WORKSPACE and
 * launches nothing; use pa_decode_splitkv with your own workspace then.  The
 * call allocates nothing and needs no clearing of the scratch.
 *
 * The first call on a device looks up that device's scratch address
 * (cudaGetSymbolAddress); make that first call before any stream capture.
 * All calls on a device share the one array, which keeps the last call's
 * contents: two calls that can run at the same time on the GPU (different
 * streams without ordering between them) race on it and both results are then
 * undefined.  Other arguments and behaviour are those of pa_decode_splitkv.
 */
pa_status pa_decode_splitkv_noalloc(void* out, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* block_tables,
                                    const int32_t* context_lens, const pa_shape* shape,
                                    float scale, int32_t max_context_len,
                                    int32_t partition_tokens, void* stream);

/*
 * Test export of the kernels' failure path (no counterpart in the pages): one
 * CTA waits, with the decode kernels' bounded wait, on an mbarrier that nothing
 * ever completes; after `timeout_ns` (1 ns .. 5 s) it gives up and records
 * PA_ERR_TIMEOUT in the device error word, which pa_device_error then returns.
 * The context stays usable.  Asynchronous on `stream`.
 */
pa_status pa_selftest_wait_timeout(uint64_t timeout_ns, void* stream);

/*
 * Test and tuning switches (no counterpart in the pages: they choose between
 * this library's own kernels, whose results agree up to rounding order).
 *   PA_SWITCH_MULTI_KERNEL    PA_KERNEL_AUTO (default): the library's choice;
 *                             PA_KERNEL_MMA: the warp-level kernel for every
 *                             q_len > 1 call; PA_KERNEL_TILE: the tcgen05 tile
 *                             kernel for every split-KV / multi-token call
 *   PA_SWITCH_TILE_COMPACT_Q  1 (default): the tile kernel stages only 16 Q rows
 *                             for units of at most 16 rows at head_dim 256;
 *                             0: it stages whole 128-row tiles
 * The initial values come from the environment variables PA_MULTI_KERNEL
 * (mma | tile) and PA_TILE_COMPACT_Q (0), read once when the library is
 * loaded; no call reads the environment.  pa_set_switch changes a switch for
 * every later call of the process (a relaxed atomic store: set it while no
 * other host thread is between a pa_workspace_size query and the call it
 * sizes).  Returns PA_ERR_INVALID_ARG for an unknown switch or value.
 * pa_get_switch returns the current value, -1 for an unknown switch.
 */
enum { PA_SWITCH_MULTI_KERNEL = 0, PA_SWITCH_TILE_COMPACT_Q = 1 };
enum { PA_KERNEL_AUTO = 0, PA_KERNEL_MMA = 1, PA_KERNEL_TILE = 2 };
pa_status pa_set_switch(int32_t which, int32_t value);
int32_t pa_get_switch(int32_t which);

/* Static, human-readable name of a status. */
const char* pa_status_string(pa_status status);

#ifdef __cplusplus
}
#endif

#endif /* PA_DECODE_H */
