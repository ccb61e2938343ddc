// Host side of the 8-bit cache (pa_rope_append_kv8, pa_decode_kv8) and of the
// latent cache (pa_rope_append_latent, pa_decode_latent).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pa_internal.h"

using namespace pa;

namespace {

struct Span {
    const void* p;
    size_t n;
};

bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.n && b.n && x < y + b.n && y < x + a.n;
}

// One array of `tokens` rows of 16-bit elements, `stride` apart.
struct Rows {
    const void* p;
    int64_t row, stride;
    Span span(int64_t tokens) const { return {p, ((size_t)(tokens - 1) * stride + row) * 2}; }
};

// Do rows of two arrays share a byte?  Rows of one stride meet if they do
// modulo the stride (slices of one fused buffer do not); arrays of different
// strides are taken to where they share a range.
bool rows_meet(const Rows& a, const Rows& b, int64_t tokens) {
    if (!overlap(a.span(tokens), b.span(tokens))) return false;
    if (a.stride != b.stride || tokens == 1) return true;
    const int64_t stride = a.stride * 2;
    const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
    const int64_t at = ((apart % stride) + stride) % stride;  // a's rows begin here in b's stride
    return at < b.row * 2 || at + a.row * 2 > stride;
}

bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.f; }

pa_status check_latent(const pa_latent_shape* s) {
    if (!s) return PA_ERR_INVALID_ARG;
    if (s->batch < 0 || s->num_heads <= 0 || s->latent_dim <= 0 || s->rope_dim <= 0 ||
        s->block_size <= 0 || s->max_blocks_per_seq <= 0 || s->num_blocks <= 0 || s->reserved != 0)
        return PA_ERR_INVALID_ARG;
    if (s->dtype != PA_F16 && s->dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (s->latent_dim != 128 && s->latent_dim != 256 && s->latent_dim != 512) return PA_ERR_UNSUPPORTED;
    if (s->rope_dim != 64) return PA_ERR_UNSUPPORTED;
    if (s->block_size != 16 && s->block_size != 32 && s->block_size != 64) return PA_ERR_UNSUPPORTED;
    if (s->batch > 65535 || s->num_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (s->num_blocks >= (int64_t(1) << 31)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)s->max_blocks_per_seq * s->block_size > (1 << 30)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

pa_status check_latent_call(const pa_latent_shape* s, int32_t q_len) {
    const pa_status st = check_latent(s);
    if (st != PA_OK) return st;
    if (q_len < 1) return PA_ERR_INVALID_ARG;
    // rows of a sequence, and row tiles of a call, inside 31 bits
    const int64_t rows = (int64_t)q_len * s->num_heads;
    if (rows > (1 << 24) || rows * s->batch > (1ll << 31) - 1 || s->batch * ((rows + 15) / 16) > 65535 * 64ll)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Tokens of the pages that max_context_len announces, inside the table's reach.
int announced_tokens(int32_t max_context_len, int block_size, int max_blocks) {
    const int64_t t = max_context_len < 1 ? 1 : max_context_len;
    const int64_t pages = (t + block_size - 1) / block_size;
    return (int)((pages < max_blocks ? pages : max_blocks) * block_size);
}

pa_status done(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

pa_status check_kv8(const pa_shape* s, int32_t q_len) {
    const pa_status st = check_shape(s);
    if (st != PA_OK) return st;
    if (q_len < 1) return PA_ERR_INVALID_ARG;
    // rows of a sequence, units of a call and tokens of a table inside 31 bits
    if ((int64_t)q_len * s->num_heads > (1 << 24)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)s->batch * s->num_heads * q_len > (1ll << 31) - 1) return PA_ERR_UNSUPPORTED;
    if ((int64_t)s->max_blocks_per_seq * s->block_size > (1 << 30)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// How a call over the 8-bit cache runs.
struct Kv8Plan {
    int kind;             // index of the kernel in kKv8
    int chunk, chunks;    // query tokens of a CTA, and how many CTAs that makes
    int64_t units;        // (sequence, kv head, chunk)
    int group_size, unit_groups;
    bool balanced;
    int cluster, part_steps;
    int64_t ctas;
    size_t ml_at, desc_at, bytes;  // workspace
};

// The kernels by head_dim and rows of a CTA.
struct Kv8Kernel {
    int head_dim, rows;
    cudaError_t (*launch)(const Kv8Launch&, cudaStream_t);
    int (*ctas)();
};
const Kv8Kernel kKv8[] = {{64, 8, launch_kv8_d64_n1, kv8_ctas_d64_n1},
                          {64, 16, launch_kv8_d64_n2, kv8_ctas_d64_n2},
                          {64, 32, launch_kv8_d64_n4, kv8_ctas_d64_n4},
                          {128, 8, launch_kv8_d128_n1, kv8_ctas_d128_n1},
                          {128, 16, launch_kv8_d128_n2, kv8_ctas_d128_n2},
                          {128, 32, launch_kv8_d128_n4, kv8_ctas_d128_n4},
                          {256, 8, launch_kv8_d256_n1, kv8_ctas_d256_n1},
                          {256, 16, launch_kv8_d256_n2, kv8_ctas_d256_n2}};
constexpr int kKv8Count = sizeof kKv8 / sizeof kKv8[0];

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Largest batch whose lengths every CTA looks through for its run (2 us).
constexpr int kMaxBalancedLens = 2048;

// Few units, up to 32 steps to a CTA: clusters of up to 8 CTAs and no second launch
// (8 kv heads; 8 sequences of 4 x 3000 tokens: 17.7 us against 27.3 in runs).  Up to 64
// steps where they fill more than half of the GPU (4 sequences of 16,384 tokens 28 us
// against 34 in runs, of 1000 .. 16,384 25.5 against 24; but one of 16,384 20 against 15).
// Else equal runs of steps over the CTAs that the GPU holds (64 sequences of 1 .. 4096
// tokens 57 us with the join, a unit to a CTA 62; 16 of 1 .. 16,384: 55 and 130).
// With more than 3 units for each of them, where the waves even out by themselves (128
// sequences of 1 .. 2048: 57 us against 60 in runs), of contexts up to 48 steps (64
// sequences of 100 .. 1500: 30 us against 34), or with more lengths than a CTA looks
// through, a unit to a CTA.
Kv8Plan plan_kv8(const pa_shape* s, int32_t q_len, int32_t max_context_len, int sms) {
    Kv8Plan pl;
    // the smallest row tile that holds a sequence's rows, or the largest there is
    const int group = s->num_heads / s->num_kv_heads;
    pl.kind = -1;
    for (int i = 0; i < kKv8Count; ++i)
        if (kKv8[i].head_dim == s->head_dim &&
            (pl.kind < 0 || (int64_t)q_len * group > kKv8[pl.kind].rows))
            pl.kind = i;
    const int per = kKv8[pl.kind].rows / group;
    pl.chunk = q_len < per ? q_len : per;
    pl.chunks = (q_len + pl.chunk - 1) / pl.chunk;
    const int64_t steps = ceil_div(announced_tokens(max_context_len, s->block_size, s->max_blocks_per_seq), 32);
    pl.units = (int64_t)s->batch * s->num_kv_heads * pl.chunks;
    const int64_t slots = (int64_t)sms * kKv8[pl.kind].ctas();
    const int64_t fill = slots / pl.units;
    pl.balanced = false;
    pl.cluster = 1;
    // (a power of two: clusters of 7 that fill the GPU took 12.8 us where 4 took 7.8)
    int64_t in_cluster = 8;
    while (in_cluster > 1 && in_cluster > std::min(fill, ceil_div(steps, 2))) in_cluster /= 2;
    const int64_t most = 2 * in_cluster * pl.units > slots ? 64 : 32;
    if (in_cluster >= 2 && ceil_div(steps, in_cluster) <= most) pl.cluster = (int)in_cluster;
    if (pl.cluster == 1 && steps > 48)
        pl.balanced = pl.units <= 3 * slots && s->batch <= kMaxBalancedLens;
    pl.part_steps = (int)ceil_div(steps, pl.cluster);
    const int64_t per_seq = (int64_t)s->num_kv_heads * pl.chunks;
    pl.unit_groups = (int)ceil_div(per_seq, 32);
    pl.group_size = (int)ceil_div(per_seq, pl.unit_groups);
    pl.ctas = pl.units * pl.cluster;
    if (pl.balanced)
        pl.ctas = std::max<int64_t>(std::min(slots / pl.group_size, (int64_t)s->batch * pl.unit_groups * steps), 1) *
                  pl.group_size;
    pl.ml_at = pl.desc_at = pl.bytes = 0;
    if (pl.balanced) {
        const size_t rows = (size_t)pl.ctas * 2 * kKv8[pl.kind].rows;
        pl.ml_at = up256(rows * s->head_dim * 4);
        pl.desc_at = up256(pl.ml_at + rows * 8);
        pl.bytes = pl.desc_at + (size_t)pl.units * sizeof(PieceDesc);
    }
    return pl;
}

// Workspace that serves every batch up to this one and every context up to this
// length.  More steps never need less; more sequences do, where a cluster or a CTA
// takes a unit, so the largest batches of each rule of plan_kv8 are asked: units
// up to a 16th, 8th, 4th and half of the slots, and the largest batch of runs.
size_t kv8_bytes_up_to(const pa_shape* s, int32_t q_len, int32_t max_context_len, int sms) {
    const Kv8Plan pl = plan_kv8(s, q_len, max_context_len, sms);
    const int64_t per_seq = pl.units / s->batch, slots = (int64_t)sms * kKv8[pl.kind].ctas();
    const int64_t runs = std::min<int64_t>(3 * slots / per_seq, kMaxBalancedLens);
    size_t bytes = pl.bytes;
    pa_shape less = *s;
    for (const int64_t batch : {runs, slots / (2 * per_seq), slots / (4 * per_seq), slots / (8 * per_seq),
                                slots / (16 * per_seq)}) {
        if (batch < 1 || batch >= s->batch) continue;
        less.batch = (int32_t)batch;
        bytes = std::max(bytes, plan_kv8(&less, q_len, max_context_len, sms).bytes);
    }
    return bytes;
}

// How a call over the latent cache runs: row tiles of 16, 32 or 64, the CTAs in
// groups that walk the same tokens; equal runs of tiles over one CTA an SM,
// whatever the lengths, where the batch is small enough for each CTA to look
// all lengths through (2048: 2 us), else one group to a (sequence, row group).
struct LatentPlan {
    int row_tile, row_tiles, row_groups, group_size;
    bool balanced;
    int64_t ctas;
    size_t ml_at, desc_at, bytes;  // workspace; bytes 0: no sequence can be cut
};

LatentPlan plan_latent(const pa_latent_shape* s, int32_t q_len, int32_t max_context_len, int sms) {
    LatentPlan pl;
    const int64_t rows = (int64_t)q_len * s->num_heads;
    pl.row_tile = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    pl.row_tiles = (int)ceil_div(rows, pl.row_tile);
    pl.row_groups = (int)ceil_div(pl.row_tiles, 8);
    pl.group_size = (int)ceil_div(pl.row_tiles, pl.row_groups);
    pl.balanced = s->batch <= kMaxBalancedLens;
    int64_t groups = (int64_t)s->batch * pl.row_groups;
    if (pl.balanced) {
        const int64_t tiles = ceil_div(announced_tokens(max_context_len, s->block_size, s->max_blocks_per_seq), 64);
        groups = std::max<int64_t>(std::min<int64_t>(sms / pl.group_size, groups * tiles), 1);
    }
    pl.ctas = groups * pl.group_size;
    pl.ml_at = pl.desc_at = pl.bytes = 0;
    if (pl.balanced && groups > 1) {
        const size_t records = (size_t)pl.ctas * 2 * pl.row_tile;
        pl.ml_at = up256(records * s->latent_dim * 4);
        pl.desc_at = up256(pl.ml_at + records * 8);
        pl.bytes = pl.desc_at + (size_t)s->batch * pl.row_tiles * sizeof(PieceDesc);
    }
    return pl;
}

}  // namespace

extern "C" {

pa_status pa_rope_append_kv8(void* q_out, void* k_cache, void* v_cache, float* k_scales,
                             float* v_scales, const void* q, const void* k_new, const void* v_new,
                             const int32_t* rotary_positions, const int64_t* phases,
                             const int32_t* axes, const int32_t* block_tables,
                             const int32_t* context_lens, const pa_shape* shape, int32_t q_len,
                             const pa_rope* rope, void* stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (!rope || q_len < 1 || rope->num_axes < 1 || rope->rotary_dim < 0 ||
        rope->rotary_dim > shape->head_dim || (rope->interleaved != 0 && rope->interleaved != 1))
        return PA_ERR_INVALID_ARG;
    if (rope->rotary_dim == 0 || rope->rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    const int64_t q_row = (int64_t)shape->num_heads * shape->head_dim;
    const int64_t kv_row = (int64_t)shape->num_kv_heads * shape->head_dim;
    if (rope->q_stride < q_row || rope->q_out_stride < q_row || rope->k_stride < kv_row ||
        rope->v_stride < kv_row)
        return PA_ERR_INVALID_ARG;
    if (rope->q_stride % 8 || rope->q_out_stride % 8 || rope->k_stride % 8 || rope->v_stride % 8)
        return PA_ERR_UNSUPPORTED;
    // query items of a page's tokens, and the tokens of a call, in 31 bits
    const int64_t tokens = (int64_t)shape->batch * q_len;
    if (q_row / 16 > (1 << 25) || tokens > (1ll << 31) - 1 || q_len > (1 << 30)) return PA_ERR_UNSUPPORTED;
    if (shape->batch == 0) return PA_OK;
    if (!q_out || !k_cache || !v_cache || !k_scales || !v_scales || !q || !k_new || !v_new ||
        !rotary_positions || !phases || !axes || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) ||
        !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(phases, 8) ||
        !aligned(rotary_positions, 4) || !aligned(axes, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(k_scales, 4) || !aligned(v_scales, 4))
        return PA_ERR_INVALID_ARG;
    if (q_out == q && rope->q_out_stride != rope->q_stride) return PA_ERR_INVALID_ARG;
    // what one CTA writes others may still be to read: every output apart from
    // the others and from the inputs
    const Rows qo{q_out, q_row, rope->q_out_stride}, qi{q, q_row, rope->q_stride},
        kn{k_new, kv_row, rope->k_stride}, vn{v_new, kv_row, rope->v_stride};
    if ((q_out != q && rows_meet(qo, qi, tokens)) || rows_meet(qo, kn, tokens) || rows_meet(qo, vn, tokens))
        return PA_ERR_INVALID_ARG;
    const size_t cache = (size_t)shape->num_blocks * shape->block_size * (size_t)kv_row;
    const size_t scales = (size_t)shape->num_blocks * shape->num_kv_heads * 4;
    const size_t pairs = (size_t)rope->rotary_dim / 2;
    const Span outs[5] = {qo.span(tokens), {k_cache, cache}, {v_cache, cache}, {k_scales, scales},
                          {v_scales, scales}};
    const Span ins[8] = {{rotary_positions, (size_t)tokens * rope->num_axes * 4},
                         {phases, pairs * 8},
                         {axes, pairs * 4},
                         {block_tables, (size_t)shape->batch * shape->max_blocks_per_seq * 4},
                         {context_lens, (size_t)shape->batch * 4},
                         qi.span(tokens),
                         kn.span(tokens),
                         vn.span(tokens)};
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < (o == 0 ? 5 : 8); ++i)  // (q_out's rows against q, k_new and v_new: above)
            if (overlap(outs[o], ins[i])) return PA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlap(outs[o], outs[i])) return PA_ERR_INVALID_ARG;
    }
    st = device_state(nullptr, nullptr);
    if (st != PA_OK) return st;
    Append8Params p;
    std::memset(&p, 0, sizeof p);
    p.q_out = q_out;
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.positions = rotary_positions;
    p.phases = phases;
    p.axes = axes;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_blocks = shape->num_blocks;
    p.q_stride = rope->q_stride;
    p.k_stride = rope->k_stride;
    p.v_stride = rope->v_stride;
    p.q_out_stride = rope->q_out_stride;
    p.batch = shape->batch;
    p.q_len = q_len;
    p.num_heads = shape->num_heads;
    p.num_kv_heads = shape->num_kv_heads;
    p.head_dim = shape->head_dim;
    p.block_size = shape->block_size;
    p.max_blocks = shape->max_blocks_per_seq;
    p.rotary_dim = rope->rotary_dim;
    p.num_axes = rope->num_axes;
    p.interleaved = rope->interleaved;
    return done(launch_append8(p, shape->kv_dtype == PA_BF16, use_pdl(),
                               static_cast<cudaStream_t>(stream)));
}

size_t pa_workspace_size_kv8(const pa_shape* shape, int32_t q_len, int32_t max_context_len) {
    int sms = 0;
    if (check_kv8(shape, q_len) != PA_OK || max_context_len < 0 || shape->batch == 0 ||
        device_state(&sms, nullptr) != PA_OK)
        return 0;
    return kv8_bytes_up_to(shape, q_len, max_context_len, sms);
}

pa_status pa_decode_kv8(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const float* k_scales, const float* v_scales, const int32_t* block_tables,
                        const int32_t* context_lens, const pa_shape* shape, int32_t q_len,
                        float scale, int32_t max_context_len, void* workspace,
                        size_t workspace_bytes, void* stream) {
    pa_status st = check_kv8(shape, q_len);
    if (st != PA_OK) return st;
    if (max_context_len < 0 || !scale_ok(scale)) return PA_ERR_INVALID_ARG;
    if (shape->batch == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    const int D = shape->head_dim, Hkv = shape->num_kv_heads, BS = shape->block_size;
    const size_t rows = (size_t)shape->batch * q_len * shape->num_heads;
    const size_t cache = (size_t)shape->num_blocks * BS * Hkv * D;
    const size_t scales = (size_t)shape->num_blocks * Hkv * 4;
    const Span o{out, rows * D * (shape->out_dtype == PA_F32 ? 4 : 2)};
    const Span ins[7] = {{q, rows * D * 2},
                         {k_cache, cache},
                         {v_cache, cache},
                         {k_scales, scales},
                         {v_scales, scales},
                         {block_tables, (size_t)shape->batch * shape->max_blocks_per_seq * 4},
                         {context_lens, (size_t)shape->batch * 4}};
    for (const Span& i : ins)
        if (overlap(o, i)) return PA_ERR_INVALID_ARG;
    int sms = 0;
    int32_t* err = nullptr;
    st = device_state(&sms, &err);
    if (st != PA_OK) return st;
    const Kv8Plan pl = plan_kv8(shape, q_len, max_context_len, sms);
    if (pl.bytes) {
        if (!workspace || !aligned(workspace, 16) || workspace_bytes < pl.bytes) return PA_ERR_WORKSPACE;
        const Span w{workspace, pl.bytes};
        if (overlap(w, o)) return PA_ERR_INVALID_ARG;
        for (const Span& i : ins)
            if (overlap(w, i)) return PA_ERR_INVALID_ARG;
    }
    Kv8Launch L;
    std::memset(&L, 0, sizeof L);
    // one kv head's rows of a page (a column block of at most 128 bytes), swizzled for the lanes' loads
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)Hkv, (uint64_t)BS, (uint64_t)shape->num_blocks};
    const uint64_t strides[3] = {(uint64_t)D, (uint64_t)D * Hkv, (uint64_t)D * Hkv * BS};
    const uint32_t box[4] = {D < 128 ? (uint32_t)D : 128u, 1u, (uint32_t)BS, 1u};
    const CUtensorMapSwizzle swizzle = D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    st = encode_tiled(&L.tmap_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, k_cache, dims, strides, box, swizzle);
    if (st == PA_OK)
        st = encode_tiled(&L.tmap_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, v_cache, dims, strides, box, swizzle);
    if (st != PA_OK) return st;
    Kv8Params& p = L.p;
    p.q = q;
    p.out = out;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    char* ws = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + pl.ml_at);
    p.part_desc = reinterpret_cast<PieceDesc*>(ws + pl.desc_at);
    p.err = err;
    p.timeout_ns = kDefaultTimeoutNs;
    p.num_blocks = shape->num_blocks;
    p.qscale = scale * 1.4426950408889634f;  // log2(e)
    p.batch = shape->batch;
    p.q_len = q_len;
    p.num_heads = shape->num_heads;
    p.num_kv_heads = Hkv;
    p.group = shape->num_heads / Hkv;
    p.max_blocks = shape->max_blocks_per_seq;
    p.q_chunk = pl.chunk;
    p.chunks = pl.chunks;
    p.group_size = pl.group_size;
    p.unit_groups = pl.unit_groups;
    p.bf16 = shape->kv_dtype == PA_BF16;
    p.token_limit = announced_tokens(max_context_len, BS, shape->max_blocks_per_seq);
    p.balanced = pl.balanced ? 1 : 0;
    p.cluster = pl.cluster;
    p.part_steps = pl.part_steps;
    p.out_dtype = shape->out_dtype;
    L.block_size = BS;
    L.units = (int)pl.units;
    L.pdl = use_pdl();
    L.grid = dim3((unsigned)pl.ctas);
    return done(kKv8[pl.kind].launch(L, static_cast<cudaStream_t>(stream)));
}

pa_status pa_rope_append_latent(void* q_out, void* cache, const void* q, const void* latent_new,
                                const void* norm_weight, const int32_t* rotary_positions,
                                const int64_t* phases, const int32_t* block_tables,
                                const int32_t* context_lens, const pa_latent_shape* shape,
                                int32_t q_len, const pa_latent_rope* rope, void* stream) {
    pa_status st = check_latent(shape);
    if (st != PA_OK) return st;
    if (!rope || q_len < 1 || (rope->interleaved != 0 && rope->interleaved != 1) ||
        !std::isfinite(rope->eps) || rope->eps < 0.f)
        return PA_ERR_INVALID_ARG;
    const int W = shape->latent_dim + shape->rope_dim;
    if (rope->q_head_stride < shape->rope_dim || rope->q_out_head_stride < shape->rope_dim ||
        rope->new_stride < W || rope->q_head_stride > (1 << 30) || rope->q_out_head_stride > (1 << 30))
        return PA_ERR_INVALID_ARG;
    const int64_t q_row = (shape->num_heads - 1) * rope->q_head_stride + shape->rope_dim;
    const int64_t out_row = (shape->num_heads - 1) * rope->q_out_head_stride + shape->rope_dim;
    if (rope->q_token_stride < q_row || rope->q_out_token_stride < out_row) return PA_ERR_INVALID_ARG;
    if (rope->q_token_stride % 8 || rope->q_head_stride % 8 || rope->q_out_token_stride % 8 ||
        rope->q_out_head_stride % 8 || rope->new_stride % 8)
        return PA_ERR_UNSUPPORTED;
    const int64_t tokens = (int64_t)shape->batch * q_len;
    if (tokens > (1ll << 31) - 1) return PA_ERR_UNSUPPORTED;
    if (shape->batch == 0) return PA_OK;
    if (!q_out || !cache || !q || !latent_new || !rotary_positions || !phases || !block_tables ||
        !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(q_out, 16) || !aligned(cache, 16) || !aligned(q, 16) || !aligned(latent_new, 16) ||
        !aligned(norm_weight, 16) || !aligned(phases, 8) || !aligned(rotary_positions, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    if (q_out == q && (rope->q_out_token_stride != rope->q_token_stride ||
                       rope->q_out_head_stride != rope->q_head_stride))
        return PA_ERR_INVALID_ARG;
    const Rows qo{q_out, out_row, rope->q_out_token_stride}, qi{q, q_row, rope->q_token_stride},
        nw{latent_new, W, rope->new_stride};
    if ((q_out != q && rows_meet(qo, qi, tokens)) || rows_meet(qo, nw, tokens)) return PA_ERR_INVALID_ARG;
    const Span outs[2] = {qo.span(tokens),
                          {cache, (size_t)shape->num_blocks * shape->block_size * W * 2}};
    const Span ins[7] = {{rotary_positions, (size_t)tokens * 4},
                         {phases, (size_t)shape->rope_dim / 2 * 8},
                         {block_tables, (size_t)shape->batch * shape->max_blocks_per_seq * 4},
                         {context_lens, (size_t)shape->batch * 4},
                         {norm_weight, norm_weight ? (size_t)shape->latent_dim * 2 : 0},
                         qi.span(tokens),
                         nw.span(tokens)};
    if (overlap(outs[0], outs[1])) return PA_ERR_INVALID_ARG;
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < (o == 0 ? 5 : 7); ++i)
            if (overlap(outs[o], ins[i])) return PA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_state(&sms, nullptr);
    if (st != PA_OK) return st;
    LatentAppendParams p;
    std::memset(&p, 0, sizeof p);
    p.q_out = q_out;
    p.cache = cache;
    p.q = q;
    p.latent_new = latent_new;
    p.norm_weight = norm_weight;
    p.positions = rotary_positions;
    p.phases = phases;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_blocks = shape->num_blocks;
    p.q_token_stride = rope->q_token_stride;
    p.q_head_stride = rope->q_head_stride;
    p.q_out_token_stride = rope->q_out_token_stride;
    p.q_out_head_stride = rope->q_out_head_stride;
    p.new_stride = rope->new_stride;
    p.eps = rope->eps;
    p.batch = shape->batch;
    p.q_len = q_len;
    p.num_heads = shape->num_heads;
    p.latent_dim = shape->latent_dim;
    p.block_size = shape->block_size;
    p.max_blocks = shape->max_blocks_per_seq;
    p.interleaved = rope->interleaved;
    return done(launch_append_latent(p, shape->dtype == PA_BF16, sms, use_pdl(),
                                     static_cast<cudaStream_t>(stream)));
}

size_t pa_workspace_size_latent(const pa_latent_shape* shape, int32_t q_len, int32_t max_context_len) {
    int sms = 0;
    if (check_latent_call(shape, q_len) != PA_OK || max_context_len < 0 || shape->batch == 0 ||
        device_state(&sms, nullptr) != PA_OK)
        return 0;
    // (of the batches up to this one the largest that takes runs needs most)
    pa_latent_shape most = *shape;
    most.batch = std::min(shape->batch, kMaxBalancedLens);
    return plan_latent(&most, q_len, max_context_len, sms).bytes;
}

pa_status pa_decode_latent(void* out, const void* q, const void* cache,
                           const int32_t* block_tables, const int32_t* context_lens,
                           const pa_latent_shape* shape, int32_t q_len, float scale,
                           int32_t max_context_len, void* workspace, size_t workspace_bytes,
                           void* stream) {
    pa_status st = check_latent_call(shape, q_len);
    if (st != PA_OK) return st;
    if (max_context_len < 0 || !scale_ok(scale)) return PA_ERR_INVALID_ARG;
    if (shape->batch == 0) return PA_OK;
    if (!out || !q || !cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    const size_t rows = (size_t)shape->batch * q_len * shape->num_heads;
    const size_t W = (size_t)shape->latent_dim + shape->rope_dim;
    const Span o{out, rows * shape->latent_dim * 2};
    const Span ins[4] = {{q, rows * W * 2},
                         {cache, (size_t)shape->num_blocks * shape->block_size * W * 2},
                         {block_tables, (size_t)shape->batch * shape->max_blocks_per_seq * 4},
                         {context_lens, (size_t)shape->batch * 4}};
    for (const Span& i : ins)
        if (overlap(o, i)) return PA_ERR_INVALID_ARG;
    int sms = 0;
    int32_t* err = nullptr;
    st = device_state(&sms, &err);
    if (st != PA_OK) return st;
    const LatentPlan pl = plan_latent(shape, q_len, max_context_len, sms);
    if (pl.bytes) {
        if (!workspace || !aligned(workspace, 16) || workspace_bytes < pl.bytes) return PA_ERR_WORKSPACE;
        const Span w{workspace, pl.bytes};
        if (overlap(w, o)) return PA_ERR_INVALID_ARG;
        for (const Span& i : ins)
            if (overlap(w, i)) return PA_ERR_INVALID_ARG;
    }
    LatentLaunch L;
    std::memset(&L, 0, sizeof L);
    const CUtensorMapDataType type = shape->dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // 64 elements (128 bytes) of a page's rows, and of a row tile's queries
    const uint64_t cd[4] = {W, (uint64_t)shape->block_size, (uint64_t)shape->num_blocks, 1};
    const uint64_t cs[3] = {W * 2, W * 2 * shape->block_size, W * 2 * shape->block_size * (uint64_t)shape->num_blocks};
    const uint32_t cb[4] = {64, (uint32_t)shape->block_size, 1, 1};
    st = encode_tiled(&L.tmap_c, type, 4, cache, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != PA_OK) return st;
    const uint64_t qd[2] = {W, rows}, qs[1] = {W * 2};
    const uint32_t qb[2] = {64, (uint32_t)pl.row_tile};
    st = encode_tiled(&L.tmap_q, type, 2, q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != PA_OK) return st;
    LatentParams& p = L.p;
    char* ws = static_cast<char*>(workspace);
    p.out = out;
    p.cache = cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.part_acc = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + pl.ml_at);
    p.part_desc = reinterpret_cast<PieceDesc*>(ws + pl.desc_at);
    p.err = err;
    p.timeout_ns = kDefaultTimeoutNs;
    p.num_blocks = shape->num_blocks;
    p.qscale = scale * 1.4426950408889634f;  // log2(e)
    p.batch = shape->batch;
    p.q_len = q_len;
    p.num_heads = shape->num_heads;
    p.block_size = shape->block_size;
    p.max_blocks = shape->max_blocks_per_seq;
    p.token_limit = announced_tokens(max_context_len, shape->block_size, shape->max_blocks_per_seq);
    p.row_tiles = pl.row_tiles;
    p.group_size = pl.group_size;
    p.row_groups = pl.row_groups;
    p.balanced = pl.bytes ? 1 : 0;
    L.row_tile = pl.row_tile;
    L.ctas = (int)pl.ctas;
    L.sms = sms;
    L.bf16 = shape->dtype == PA_BF16;
    L.pdl = use_pdl();
    L.join = pl.bytes != 0;
    cudaStream_t stm = static_cast<cudaStream_t>(stream);
    return done(shape->latent_dim == 128   ? launch_latent_r128(L, stm)
                : shape->latent_dim == 256 ? launch_latent_r256(L, stm)
                                           : launch_latent_r512(L, stm));
}

}  // extern "C"
