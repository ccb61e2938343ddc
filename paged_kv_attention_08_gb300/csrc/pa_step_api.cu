// Host side of the entry points around attention in a serving step:
// pa_rope_append_kv (rotary positions and the append) and pa_evict_kv
// (eviction by accumulated weight).
#include <cstring>

#include "pa_internal.h"

using namespace pa;

namespace {

// do [a, a + na) and [b, b + nb) share a byte?
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Do rows of two arrays of `tokens` 16-bit rows share a byte?  Rows of one stride
// meet if they do modulo the stride (slices of one fused buffer do not); arrays
// of different strides are taken to where they share a range.
bool rows_meet(const void* a, int64_t a_row, int64_t a_stride, const void* b, int64_t b_row,
               int64_t b_stride, int64_t tokens) {
    const size_t na = ((size_t)(tokens - 1) * a_stride + a_row) * 2;
    const size_t nb = ((size_t)(tokens - 1) * b_stride + b_row) * 2;
    if (!overlap(a, na, b, nb)) return false;
    if (a_stride != b_stride || tokens == 1) return true;
    const int64_t stride = a_stride * 2;
    const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b));
    const int64_t at = ((apart % stride) + stride) % stride;  // a's rows begin here in b's stride
    return at < b_row * 2 || at + a_row * 2 > stride;
}

}  // namespace

extern "C" {

pa_status pa_rope_append_kv(void* q_out, void* k_cache, void* v_cache, const void* q,
                            const void* k_new, const void* v_new, const int32_t* rotary_positions,
                            const int64_t* phases, const int32_t* axes,
                            const int32_t* block_tables, const int32_t* context_lens,
                            const pa_shape* shape, int32_t q_len, const pa_rope* rope,
                            void* stream) {
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
    if (q_out == q && rope->q_out_stride != rope->q_stride) return PA_ERR_INVALID_ARG;
    if (rope->q_stride % 8 || rope->q_out_stride % 8 || rope->k_stride % 8 || rope->v_stride % 8)
        return PA_ERR_UNSUPPORTED;
    const int64_t tokens = (int64_t)shape->batch * q_len;
    const int64_t per_token =
        (int64_t)(shape->num_heads + 2ll * shape->num_kv_heads) * (shape->head_dim / 16);
    // flattened items of a call, and those of one token, in 31 bits
    if (per_token >= (1 << 28) || (tokens > 0 && tokens > (1ll << 38) / per_token))
        return PA_ERR_UNSUPPORTED;
    if (shape->batch == 0) return PA_OK;
    if (!q_out || !k_cache || !v_cache || !q || !k_new || !v_new || !rotary_positions || !phases ||
        !axes || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q, 16) ||
        !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(phases, 8) ||
        !aligned(rotary_positions, 4) || !aligned(axes, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    // items of q_out are written while others of the inputs are still to be read
    const size_t cache_bytes =
        (size_t)shape->num_blocks * shape->block_size * (size_t)kv_row * 2;
    const size_t out_bytes = ((size_t)(tokens - 1) * rope->q_out_stride + q_row) * 2;
    if ((q_out != q && rows_meet(q_out, q_row, rope->q_out_stride, q, q_row, rope->q_stride, tokens)) ||
        rows_meet(q_out, q_row, rope->q_out_stride, k_new, kv_row, rope->k_stride, tokens) ||
        rows_meet(q_out, q_row, rope->q_out_stride, v_new, kv_row, rope->v_stride, tokens) ||
        overlap(q_out, out_bytes, k_cache, cache_bytes) ||
        overlap(q_out, out_bytes, v_cache, cache_bytes))
        return PA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_state(&sms, nullptr);
    if (st != PA_OK) return st;
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
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
    return launch_rope_append(p, shape->kv_dtype == PA_BF16, sms, use_pdl(),
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_evict_kv(void* k_cache, void* v_cache, const float* weights,
                      const int32_t* block_tables, const int32_t* context_lens,
                      const int32_t* new_block_tables, float* new_weights, int32_t* new_lens,
                      int32_t* kept, const pa_shape* shape, int32_t new_max_blocks_per_seq,
                      int32_t budget, int32_t sink, int32_t recent, void* stream) {
    pa_status st = check_shape(shape);
    if (st != PA_OK) return st;
    if (new_max_blocks_per_seq < 1 || budget < 1 || sink < 0 || recent < 0 ||
        (int64_t)sink + recent > budget)
        return PA_ERR_INVALID_ARG;
    const int64_t new_width = (int64_t)new_max_blocks_per_seq * shape->block_size;
    if (budget > new_width) return PA_ERR_INVALID_ARG;
    // token indexes and the loops over them stay inside 31 bits
    if ((int64_t)shape->max_blocks_per_seq * shape->block_size > (1 << 30) || new_width > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (shape->batch == 0) return PA_OK;
    if (!k_cache || !v_cache || !weights || !block_tables || !context_lens || !new_block_tables ||
        !new_weights || !new_lens || !kept)
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(new_block_tables, 4) ||
        !aligned(new_weights, 4) || !aligned(new_lens, 4) || !aligned(kept, 4))
        return PA_ERR_INVALID_ARG;
    // the same tensors in place, or others: nothing that overlaps in part
    const size_t units = (size_t)shape->batch * shape->num_kv_heads;
    const size_t width = (size_t)shape->max_blocks_per_seq * shape->block_size;
    const bool same_table = block_tables == new_block_tables;
    const bool same_weights = weights == new_weights;
    if ((same_table || same_weights) && new_max_blocks_per_seq != shape->max_blocks_per_seq)
        return PA_ERR_INVALID_ARG;
    const size_t w_bytes = units * width * 4, nw_bytes = units * (size_t)new_width * 4;
    const size_t t_bytes = (size_t)shape->batch * shape->max_blocks_per_seq * 4;
    const size_t l_bytes = (size_t)shape->batch * 4, k_bytes = units * (size_t)budget * 4;
    if (!same_weights && overlap(weights, w_bytes, new_weights, nw_bytes)) return PA_ERR_INVALID_ARG;
    // the outputs lie apart from each other and from every input
    const size_t nt_bytes = (size_t)shape->batch * new_max_blocks_per_seq * 4;
    const struct {
        const void* p;
        size_t n;
    } outs[3] = {{kept, k_bytes}, {new_lens, l_bytes}, {new_weights, nw_bytes}},
      ins[4] = {{block_tables, t_bytes},
                {context_lens, l_bytes},
                {new_block_tables, nt_bytes},
                {weights, w_bytes}};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if (!(o == 2 && i == 3) && overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
                return PA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlap(outs[o].p, outs[o].n, outs[i].p, outs[i].n)) return PA_ERR_INVALID_ARG;
    }
    st = device_state(nullptr, nullptr);
    if (st != PA_OK) return st;
    EvictParams p;
    std::memset(&p, 0, sizeof p);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.weights = weights;
    p.new_weights = new_weights;
    p.block_tables = block_tables;
    p.new_block_tables = new_block_tables;
    p.context_lens = context_lens;
    p.new_lens = new_lens;
    p.kept = kept;
    p.num_blocks = shape->num_blocks;
    p.batch = shape->batch;
    p.num_kv_heads = shape->num_kv_heads;
    p.head_dim = shape->head_dim;
    p.block_size = shape->block_size;
    p.max_blocks = shape->max_blocks_per_seq;
    p.new_max_blocks = new_max_blocks_per_seq;
    p.budget = budget;
    p.sink = sink;
    p.recent = recent;
    return launch_evict(p, same_table || same_weights, use_pdl(),
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // extern "C"
