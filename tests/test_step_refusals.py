"""CPU tests of what the serving-step operators refuse, at the C ABI and in the
binding: every call here is built to fail its checks, so none reaches a launch."""
import ctypes

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
from paged_kv_attention_08_gb300 import build as pa_build

FAKE = 0x10000  # 16-byte aligned, never dereferenced
FAR = 1 << 40   # apart from everything


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    pa._load()
    return pa._lib


def shape(**kw):
    base = dict(batch=4, num_heads=32, num_kv_heads=8, head_dim=128, block_size=16,
                max_blocks_per_seq=128, num_blocks=512, kv_dtype=pa.F16, out_dtype=pa.F32)
    base.update(kw)
    return pa._Shape(**base)


def rope(**kw):
    base = dict(rotary_dim=128, num_axes=3, interleaved=0, reserved=0, q_stride=4096,
                q_out_stride=4096, k_stride=1024, v_stride=1024)
    base.update(kw)
    return pa._Rope(**base)


def call_rope(lib, s, r, ptrs=None, q_len=1):
    p = [FAKE] * 11
    p[0] = FAR
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.pa_rope_append_kv(*p, ctypes.byref(s), q_len, ctypes.byref(r) if r else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rotary_dim=0), 2), (dict(rotary_dim=24), 2), (dict(rotary_dim=144), 1),
    (dict(rotary_dim=-16), 1), (dict(num_axes=0), 1), (dict(interleaved=2), 1),
    (dict(q_stride=4088), 1), (dict(q_stride=4100), 2), (dict(k_stride=1016), 1),
    (dict(v_stride=1028), 2), (dict(q_out_stride=0), 1),
])
def test_rope_refuses_embeddings(lib, kw, code):
    assert call_rope(lib, shape(), rope(**kw)) == code


def test_rope_refuses_the_rest(lib):
    s, r = shape(), rope()
    assert call_rope(lib, s, r, q_len=0) == 1
    assert call_rope(lib, s, None) == 1
    for i in range(11):
        assert call_rope(lib, s, r, {i: None}) == 1
        odd = 8 if i in (0, 1, 2, 3, 4, 5) else (4 if i == 7 else 2)
        assert call_rope(lib, s, r, {i: FAR + odd}) == 1
    # q_out on q itself needs q's stride
    assert call_rope(lib, s, rope(q_out_stride=8192), {0: FAKE}) == 1
    assert call_rope(lib, shape(head_dim=96), r) == 2
    assert call_rope(lib, shape(batch=65535, max_blocks_per_seq=1), rope(), q_len=1 << 30) == 2
    assert call_rope(lib, shape(batch=0), r, {i: None for i in range(11)}) == 0


def call_evict(lib, s, ptrs=None, new_mb=64, budget=1024, sink=4, recent=16):
    p = [FAKE << (2 * i) for i in range(9)]
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.pa_evict_kv(*p, ctypes.byref(s), new_mb, budget, sink, recent, None)


@pytest.mark.parametrize("kw", [dict(budget=0), dict(sink=-1), dict(recent=-1), dict(new_mb=0),
                                dict(sink=1000, recent=25), dict(new_mb=63),
                                dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1)])
def test_evict_refuses_budgets(lib, kw):
    assert call_evict(lib, shape(), **kw) == 1


def test_evict_refuses_the_rest(lib):
    s = shape()
    for i in range(9):
        assert call_evict(lib, s, {i: None}) == 1
        assert call_evict(lib, s, {i: FAR + 2}) == 1
    same_table = {3: FAR, 5: FAR}
    assert call_evict(lib, s, same_table, new_mb=100) == 1   # in place with another width
    w_bytes = 4 * 8 * 128 * 16 * 4
    assert call_evict(lib, s, {2: FAR, 6: FAR + 64}) == 1     # overlapping weights
    assert call_evict(lib, s, {2: FAR, 8: FAR + w_bytes - 4}) == 1   # kept inside the weights
    assert call_evict(lib, s, {4: FAR, 7: FAR}) == 1          # new_lens on context_lens
    assert call_evict(lib, shape(max_blocks_per_seq=(1 << 26) + 1)) == 2
    assert call_evict(lib, shape(block_size=8)) == 2
    assert call_evict(lib, shape(batch=0), {i: None for i in range(9)}) == 0


@pytest.mark.parametrize("out,size", [(6, 4 * 8 * 64 * 16 * 4), (7, 4 * 4), (8, 4 * 8 * 1024 * 4)])
@pytest.mark.parametrize("other,length", [(3, 4 * 128 * 4), (4, 4 * 4), (5, 4 * 64 * 4), (6, 4 * 8 * 64 * 16 * 4),
                                          (7, 4 * 4), (8, 4 * 8 * 1024 * 4)])
def test_evict_refuses_outputs_that_overlap(lib, out, size, other, length):
    if out == other:
        return
    far = 1 << 40
    assert call_evict(lib, shape(), {out: far, other: far + size - 4}) == 1
    assert call_evict(lib, shape(), {out: far + length - 4, other: far}) == 1


def rope_args(**kw):
    B, Q, H, Hkv, D = 2, 3, 4, 2, 64
    t = dict(q_out=torch.zeros(B, Q, H, D, dtype=torch.float16),
             k_cache=torch.zeros(4, 16, Hkv, D, dtype=torch.float16),
             v_cache=torch.zeros(4, 16, Hkv, D, dtype=torch.float16),
             q=torch.zeros(B, Q, H, D, dtype=torch.float16),
             k_new=torch.zeros(B, Q, Hkv, D, dtype=torch.float16),
             v_new=torch.zeros(B, Q, Hkv, D, dtype=torch.float16),
             rotary_positions=torch.zeros(3, B, Q, dtype=torch.int32),
             phases=torch.zeros(32, dtype=torch.int64), axes=torch.zeros(32, dtype=torch.int32),
             block_tables=torch.zeros(B, 2, dtype=torch.int32),
             context_lens=torch.zeros(B, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,error", [
    (dict(q_out=torch.zeros(2, 3, 4, 128, dtype=torch.float16)), ValueError),
    (dict(q_out=torch.zeros(2, 3, 4, 64)), TypeError),
    (dict(v_cache=torch.zeros(4, 16, 2, 128, dtype=torch.float16)), ValueError),
    (dict(k_new=torch.zeros(2, 3, 3, 64, dtype=torch.float16)), ValueError),
    (dict(v_new=torch.zeros(2, 2, 3, 64, dtype=torch.float16).transpose(1, 2)), ValueError),
    (dict(k_new=torch.zeros(2, 5, 2, 64, dtype=torch.float16)[:, :3]), ValueError),
    (dict(q=torch.zeros(2, 3, 4, 128, dtype=torch.float16)[..., ::2]), ValueError),
    (dict(rotary_positions=torch.zeros(3, 2, 4, dtype=torch.int32)), ValueError),
    (dict(rotary_positions=torch.zeros(3, 2, 3)), TypeError),
    (dict(phases=torch.zeros(32)), TypeError),
    (dict(axes=torch.zeros(31, dtype=torch.int32)), ValueError),
    (dict(axes=torch.zeros(32, dtype=torch.int64)), TypeError),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16)), ValueError),
    (dict(), ValueError),   # not on a GPU
])
def test_binding_refuses_rope(kw, error):
    with pytest.raises(error):
        pa.rope_append_kv(**rope_args(**kw))


def test_rope_phases_refuses_and_wraps():
    with pytest.raises(TypeError):
        pa.rope_phases(torch.zeros(4))
    with pytest.raises(TypeError):
        pa.rope_phases(torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        pa.rope_phases(torch.tensor([1.0, float("inf")], dtype=torch.float64))
    import math
    f = torch.tensor([0.0, math.pi / 2, math.pi, 3 * math.pi / 2, -math.pi / 2, 2 * math.pi],
                     dtype=torch.float64)
    got = pa.rope_phases(f).tolist()
    assert got == [0, 1 << 62, -(1 << 63), -(1 << 62), -(1 << 62), 0]


def evict_args(**kw):
    B, Hkv = 2, 2
    t = dict(k_cache=torch.zeros(4, 16, Hkv, 64, dtype=torch.float16),
             v_cache=torch.zeros(4, 16, Hkv, 64, dtype=torch.float16),
             weights=torch.zeros(B, Hkv, 64), block_tables=torch.zeros(B, 4, dtype=torch.int32),
             context_lens=torch.zeros(B, dtype=torch.int32),
             new_block_tables=torch.zeros(B, 2, dtype=torch.int32),
             new_weights=torch.zeros(B, Hkv, 32), new_lens=torch.zeros(B, dtype=torch.int32),
             kept=torch.zeros(B, Hkv, 20, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,error", [
    (dict(v_cache=torch.zeros(4, 16, 2, 64)), TypeError),
    (dict(v_cache=torch.zeros(5, 16, 2, 64, dtype=torch.float16)), ValueError),
    (dict(weights=torch.zeros(2, 2, 63)), ValueError),
    (dict(weights=torch.zeros(2, 2, 64, dtype=torch.float64)), TypeError),
    (dict(new_weights=torch.zeros(2, 2, 64)), ValueError),
    (dict(new_block_tables=torch.zeros(3, 2, dtype=torch.int32)), ValueError),
    (dict(new_block_tables=torch.zeros(2, 2, dtype=torch.int64)), TypeError),
    (dict(new_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(kept=torch.zeros(2, 20, dtype=torch.int32)), ValueError),
    (dict(kept=torch.zeros(2, 2, 20, dtype=torch.int64)), TypeError),
    (dict(), ValueError),   # not on a GPU
])
def test_binding_refuses_evict(kw, error):
    with pytest.raises(error):
        pa.evict_kv(**evict_args(**kw))


def call_prefix(lib, s, ptrs=None, num_prefixes=2, max_prefix_blocks=100, q_len=1, scale=0.1,
                max_prefix_len=100, max_len=100, ws=FAKE, ws_bytes=1 << 20):
    p = [FAKE] * 8
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.pa_decode_shared_prefix(*p, ctypes.byref(s), num_prefixes, max_prefix_blocks, q_len,
                                       scale, max_prefix_len, max_len, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_prefixes=0), 1), (dict(num_prefixes=3), 1), (dict(num_prefixes=-1), 1),
    (dict(max_prefix_blocks=0), 1), (dict(q_len=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(max_prefix_len=-1), 1), (dict(max_len=-1), 1),
    (dict(max_prefix_blocks=1 << 28), 2), (dict(q_len=1 << 27), 2),
])
def test_prefix_refuses_arguments(lib, kw, code):
    assert call_prefix(lib, shape(), **kw) == code


def test_prefix_refuses_the_rest(lib):
    for i in range(8):
        assert call_prefix(lib, shape(), {i: None}) == 1
        assert call_prefix(lib, shape(), {i: FAR + 2}) == 1
    for i in range(4):
        assert call_prefix(lib, shape(), {i: FAR + 8}) == 1
    assert call_prefix(lib, shape(num_heads=24)) == 2
    assert call_prefix(lib, shape(batch=0), {i: None for i in range(8)}, ws=None) == 0
    assert lib.pa_workspace_size_shared_prefix(ctypes.byref(shape()), 3, 100, 1, 100, 100) == 0
    assert lib.pa_workspace_size_shared_prefix(ctypes.byref(shape(batch=0)), 1, 100, 1, 100, 100) == 0


def call_accumulate(lib, s, ptrs=None, q_len=1, scale=0.1, max_len=100, ws=FAKE, ws_bytes=1 << 20):
    p = [FAKE] * 8
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.pa_decode_accumulate(*p, ctypes.byref(s), q_len, scale, max_len, ws, ws_bytes, None)


def test_accumulate_refuses(lib):
    s = shape()
    for kw in (dict(q_len=0), dict(scale=-1.0), dict(scale=float("inf")), dict(max_len=-1)):
        assert call_accumulate(lib, s, **kw) == 1
    assert call_accumulate(lib, s, q_len=1 << 27) == 2
    for i in range(8):
        assert call_accumulate(lib, s, {i: None}) == 1
        assert call_accumulate(lib, s, {i: FAR + 2}) == 1
    # weights that overlap in part
    assert call_accumulate(lib, s, {1: FAR + 16, 2: FAR}) == 1
    assert call_accumulate(lib, shape(kv_dtype=pa.F32)) == 2
    assert call_accumulate(lib, shape(batch=0), {i: None for i in range(8)}, ws=None) == 0
    assert lib.pa_workspace_size_accumulate(ctypes.byref(shape(head_dim=80)), 1, 100) == 0
    assert lib.pa_workspace_size_accumulate(ctypes.byref(s), 0, 100) == 0


def attention_args(**kw):
    B, H, Hkv, D = 4, 4, 2, 64
    t = dict(out=torch.zeros(B, H, D, dtype=torch.float16), q=torch.zeros(B, H, D, dtype=torch.float16),
             k_cache=torch.zeros(4, 16, Hkv, D, dtype=torch.float16),
             v_cache=torch.zeros(4, 16, Hkv, D, dtype=torch.float16),
             block_tables=torch.zeros(B, 2, dtype=torch.int32),
             context_lens=torch.zeros(B, dtype=torch.int32), scale=0.1, max_context_len=32)
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,error", [
    (dict(prefix_tables=torch.zeros(3, 5, dtype=torch.int32), prefix_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(prefix_tables=torch.zeros(0, 5, dtype=torch.int32), prefix_lens=torch.zeros(0, dtype=torch.int32)), ValueError),
    (dict(prefix_tables=torch.zeros(5, dtype=torch.int32)), ValueError),
    (dict(prefix_tables=torch.zeros(2, 5)), TypeError),
    (dict(prefix_lens=torch.zeros(1, dtype=torch.int32)), ValueError),
    (dict(prefix_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(out=torch.zeros(4, 4, 128, dtype=torch.float16)), ValueError),
    (dict(out=torch.zeros(4, 4, 64, dtype=torch.bfloat16)), TypeError),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(), ValueError),   # not on a GPU
])
def test_binding_refuses_prefix(kw, error):
    args = attention_args(prefix_tables=torch.zeros(2, 5, dtype=torch.int32),
                          prefix_lens=torch.zeros(2, dtype=torch.int32), max_prefix_len=50)
    args.update(kw)
    with pytest.raises(error):
        pa.decode_shared_prefix(**args)


@pytest.mark.parametrize("kw,error", [
    (dict(new_weights=torch.zeros(4, 2, 31)), ValueError),
    (dict(new_weights=torch.zeros(4, 4, 32)), ValueError),
    (dict(new_weights=torch.zeros(4, 2, 32, dtype=torch.float16)), TypeError),
    (dict(weights=torch.zeros(4, 2, 16)), ValueError),
    (dict(weights=torch.zeros(4, 2, 32, dtype=torch.float64)), TypeError),
    (dict(q=torch.zeros(4, 4, 64)), TypeError),
    (dict(q=torch.zeros(4, 1, 4, 64, dtype=torch.float16)), ValueError),
    (dict(), ValueError),   # not on a GPU
])
def test_binding_refuses_accumulate(kw, error):
    args = attention_args(new_weights=torch.zeros(4, 2, 32))
    args.update(kw)
    with pytest.raises(error):
        pa.decode_accumulate(**args)
