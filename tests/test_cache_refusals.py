"""CPU tests of what the operators on the 8-bit and the latent cache refuse, at
the C ABI and in the binding: every call here is built to fail its checks (or to
hold an empty batch), so none reaches a launch."""
import ctypes
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
from paged_kv_attention_08_gb300 import build as pa_build

FAR = 1 << 40
STEP = 1 << 36   # apart from everything


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


def latent(**kw):
    base = dict(batch=4, num_heads=16, latent_dim=512, rope_dim=64, block_size=64,
                max_blocks_per_seq=32, num_blocks=512, dtype=pa.BF16, reserved=0)
    base.update(kw)
    return pa._LatentShape(**base)


def latent_rope(**kw):
    base = dict(interleaved=0, eps=1e-6, q_token_stride=16 * 192, q_head_stride=192,
                q_out_token_stride=16 * 576, q_out_head_stride=576, new_stride=576)
    base.update(kw)
    return pa._LatentRope(**base)


def pointers(n, ptrs):
    p = [FAR + i * STEP for i in range(n)]
    for i, v in (ptrs or {}).items():
        p[i] = v
    return p


def append8(lib, s, r, ptrs=None, q_len=1):
    return lib.pa_rope_append_kv8(*pointers(13, ptrs), ctypes.byref(s), q_len,
                                  ctypes.byref(r) if r else None, None)


def kv8(lib, s, ptrs=None, q_len=1, scale=0.1, longest=100):
    return lib.pa_decode_kv8(*pointers(8, ptrs), ctypes.byref(s), q_len, scale, longest,
                             FAR + 20 * STEP, 1 << 40, None)


def append_latent(lib, s, r, ptrs=None, q_len=1):
    return lib.pa_rope_append_latent(*pointers(9, ptrs), ctypes.byref(s), q_len,
                                     ctypes.byref(r) if r else None, None)


def decode_latent(lib, s, ptrs=None, q_len=1, scale=0.1, longest=100):
    return lib.pa_decode_latent(*pointers(5, ptrs), ctypes.byref(s), q_len, scale, longest,
                                FAR + 20 * STEP, 1 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rotary_dim=0), 2), (dict(rotary_dim=24), 2), (dict(rotary_dim=144), 1),
    (dict(num_axes=0), 1), (dict(interleaved=2), 1), (dict(q_stride=4088), 1),
    (dict(q_stride=4100), 2), (dict(k_stride=1016), 1), (dict(v_stride=1028), 2),
    (dict(q_out_stride=0), 1)])
def test_append8_refuses_embeddings(lib, kw, code):
    assert append8(lib, shape(), rope(**kw)) == code


def test_append8_refuses_the_rest(lib):
    s, r = shape(), rope()
    assert append8(lib, s, r, q_len=0) == 1
    assert append8(lib, s, None) == 1
    for i in range(13):
        assert append8(lib, s, r, {i: None}) == 1
        odd = 8 if i in (0, 1, 2, 5, 6, 7) else 4 if i == 9 else 2
        assert append8(lib, s, r, {i: FAR + i * STEP + odd}) == 1
        # every output apart from everything else (q_out may be q)
        for o in range(5):
            if i != o and (o, i) != (0, 5):
                assert append8(lib, s, r, {i: FAR + o * STEP}) == 1, (o, i)
    assert append8(lib, s, rope(q_out_stride=8192), {0: FAR + 5 * STEP}) == 1
    assert append8(lib, shape(head_dim=96), r) == 2
    assert append8(lib, shape(block_size=64), r) == 2
    assert append8(lib, shape(batch=65535), r, q_len=1 << 30) == 2
    assert append8(lib, shape(batch=0), r, {i: None for i in range(13)}) == 0


def test_kv8_refuses(lib):
    s = shape()
    for i in range(8):
        assert kv8(lib, s, {i: None}) == 1
        assert kv8(lib, s, {i: FAR + i * STEP + (8 if i < 4 else 2)}) == 1
        if i:
            assert kv8(lib, s, {i: FAR}) == 1           # out on an input
    assert kv8(lib, s, q_len=0) == 1
    assert kv8(lib, s, longest=-1) == 1
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert kv8(lib, s, scale=scale) == 1
    assert kv8(lib, shape(num_heads=24)) == 2            # a group of three
    assert kv8(lib, shape(head_dim=96)) == 2
    assert kv8(lib, shape(block_size=8)) == 2
    assert kv8(lib, shape(kv_dtype=pa.F32)) == 2
    assert kv8(lib, shape(out_dtype=pa.BF16)) == 2
    assert kv8(lib, s, q_len=1 << 30) == 2
    assert kv8(lib, shape(max_blocks_per_seq=(1 << 26) + 1)) == 2
    assert kv8(lib, shape(batch=0), {i: None for i in range(8)}) == 0
    assert lib.pa_workspace_size_kv8(ctypes.byref(shape(head_dim=96)), 1, 100) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(interleaved=2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(q_head_stride=56), 1), (dict(q_head_stride=196, q_token_stride=16 * 200), 2),
    (dict(q_token_stride=15 * 192 + 56), 1), (dict(q_out_token_stride=15 * 576 + 56), 1),
    (dict(q_out_head_stride=0), 1), (dict(new_stride=568), 1), (dict(new_stride=580), 2),
    (dict(q_token_stride=16 * 192 + 4), 2), (dict(q_head_stride=1 << 31, q_token_stride=1 << 40), 1)])
def test_append_latent_refuses_strides(lib, kw, code):
    assert append_latent(lib, latent(), latent_rope(**kw)) == code


def test_append_latent_refuses_the_rest(lib):
    s, r = latent(), latent_rope()
    assert append_latent(lib, s, r, q_len=0) == 1
    assert append_latent(lib, s, None) == 1
    for i in range(9):
        if i != 4:
            assert append_latent(lib, s, r, {i: None}) == 1
        odd = 8 if i in (0, 1, 2, 3, 4) else 4 if i == 6 else 2
        assert append_latent(lib, s, r, {i: FAR + i * STEP + odd}) == 1
        for o in range(2):
            if i != o and (o, i) != (0, 2):
                assert append_latent(lib, s, r, {i: FAR + o * STEP}) == 1, (o, i)
    assert append_latent(lib, s, r, {0: FAR + 2 * STEP}) == 1    # q with another stride
    for kw in (dict(latent_dim=384), dict(rope_dim=32), dict(block_size=8), dict(dtype=pa.F32),
               dict(num_heads=65536), dict(batch=65536), dict(num_blocks=1 << 31),
               dict(max_blocks_per_seq=(1 << 24) + 1)):
        assert append_latent(lib, latent(**kw), latent_rope(q_token_stride=1 << 30,
                                                            q_out_token_stride=1 << 30)) == 2, kw
    assert append_latent(lib, latent(batch=0), r, {i: None for i in range(9)}) == 0


def test_decode_latent_refuses(lib):
    s = latent()
    for i in range(5):
        assert decode_latent(lib, s, {i: None}) == 1
        assert decode_latent(lib, s, {i: FAR + i * STEP + (8 if i < 3 else 2)}) == 1
        if i:
            assert decode_latent(lib, s, {i: FAR}) == 1  # out on an input
    assert decode_latent(lib, s, q_len=0) == 1
    assert decode_latent(lib, s, longest=-1) == 1
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert decode_latent(lib, s, scale=scale) == 1
    for kw in (dict(latent_dim=64), dict(rope_dim=128), dict(block_size=128), dict(dtype=pa.F32),
               dict(max_blocks_per_seq=(1 << 24) + 1)):
        assert decode_latent(lib, latent(**kw)) == 2, kw
    assert decode_latent(lib, s, q_len=1 << 30) == 2
    assert decode_latent(lib, latent(num_heads=0)) == 1
    assert decode_latent(lib, latent(batch=0), {i: None for i in range(5)}) == 0
    assert lib.pa_workspace_size_latent(ctypes.byref(latent(latent_dim=64)), 1, 100) == 0


# ---- the binding ----

def kv8_tensors(**kw):
    t = dict(out=torch.zeros(2, 4, 64, dtype=torch.float16), q=torch.zeros(2, 4, 64, dtype=torch.float16),
             k_cache=torch.zeros(4, 16, 2, 64).to(torch.float8_e4m3fn),
             v_cache=torch.zeros(4, 16, 2, 64).to(torch.float8_e4m3fn),
             k_scales=torch.ones(4, 2), v_scales=torch.ones(4, 2),
             block_tables=torch.zeros(2, 2, dtype=torch.int32),
             context_lens=torch.zeros(2, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,error", [
    (dict(out=torch.zeros(2, 4, 128, dtype=torch.float16)), ValueError),
    (dict(out=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), TypeError),
    (dict(q=torch.zeros(2, 4, 128, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 4, 64)), TypeError),
    (dict(k_cache=torch.zeros(4, 16, 2, 64, dtype=torch.float16)), TypeError),
    (dict(v_cache=torch.zeros(4, 16, 2, 32).to(torch.float8_e4m3fn)), ValueError),
    (dict(v_cache=torch.zeros(4, 16, 2, 64).to(torch.float8_e5m2)), TypeError),
    (dict(k_scales=torch.ones(4, 2, 1)), ValueError),
    (dict(v_scales=torch.ones(3, 2)), ValueError),
    (dict(v_scales=torch.ones(4, 2, dtype=torch.float64)), TypeError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int32)), ValueError),
    (dict(block_tables=torch.zeros(2, 2, dtype=torch.int64)), TypeError),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(max_context_len=1 << 31), ValueError),
    ({}, ValueError),                                    # CPU tensors
])
def test_binding_refuses_kv8(kw, error):
    args = dict(kv8_tensors(), scale=0.1, max_context_len=10)
    args.update(kw)
    with pytest.raises(error):
        pa.decode_kv8(**args)


def append8_tensors(**kw):
    B, Q, H, Hkv, D = 2, 3, 4, 2, 64
    t = dict(q_out=torch.zeros(B, Q, H, D, dtype=torch.float16),
             k_cache=torch.zeros(4, 16, Hkv, D).to(torch.float8_e4m3fn),
             v_cache=torch.zeros(4, 16, Hkv, D).to(torch.float8_e4m3fn),
             k_scales=torch.ones(4, Hkv), v_scales=torch.ones(4, Hkv),
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
    (dict(k_cache=torch.zeros(4, 16, 2, 64, dtype=torch.float16)), TypeError),
    (dict(k_scales=torch.ones(4, 3)), ValueError),
    (dict(v_scales=torch.ones(4, 2, dtype=torch.float16)), TypeError),
    (dict(k_new=torch.zeros(2, 3, 3, 64, dtype=torch.float16)), ValueError),
    (dict(v_new=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)), TypeError),
    (dict(v_new=torch.zeros(2, 3, 64, 2, dtype=torch.float16).transpose(2, 3)), ValueError),
    (dict(rotary_positions=torch.zeros(3, 2, 2, dtype=torch.int32)), ValueError),
    (dict(rotary_positions=torch.zeros(3, 2, 3)), TypeError),
    (dict(phases=torch.zeros(32)), TypeError),
    (dict(axes=torch.zeros(31, dtype=torch.int32)), ValueError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(2)), TypeError),
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 0, 4, 64, dtype=torch.float16)), ValueError),
    ({}, ValueError),
])
def test_binding_refuses_append8(kw, error):
    with pytest.raises(error):
        pa.rope_append_kv8(**append8_tensors(**kw))


def append_latent_tensors(**kw):
    B, Q, H, R = 2, 3, 4, 128
    t = dict(q_out=torch.zeros(B, Q, H, 64, dtype=torch.float16),
             cache=torch.zeros(4, 16, R + 64, dtype=torch.float16),
             q=torch.zeros(B, Q, H, 64, dtype=torch.float16),
             latent_new=torch.zeros(B, Q, R + 64, dtype=torch.float16),
             norm_weight=torch.ones(R, dtype=torch.float16),
             rotary_positions=torch.zeros(B, Q, dtype=torch.int32),
             phases=torch.zeros(32, dtype=torch.int64),
             block_tables=torch.zeros(B, 2, dtype=torch.int32),
             context_lens=torch.zeros(B, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,error", [
    (dict(q_out=torch.zeros(2, 3, 4, 32, dtype=torch.float16)), ValueError),
    (dict(q_out=torch.zeros(2, 3, 4, 64)), TypeError),
    (dict(cache=torch.zeros(4, 16, 192)), TypeError),
    (dict(cache=torch.zeros(4, 16, 1, 192, dtype=torch.float16)), ValueError),
    (dict(latent_new=torch.zeros(2, 3, 191, dtype=torch.float16)), ValueError),
    (dict(latent_new=torch.zeros(2, 192, dtype=torch.float16)), ValueError),
    (dict(latent_new=torch.zeros(3, 2, 192, dtype=torch.float16).transpose(0, 1)), ValueError),
    (dict(norm_weight=torch.ones(127, dtype=torch.float16)), ValueError),
    (dict(norm_weight=torch.ones(128)), TypeError),
    (dict(rotary_positions=torch.zeros(1, 2, 3, dtype=torch.int32)), ValueError),
    (dict(rotary_positions=torch.zeros(2, 3)), TypeError),
    (dict(phases=torch.zeros(31, dtype=torch.int64)), ValueError),
    (dict(q=torch.zeros(2, 3, 64, 4, dtype=torch.float16).transpose(2, 3)), ValueError),
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16)), ValueError),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    ({}, ValueError),
])
def test_binding_refuses_append_latent(kw, error):
    with pytest.raises(error):
        pa.rope_append_latent(**append_latent_tensors(**kw))


@pytest.mark.parametrize("kw,error", [
    (dict(out=torch.zeros(2, 5, 128, dtype=torch.float16)), ValueError),
    (dict(out=torch.zeros(2, 4, 128)), TypeError),
    (dict(out=torch.zeros(2, 4, 192, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 4, 200, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(2, 4, 192, dtype=torch.bfloat16)), TypeError),
    (dict(cache=torch.zeros(4, 16, 1, 192, dtype=torch.float16)), ValueError),
    (dict(block_tables=torch.zeros(2, 2)), TypeError),
    (dict(context_lens=torch.zeros(1, dtype=torch.int32)), ValueError),
    (dict(max_context_len=-(1 << 31) - 1), ValueError),
    ({}, ValueError),
])
def test_binding_refuses_decode_latent(kw, error):
    args = dict(out=torch.zeros(2, 4, 128, dtype=torch.float16),
                q=torch.zeros(2, 4, 192, dtype=torch.float16),
                cache=torch.zeros(4, 16, 192, dtype=torch.float16),
                block_tables=torch.zeros(2, 2, dtype=torch.int32),
                context_lens=torch.zeros(2, dtype=torch.int32), scale=0.1, max_context_len=10)
    args.update(kw)
    with pytest.raises(error):
        pa.decode_latent(**args)
