"""Outputs of pa.rope_append_kv that lie over its inputs, and rows of weights that
are too long: refused at the C ABI (CPU: every call is built to fail its checks) and
in the binding; slices of one buffer that do not meet are taken."""
import ctypes

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
from paged_kv_attention_08_gb300 import build as pa_build

# far apart, never dereferenced: 4 sequences of 3 tokens, 8 heads on 2 of 64
Q, K, V, OUT, KC, VC, REST = (i << 32 for i in range(1, 8))
ROW, KV_ROW, TOKENS = 8 * 64, 2 * 64, 12


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    pa._load()
    return pa._lib


def call(lib, q_out, q=Q, k=K, v=V, kc=KC, vc=VC, q_stride=ROW, q_out_stride=ROW, k_stride=KV_ROW,
         v_stride=KV_ROW, batch=4, q_len=3):
    s = pa._Shape(batch, 8, 2, 64, 16, 4, 32, pa.F16, pa.F32)
    r = pa._Rope(64, 1, 0, 0, q_stride, q_out_stride, k_stride, v_stride)
    return lib.pa_rope_append_kv(q_out, kc, vc, q, k, v, REST, REST, REST, REST, REST, ctypes.byref(s),
                                 q_len, ctypes.byref(r), None)


@pytest.mark.parametrize("off", [16, -16, ROW * 2, 2 * ROW * (TOKENS - 1), -2 * ROW * (TOKENS - 1)])
def test_rope_refuses_queries_shifted_over_themselves(lib, off):
    assert call(lib, Q + off) == 1


def test_rope_refuses_queries_over_the_other_inputs(lib):
    fused = ROW + 2 * KV_ROW                      # q, k and v of a token side by side
    for off in (0, 16, 2 * KV_ROW - 16, 2 * KV_ROW * (TOKENS - 1)):
        assert call(lib, K + off) == 1            # another stride, the same range
        assert call(lib, V + off) == 1
    strides = dict(q_stride=fused, k_stride=fused, v_stride=fused)
    k, v = Q + 2 * ROW, Q + 2 * (ROW + KV_ROW)
    for off in (16, 2 * KV_ROW, -16, 2 * (fused - 8)):
        assert call(lib, Q + off, k=k, v=v, q_out_stride=fused, **strides) == 1
    assert call(lib, Q, k=Q + 2 * ROW - 16, v=v, q_out_stride=fused, **strides) == 1
    assert call(lib, Q + 16, batch=1, q_len=1) == 1
    assert call(lib, K - 2 * ROW + 16, batch=1, q_len=1, q_out_stride=8 * ROW) == 1


def test_rope_refuses_queries_in_the_caches(lib):
    cache = 32 * 16 * KV_ROW * 2
    for at in (KC, KC + cache - 16, VC + 4096, VC - 2 * ROW * TOKENS + 16):
        assert call(lib, at) == 1


def test_accumulate_refuses_rows_of_weights_past_30_bits(lib):
    def at(blocks):
        s = pa._Shape(1, 8, 2, 64, 16, blocks, 32, pa.F16, pa.F32)
        return lib.pa_decode_accumulate(Q, K, V, Q, KC, VC, REST, REST, ctypes.byref(s), 1, 0.1, 64, None, 0,
                                        None)

    assert at((1 << 26) + 1) == 2 and at((1 << 27) - 1) == 2


@pytest.mark.gpu
def test_rope_takes_slices_of_one_buffer():
    dev, H, Hkv, D, bs = "cuda:0", 8, 2, 64, 16
    g = torch.Generator().manual_seed(1)
    buf = torch.randn((4, 3, 2 * H + 2 * Hkv, D), generator=g).half().to(dev)
    q, k, v = buf[:, :, :H], buf[:, :, H:H + Hkv], buf[:, :, H + Hkv:H + 2 * Hkv]
    beside = buf[:, :, H + 2 * Hkv:]
    phases = pa.rope_phases(1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).to(dev)
    axes = torch.zeros(32, dtype=torch.int32, device=dev)
    pos = torch.arange(12, dtype=torch.int32, device=dev).view(1, 4, 3)
    table = torch.arange(4, dtype=torch.int32, device=dev).view(4, 1)
    lens = torch.full((4,), 7, dtype=torch.int32, device=dev)

    def turned(q_out):
        kc, vc = (torch.zeros((4, bs, Hkv, D), dtype=torch.half, device=dev) for _ in range(2))
        pa.rope_append_kv(q_out, kc, vc, q, k, v, pos, phases, axes, table, lens)
        torch.cuda.synchronize()
        return q_out.clone(), kc, vc

    want = turned(torch.empty((4, 3, H, D), dtype=torch.half, device=dev))
    for got in (turned(beside), turned(q)):       # (q last: it is turned in place)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(pa.PaError, match="INVALID_ARG"):
        turned(buf[:, :, 1:H + 1])                # one head on
    with pytest.raises(pa.PaError, match="INVALID_ARG"):
        turned(buf[:, :, H:2 * H])                # over k and v
