"""Numbers that the serving-step entry points of the binding take: those that
do not fit in the C ABI's 32 bits are refused instead of wrapping (CPU: the
refusal comes before the check that the tensors are on a GPU), and numpy's and a
tensor's are taken as the decode calls take them (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_08_gb300 as pa

B, H, Hkv, D, bs, mb = 2, 8, 2, 64, 16, 4


def tensors(dev):
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn((16, bs, Hkv, D), generator=g).half().to(dev) for _ in range(2))
    return dict(q=torch.randn((B, H, D), generator=g).half().to(dev), k_cache=kc, v_cache=vc,
                block_tables=torch.arange(B * mb, dtype=torch.int32).view(B, mb).to(dev),
                context_lens=torch.tensor([40, 7], dtype=torch.int32, device=dev))


def calls(t, one, scale, zero):
    """Every entry point with `one` for its announced lengths."""
    dev = t["q"].device
    prefix = torch.tensor([[9, 10]], dtype=torch.int32, device=dev)
    plens = torch.tensor([20], dtype=torch.int32, device=dev)
    w = torch.zeros((B, Hkv, mb * bs), device=dev)
    out = torch.zeros_like(t["q"])
    attn = (out, t["q"], t["k_cache"], t["v_cache"])
    lens = (t["block_tables"], t["context_lens"])
    new_lens = torch.zeros((B,), dtype=torch.int32, device=dev)
    kept = torch.zeros((B, Hkv, 20), dtype=torch.int32, device=dev)
    return [
        lambda: pa.decode_shared_prefix(*attn, prefix, plens, *lens, scale, one, one),
        lambda: pa.decode_accumulate(out, w, *attn[1:], *lens, scale, one).clone(),
        lambda: (pa.evict_kv(t["k_cache"].clone(), t["v_cache"].clone(), w, *lens, lens[0], w.clone(),
                             new_lens, kept, sink=zero, recent=zero), kept.clone())[1],
    ]


@pytest.mark.parametrize("big", [1 << 31, 1 << 32, (1 << 40) + 64, -(1 << 31) - 1])
def test_numbers_past_32_bits_are_refused(big):
    t = tensors("cpu")
    for call in calls(t, big, 0.1, big):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.gpu
def test_numbers_of_every_kind():
    t = tensors("cuda:0")
    want = [call().clone() for call in calls(t, 64, 0.125, 3)]
    kinds = [(np.int64(64), np.float32(0.125), np.int32(3)),
             (torch.tensor(64), torch.tensor(0.125), torch.tensor(3)),
             (t["context_lens"].max() + 24, np.float64(0.125), np.int64(3))]
    for one, scale, three in kinds:
        for call, w in zip(calls(t, one, scale, three), want):
            assert torch.equal(call(), w)
    q, kc, bt = t["q"], t["k_cache"], t["block_tables"]
    assert pa.workspace_size_accumulate(q, kc, bt, q.dtype, np.int64(64)) == \
        pa.workspace_size_accumulate(q, kc, bt, q.dtype, 64)
    with pytest.raises(ValueError, match="32 bits"):
        pa.workspace_size_accumulate(q, kc, bt, q.dtype, 1 << 32)
    assert pa.device_error() == 0
