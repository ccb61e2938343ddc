"""The serving-step operators on pages whose element offsets pass 2^31 (a cache
of 4.6 GB for each of keys and values): the same bits as on a small cache."""
import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BIG = 140000   # blocks of 16 x 8 x 128 elements: 2.29e9 elements


@pytest.fixture(scope="module")
def caches():
    return [torch.empty((BIG, 16, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]


def both(caches, small_k, small_v):
    """The small caches' blocks as the last blocks of the big ones; the offset of their numbers."""
    first = BIG - len(small_k)
    assert first * 16 * 8 * 128 > 2 ** 31
    for big, small in zip(caches, (small_k, small_v)):
        big[first:] = small
    return first


def test_all_operators(caches):
    B, H, Hkv, D, bs, budget = 3, 32, 8, 128, 16, 48
    lens = [100, 37, 64]
    table, n1 = ref.tables(lens, bs, 1, width=8)
    new_table, n2 = ref.tables([budget] * B, bs, 2, first=n1)
    ptable, pool = ref.tables([70], bs, 3, first=n2)
    k = ref.normal((pool, bs, Hkv, D), torch.bfloat16, 4).to(DEV)
    v = ref.normal((pool, bs, Hkv, D), torch.bfloat16, 5).to(DEV)
    first = both(caches, k, v)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    plens = torch.tensor([70], dtype=torch.int32, device=DEV)
    phases = pa.rope_phases(1e4 ** (-torch.arange(64).double() / 64)).to(DEV)
    axes = torch.zeros(64, dtype=torch.int32, device=DEV)
    qkv = ref.normal((B, 1, H + 2 * Hkv, D), torch.bfloat16, 6).to(DEV)
    pos = (lens_d - 1).view(1, B, 1).contiguous()
    w0 = torch.rand((B, Hkv, table.shape[1] * bs), generator=torch.Generator().manual_seed(7)).to(DEV)
    results = []
    for kc, vc, shift in ((k, v, 0), (caches[0], caches[1], first)):
        def t(x):
            return torch.where(x >= 0, x + shift, x).to(torch.int32).to(DEV)
        q = torch.empty((B, 1, H, D), dtype=torch.bfloat16, device=DEV)
        pa.rope_append_kv(q, kc, vc, qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:], pos, phases,
                          axes, t(table), lens_d)
        out, many, pre = (torch.empty_like(q) for _ in range(3))
        w = w0.clone()
        pa.decode_accumulate(out, w, q, kc, vc, t(table), lens_d, 0.09, 100)
        q5 = q.expand(B, 9, H, D).contiguous()
        many = torch.empty_like(q5)
        pa.decode_accumulate(many, w, q5, kc, vc, t(table), lens_d, 0.09, 100)   # the tile kernels
        pa.decode_shared_prefix(pre, q, kc, vc, t(ptable), plens, t(table), lens_d, 0.09, 70, 100)
        kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device=DEV)
        new_lens = torch.empty((B,), dtype=torch.int32, device=DEV)
        new_w = torch.empty((B, Hkv, new_table.shape[1] * bs), device=DEV)
        pa.evict_kv(kc, vc, w, t(table), lens_d, t(new_table), new_w, new_lens, kept, sink=1, recent=5)
        in_place_w = w.clone()
        pa.evict_kv(kc, vc, in_place_w, (tt := t(table)), lens_d, tt, in_place_w, new_lens, kept, 1, 5)
        torch.cuda.synchronize()
        tail = slice(shift, shift + pool) if shift else slice(0, pool)
        results.append([x.clone() for x in (q, out, many, pre, w, kept, new_lens, new_w, in_place_w,
                                            kc[tail], vc[tail])])
    for small, big in zip(*results):
        assert torch.equal(small, big)
    assert pa.device_error() == 0
