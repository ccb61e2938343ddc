"""The serving-step operators together, as a loop over one cache uses them,
against the 64-bit definitions: prompt and steps through rope_append_kv and
decode_accumulate, an eviction in place, more steps on what is left; and samples
that share a prompt through decode_shared_prefix.  After each call the
reference goes on from the GPU's own state (the cache, the weights), so that
each comparison covers one call and keeps that call's bound."""
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rotary(D, naxes):
    half = D // 2
    inv_freq = 1e4 ** (-torch.arange(half).double() * 2 / D)
    axes = (torch.arange(half) % naxes).to(torch.int32)
    return inv_freq, axes, pa.rope_phases(inv_freq.to(DEV)), axes.to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_steps_eviction_and_more_steps(dtype):
    B, H, Hkv, D, bs, naxes, budget = 2, 8, 2, 64, 16, 3, 24
    scale, mb = 1 / math.sqrt(D), 8
    inv_freq, axes, phases, axes_d = rotary(D, naxes)
    g = torch.Generator().manual_seed(0)
    table = torch.randperm(B * mb + 3, generator=g)[:B * mb].reshape(B, mb).to(torch.int32)
    # unwritten slots hold NaN: nothing may read them
    kc = torch.full((B * mb + 3, bs, Hkv, D), float("nan"), dtype=dtype, device=DEV)
    vc = kc.clone()
    weights = torch.zeros((B, Hkv, mb * bs), device=DEV)
    lens = torch.tensor([45, 33], dtype=torch.int32)          # after the prompt
    positions = lens.clone()                                   # of the next token, never evicted
    table_d = table.to(DEV)

    def step(Q, lens, pos, seed):
        """Q new tokens of each sequence: append, attend, accumulate; all checked."""
        qkv = ref.normal((B, Q, H + 2 * Hkv, D), dtype, seed).to(DEV)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        before_k, before_v, before_w = kc.cpu(), vc.cpu(), weights.cpu()
        q_out = torch.empty((B, Q, H, D), dtype=dtype, device=DEV)
        lens_d = lens.to(DEV)
        pa.rope_append_kv(q_out, kc, vc, q, k, v, pos.to(DEV), phases, axes_d, table_d, lens_d)
        out = torch.empty_like(q_out)
        pa.decode_accumulate(out, weights, q_out, kc, vc, table_d, lens_d, scale, mb * bs)
        want_q, want_k, want_v = ref.rope_append(q.cpu(), before_k, before_v, k.cpu(), v.cpu(), pos,
                                                 inv_freq, axes, table, lens, False)
        half = torch.finfo(dtype).eps / 2
        big = 2 * max(q.abs().max().item(), k.abs().max().item())
        slack = big * (5 * 2.0 ** -23 + math.pi * 2.0 ** -24) + 2.0 ** -25  # as in the append's tests
        for got, want in ((q_out.cpu(), want_q), (kc.cpu(), want_k)):
            assert torch.equal(got.isnan(), want.isnan())
            err = (got.double() - want).abs() - half * want.abs() - slack
            assert torch.nan_to_num(err, -1.0).max() <= 0
        assert torch.equal(torch.nan_to_num(vc.cpu().double(), 9.0), torch.nan_to_num(want_v, 9.0))
        want_out, want_w = ref.accumulate(before_w, q_out.cpu(), kc.cpu(), vc.cpu(), table, lens, scale)
        T = int(lens.max())
        ref.close_out(out.cpu(), want_out, ref.out_slack(q_out.cpu(), kc.cpu(), vc.cpu(), scale, T))
        rows = Q * H // Hkv
        rel = ref.weight_slack(q_out.cpu(), kc.cpu(), scale, T)
        bound = rel * (want_w - before_w.double()) + (rows + 2) * 2.0 ** -23 * want_w
        assert ((weights.cpu().double() - want_w).abs() <= bound).all()

    Q = int(lens.max())                                        # the shorter prompt is padded in front
    at = lens.view(B, 1) - Q + torch.arange(Q)
    step(Q, lens, torch.stack([at, at // 7, at % 7]).to(torch.int32).contiguous(), 1)
    for i in range(4):
        lens = lens + 1
        step(1, lens, positions.view(1, B, 1).expand(3, B, 1).contiguous(), 10 + i)
        positions = positions + 1

    before = kc.cpu(), vc.cpu(), weights.cpu()
    new_lens = torch.empty((B,), dtype=torch.int32, device=DEV)
    kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device=DEV)
    pa.evict_kv(kc, vc, weights, table_d, lens.to(DEV), table_d, weights, new_lens, kept, sink=2, recent=8)
    want = ref.evict(*before, table, lens, table, budget, 2, 8)
    for got, w in zip((kc, vc, weights, new_lens, kept), want):
        assert torch.equal(torch.nan_to_num(got.cpu().float(), 9.0), torch.nan_to_num(w.float(), 9.0))
    lens = new_lens.cpu()
    assert lens.tolist() == [budget, budget]
    for i in range(3):                                         # slots and rotary positions differ now
        lens = lens + 1
        step(1, lens, positions.view(1, B, 1).expand(3, B, 1).contiguous(), 20 + i)
        positions = positions + 1
    assert pa.device_error() == 0


def test_samples_of_one_prompt():
    n, H, Hkv, D, bs, P = 6, 8, 2, 128, 16, 90
    dtype, scale = torch.bfloat16, 1 / math.sqrt(128)
    inv_freq, axes, phases, axes_d = rotary(D, 1)
    ptable, first = ref.tables([P], bs, 1)
    own, pool = ref.tables([3 * bs] * n, bs, 2, first=first)
    kc = torch.full((pool, bs, Hkv, D), float("nan"), dtype=dtype, device=DEV)
    vc = kc.clone()

    def new_tokens(B, Q, seed):
        t = ref.normal((B, Q, H + 2 * Hkv, D), dtype, seed).to(DEV)
        return t[:, :, :H], t[:, :, H:H + Hkv], t[:, :, H + Hkv:]

    q, k, v = new_tokens(1, P, 3)
    pos = torch.arange(P, dtype=torch.int32).view(1, 1, P).to(DEV)
    plens = torch.tensor([P], dtype=torch.int32, device=DEV)
    pa.rope_append_kv(torch.empty((1, P, H, D), dtype=dtype, device=DEV), kc, vc, q, k, v, pos, phases,
                      axes_d, ptable.to(DEV), plens)
    lens = torch.zeros((n,), dtype=torch.int32)
    for Q, seed in ((1, 4), (1, 5), (3, 6), (1, 7)):           # single tokens, and drafted ones
        pos = (P + lens.view(1, n, 1) + torch.arange(Q)).to(torch.int32)
        lens = lens + Q
        q, k, v = new_tokens(n, Q, seed)
        q_out = torch.empty((n, Q, H, D), dtype=dtype, device=DEV)
        pa.rope_append_kv(q_out, kc, vc, q, k, v, pos.contiguous().to(DEV), phases, axes_d, own.to(DEV),
                          lens.to(DEV))
        out = torch.empty_like(q_out)
        pa.decode_shared_prefix(out, q_out, kc, vc, ptable.to(DEV), plens, own.to(DEV), lens.to(DEV),
                                scale, P, 3 * bs)
        want = ref.shared_prefix(q_out.cpu(), kc.cpu(), vc.cpu(), ptable, plens.cpu(), own, lens, scale)
        ref.close_out(out.cpu(), want, ref.out_slack(q_out.cpu(), kc.cpu(), vc.cpu(), scale, P + 50))
    assert pa.device_error() == 0


@pytest.mark.parametrize("Q", [1, 40])
def test_an_empty_batch_launches_nothing(Q):
    H, Hkv, D, bs = 8, 2, 64, 16
    kc = torch.ones((4, bs, Hkv, D), dtype=torch.float16, device=DEV)
    vc = kc.clone()

    def none(*shape, dtype=torch.int32):
        return torch.empty((0,) + shape, dtype=dtype, device=DEV)

    q, kv = none(Q, H, D, dtype=torch.float16), none(Q, Hkv, D, dtype=torch.float16)
    table, lens, w = none(3), none(), none(Hkv, 3 * bs, dtype=torch.float32)
    phases = pa.rope_phases(torch.ones(32, dtype=torch.float64)).to(DEV)
    pa.rope_append_kv(q, kc, vc, q, kv, kv, torch.empty((2, 0, Q), dtype=torch.int32, device=DEV), phases,
                      torch.zeros(32, dtype=torch.int32, device=DEV), table, lens)
    assert pa.workspace_size_accumulate(q, kc, table, torch.float16, 48) >= 0
    pa.decode_accumulate(q.clone(), w, q, kc, vc, table, lens, 0.1, 48)
    ptable, plens = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    assert pa.workspace_size_shared_prefix(q, kc, ptable, table, torch.float16, 20, 48) == 0
    pa.decode_shared_prefix(q.clone(), q, kc, vc, ptable, plens, table, lens, 0.1, 20, 48)
    pa.evict_kv(kc, vc, w, table, lens, table, w, none(), none(Hkv, 7))
    torch.cuda.synchronize()
    assert (kc == 1).all() and (vc == 1).all()


def test_the_readme_example_runs():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = re.search(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S).group(1)
    names = {}
    exec(code, names)
    torch.cuda.synchronize()
    assert names["new_lens"].tolist() == [names["budget"]] * names["B"]
    assert torch.isfinite(names["out"].float()).all() and pa.device_error() == 0
