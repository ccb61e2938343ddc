"""GPU tests of pa.rope_append_kv against the 64-bit definition.

Tolerance of one turned element, x cos a - y sin a of 16-bit x, y:
  - the result's rounding to the cache's type: eps / 2 relative;
  - fp32 arithmetic: two products, one sum (2^-24 each, relative to terms of
    at most |x| + |y|), and sine and cosine within 2 ulp (2 * 2^-23, of values
    up to 1): 5 * 2^-23 of |x| + |y| covers them;
  - the angle: the kernel's fraction of a turn is a 32-bit integer rounded to
    24 bits (pi * 2^-25 rad) and truncated from 64 bits (2 pi * 2^-32 rad); the
    table's own rounding is 2^-53 relative twice, as is the reference's
    product: 3 * 2^-53 * pos * f rad in all;
  - half a step of fp16's smallest numbers, 2^-25.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(seed, B, Q, H, Hkv, D, bs, rot, naxes, dtype, lens, far=1000, fused=True):
    g = torch.Generator().manual_seed(seed)
    table, pool = ref.tables(lens, bs, seed)
    half = rot // 2
    c = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32),
             inv_freq=1e4 ** (-torch.arange(half).double() * 2 / rot),
             axes=(torch.arange(half) * 7 % naxes).to(torch.int32),
             pos=torch.randint(-far, far, (naxes, B, Q), generator=g, dtype=torch.int64).to(torch.int32),
             k_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 1),
             v_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 2))
    if fused:
        qkv = ref.normal((B, Q, H + 2 * Hkv, D), dtype, seed + 3)
        c["qkv"] = qkv
        c.update(q=qkv[:, :, :H], k=qkv[:, :, H:H + Hkv], v=qkv[:, :, H + Hkv:])
    else:
        c.update(q=ref.normal((B, Q, H, D), dtype, seed + 3),
                 k=ref.normal((B, Q, Hkv, D), dtype, seed + 4),
                 v=ref.normal((B, Q, Hkv, D), dtype, seed + 5))
    return c


def run(c, interleaved, in_place=False):
    d = {k: v.to(DEV) for k, v in c.items()}
    if "qkv" in c:  # views of the one tensor, as on the host
        H, Hkv = c["q"].shape[2], c["k"].shape[2]
        d.update(q=d["qkv"][:, :, :H], k=d["qkv"][:, :, H:H + Hkv], v=d["qkv"][:, :, H + Hkv:])
    q_out = d["q"] if in_place else torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype,
                                               device=DEV)
    phases = pa.rope_phases(d["inv_freq"])
    pa.rope_append_kv(q_out, d["k_cache"], d["v_cache"], d["q"], d["k"], d["v"], d["pos"], phases,
                      d["axes"], d["table"], d["lens"], interleaved=interleaved)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return q_out.cpu(), d["k_cache"].cpu(), d["v_cache"].cpu()


def check(c, got, interleaved, far):
    want = ref.rope_append(c["q"], c["k_cache"], c["v_cache"], c["k"], c["v"], c["pos"],
                           c["inv_freq"], c["axes"], c["table"], c["lens"], interleaved)
    eps = torch.finfo(c["q"].dtype).eps
    big = 2 * max(c["q"].abs().max().item(), c["k"].abs().max().item())  # |x| + |y| at most
    slack = big * (5 * 2.0 ** -23 + np.pi * 2.0 ** -25 + 2 * np.pi * 2.0 ** -32
                   + 3 * 2.0 ** -53 * far) + 2.0 ** -25
    for g, w in zip(got[:2], want[:2]):
        err = (g.double() - w).abs()
        assert (err <= eps / 2 * w.abs() + slack).all(), err.max().item()
    assert torch.equal(got[2].double(), want[2])           # values are copied
    # cache slots that no new token went to keep their bits
    B, Q = c["q"].shape[:2]
    bs = c["k_cache"].shape[1]
    touched = {ref.slot(c["table"][b], int(c["lens"][b]) - Q + i, bs, len(c["k_cache"]))
               for b in range(B) for i in range(Q)} - {None}
    same = torch.ones(c["k_cache"].shape[:2], dtype=torch.bool)
    for at in touched:
        same[at] = False
    assert torch.equal(got[1][same], c["k_cache"][same])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,rot,naxes", [
    (1, 1, 1, 1, 64, 16, 16, 1),
    (8, 1, 32, 8, 128, 16, 128, 3),
    (3, 7, 8, 2, 64, 32, 32, 2),
    (2, 33, 16, 1, 256, 16, 64, 4),
    (5, 5, 4, 4, 256, 32, 256, 3),
    (2, 131, 1, 1, 64, 16, 64, 1),
    (3, 1700, 4, 2, 64, 16, 48, 3),
])
def test_matches_definition(B, Q, H, Hkv, D, bs, rot, naxes, dtype, interleaved):
    lens = [Q + 5 * b for b in range(B)]
    if B > 1:
        lens[-1] = Q // 2      # padding before its first token
        lens[0] = Q + 3 * bs + 1
    c = case(B * 100 + Q, B, Q, H, Hkv, D, bs, rot, naxes, dtype, lens)
    check(c, run(c, interleaved), interleaved, 1000)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions_lose_nothing(far):
    c = case(5, 2, 9, 4, 2, 128, 16, 128, 3, torch.float16, [9, 30], far=far)
    check(c, run(c, False), False, far)


def test_in_place_and_separate_tensors():
    c = case(6, 3, 4, 8, 2, 128, 16, 128, 2, torch.bfloat16, [4, 40, 17], fused=False)
    check(c, run(c, True), True, 1000)
    check(c, run(c, True, in_place=True), True, 1000)
    c = case(7, 3, 4, 8, 2, 128, 16, 64, 2, torch.bfloat16, [4, 40, 17])
    check(c, run(c, False, in_place=True), False, 1000)


def test_padding_masked_pages_lengths_past_the_table_and_foreign_axes():
    c = case(8, 6, 3, 4, 2, 64, 16, 64, 2, torch.bfloat16, [3, 0, -5, 2, 50, 50])
    c["table"][4, 3] = -1                       # the new tokens' page is masked
    c["table"][5, 3] = c["k_cache"].shape[0]    # and here out of range
    c["lens"][0] = 1 << 30                      # past the table's reach
    c["axes"][5] = 2                            # outside [0, 2): not turned
    c["axes"][9] = -1
    check(c, run(c, False), False, 1000)


def test_one_token_form_other_stream_and_graph():
    c = case(9, 4, 1, 8, 2, 128, 16, 128, 3, torch.bfloat16, [1, 20, 33, 16], fused=False)
    want = run(c, False)
    d = {k: v.to(DEV) for k, v in c.items()}
    phases = pa.rope_phases(d["inv_freq"])
    q_out = torch.zeros_like(d["q"])
    args = (q_out[:, 0], d["k_cache"], d["v_cache"], d["q"][:, 0], d["k"][:, 0], d["v"][:, 0],
            d["pos"][:, :, 0].contiguous(), phases, d["axes"], d["table"], d["lens"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream(DEV)
    pa.rope_append_kv(*args, stream=side)
    side.synchronize()
    for got, w in zip((q_out, d["k_cache"], d["v_cache"]), want):
        assert torch.equal(got.cpu(), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.rope_append_kv(*args)
    d["q"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out.cpu(), -want[0])


def test_append_then_attend_equals_plain_append():
    """Angles of zero: rope_append_kv is append_kv, and attention sees its keys."""
    c = case(10, 3, 1, 8, 2, 128, 16, 128, 1, torch.float16, [5, 40, 16], fused=False)
    d = {k: v.to(DEV) for k, v in c.items()}
    d["pos"].zero_()
    kc, vc = d["k_cache"].clone(), d["v_cache"].clone()
    pa.append_kv(kc, vc, d["k"][:, 0], d["v"][:, 0], d["table"], d["lens"] - 1)
    q_out = torch.zeros_like(d["q"])
    pa.rope_append_kv(q_out, d["k_cache"], d["v_cache"], d["q"], d["k"], d["v"], d["pos"],
                      pa.rope_phases(d["inv_freq"]), d["axes"], d["table"], d["lens"])
    out = [torch.zeros((3, 8, 128), device=DEV) for _ in range(2)]
    pa.decode(out[0], d["q"][:, 0].contiguous(), kc, vc, d["table"], d["lens"], 0.1)
    pa.decode(out[1], q_out[:, 0].contiguous(), d["k_cache"], d["v_cache"], d["table"], d["lens"], 0.1)
    assert torch.equal(q_out, d["q"]) and torch.equal(kc, d["k_cache"]) and torch.equal(vc, d["v_cache"])
    assert torch.equal(out[0], out[1])
