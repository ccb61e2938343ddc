"""GPU tests of the latent cache: pa.rope_append_latent and pa.decode_latent
against their 64-bit definitions."""
import math

import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 64


# ---- append ----

def append_case(seed, B, Q, H, R, bs, lens, dtype):
    table, pool = ref.tables([max(t, 0) for t in lens], bs, seed)
    g = torch.Generator().manual_seed(seed + 4)
    return dict(q_all=ref.normal((B, Q, H, 32 + P), dtype, seed + 1),
                new_all=ref.normal((B, Q, R + P + 24), dtype, seed + 2),
                cache=ref.normal((pool, bs, R + P), dtype, seed + 3), table=table,
                norm=(1 + 0.3 * torch.randn(R, generator=g)).to(dtype),
                pos=torch.randint(0, 1 << 22, (B, Q), generator=g, dtype=torch.int32),
                inv=1e4 ** (-torch.arange(P // 2, dtype=torch.float64) * 2 / P),
                lens=torch.tensor(lens, dtype=torch.int32))


def check_append(c, interleaved=False, norm=True, in_place=False, eps=1e-6, drop=False):
    R = c["norm"].numel()
    q, new = c["q_all"][..., 32:], c["new_all"][..., 16:16 + R + P]
    want_q, want = cref.append_latent(q, c["cache"], new, c["norm"] if norm else None, eps,
                                      c["pos"], c["inv"], c["table"], c["lens"], interleaved)
    d = {n: x.to(DEV) for n, x in c.items()}
    dq, dnew = d["q_all"][..., 32:], d["new_all"][..., 16:16 + R + P]
    whole = torch.full((*q.shape[:3], R + P), math.nan, dtype=q.dtype, device=DEV)
    q_out = dq if in_place else whole[..., R:]
    args = [q_out, d["cache"], dq, dnew, d["norm"] if norm else None, d["pos"]]
    if drop:
        args = [x.squeeze(1) if i in (0, 2, 3, 5) else x for i, x in enumerate(args)]
    pa.rope_append_latent(*args, pa.rope_phases(d["inv"]), d["table"], d["lens"], eps=eps,
                          interleaved=interleaved)
    torch.cuda.synchronize()
    half = torch.finfo(q.dtype).eps / 2
    # a turned element: see the 8-bit append; a normalised one: a sum of R squares (R + 4 roundings
    # of 2^-24 on a positive sum), a division, a root and two products
    big = 2 * max(q.double().abs().max().item(), new.double().abs().max().item())
    err = (q_out.cpu().double() - want_q).abs() - half * want_q.abs() - 2.0 ** -21 * big
    assert err.max().item() <= 0
    if not in_place:
        assert torch.isnan(whole[..., :R]).all()
    got = d["cache"].cpu().double()
    err = (got - want).abs()
    err -= half * want.abs()
    # (under fp16's smallest normal number, 2^-14, a step is 2^-24 whatever the value: half of it)
    err[..., :R] -= (R + 16) * 2.0 ** -24 * want[..., :R].abs() + 2.0 ** -25
    err[..., R:] -= 2.0 ** -21 * big
    untouched = want == c["cache"].double()
    assert torch.equal(got[untouched], want[untouched])
    assert err[~untouched].max().item() <= 0 if (~untouched).any() else True


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,R,bs,lens,interleaved", [
    (1, 1, 1, 512, 64, [1], False),
    (3, 1, 16, 512, 64, [100, 65, 64], True),
    (2, 5, 7, 256, 16, [20, 5], False),
    (2, 33, 128, 128, 32, [200, 33], True),
    (4, 3, 5, 512, 16, [3, 2, 18, 1000], False),
    (1, 700, 3, 512, 32, [701], False),
])
def test_append_matches_definition(B, Q, H, R, bs, lens, interleaved, dtype):
    check_append(append_case(B * 10 + Q, B, Q, H, R, bs, lens, dtype), interleaved)


def test_append_padding_masked_and_far_entries():
    c = append_case(5, 6, 3, 4, 256, 16, [2, 0, -7, 40, 33, 1], torch.bfloat16)
    c["table"][3, 2] = -1
    c["table"][4, 2] = c["cache"].shape[0] + 3
    c["pos"][2] = -(1 << 31)
    check_append(c)
    c["lens"][3] = 1 << 30
    check_append(c, in_place=True, norm=False)


def test_append_one_token_without_its_dimension():
    c = append_case(7, 3, 1, 16, 512, 64, [100, 65, 64], torch.bfloat16)
    check_append(c, drop=True, eps=0.5)
    c["new_all"].zero_()
    check_append(c, eps=1e-6)   # 0 / sqrt(eps)


# ---- attention ----

def case(seed, B, Q, H, R, bs, lens, dtype):
    table, pool = ref.tables(lens, bs, seed)
    return dict(q=ref.normal((B, Q, H, R + P), dtype, seed + 1),
                cache=ref.normal((pool, bs, R + P), dtype, seed + 2), table=table,
                lens=torch.tensor(lens, dtype=torch.int32))


def run(c, scale, longest=None, stream=None, own_workspace=True, drop=False):
    d = {k: v.to(DEV) for k, v in c.items()}
    if drop:
        d["q"] = d["q"].squeeze(1)
    R = c["q"].shape[-1] - P
    out = torch.full((*d["q"].shape[:-1], R), math.nan, dtype=c["q"].dtype, device=DEV)
    longest = max(0, int(c["lens"].max())) if longest is None else longest
    ws = None
    if own_workspace:
        need = pa.workspace_size_latent(d["q"], d["cache"], R, d["table"], longest)
        ws = torch.full((need // 4 + 4,), math.nan, device=DEV)
    torch.cuda.synchronize()
    pa.decode_latent(out, d["q"], d["cache"], d["table"], d["lens"], scale, longest, workspace=ws,
                     stream=stream)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu().reshape(*c["q"].shape[:-1], R)


def definition(c, scale, lens=None, cache=None):
    """(output, slack): the weights that meet the values are rounded once to the
    cache's type."""
    cache = c["cache"] if cache is None else cache
    k = cache.double().unsqueeze(2)
    R = k.shape[3] - P
    want = cref.attention(c["q"], k, k[..., :R], c["table"], c["lens"] if lens is None else lens, scale)
    tokens = max(1, c["table"].shape[1]) * k.shape[1]
    return want, cref.attention_slack(c["q"], k, k[..., :R], scale, tokens,
                                      torch.finfo(cache.dtype).eps / 2)


def check(c, scale=None, want_lens=None, **kw):
    scale = scale or (c["q"].shape[-1] // 4) ** -0.5
    want, slack = definition(c, scale, want_lens)
    ref.close_out(run(c, scale, **kw), want, slack)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,R,bs,lens", [
    (1, 1, 1, 512, 64, [1]),
    (1, 1, 16, 512, 64, [100]),
    (3, 1, 16, 512, 16, [1, 50, 16]),
    (2, 1, 128, 512, 64, [300, 65]),
    (4, 1, 20, 256, 32, [37 * b + 1 for b in range(4)]),
    (2, 1, 64, 128, 64, [33, 640]),
    (2, 3, 5, 256, 16, [65, 3]),
    (2, 2, 128, 512, 64, [40, 129]),
    (1, 7, 40, 128, 32, [200]),
    (1, 40, 3, 512, 16, [90]),
    (1, 5, 65, 256, 64, [128]),
])
def test_matches_definition(B, Q, H, R, bs, lens, dtype):
    check(case(B * 100 + Q + H, B, Q, H, R, bs, lens, dtype))


@pytest.mark.parametrize("T,H,R", [(3000, 16, 512), (9000, 128, 128), (5000, 40, 256), (2100, 128, 512)])
def test_split_contexts(T, H, R):
    check(case(T, 1, 1, H, R, 64, [T], torch.bfloat16))
    check(case(T + 1, 2, 2, H, R, 32, [T, 7], torch.float16))


@pytest.mark.parametrize("Q", [1, 3, 12])
def test_empty_sequences_and_padding(Q):
    lens = [Q, 0, max(0, Q - 2), -4, 50, Q + 1, 0, 1]
    c = case(32 + Q, 8, Q, 9, 256, 16, [max(t, 0) for t in lens], torch.bfloat16)
    c["lens"] = torch.tensor(lens, dtype=torch.int32)
    check(c)


@pytest.mark.parametrize("Q,H", [(1, 16), (6, 16), (1, 128)])
def test_masked_pages_and_nan_in_unread_places(Q, H):
    c = case(40 + Q, 4, Q, H, 512, 16, [150, 40, 41, 90], torch.bfloat16)
    c["table"][0, 3] = -1
    c["table"][0, 9] = c["cache"].shape[0] + 5
    c["table"][1, 1] = -1
    c["table"][2, :] = -1
    used = c["table"].flatten()
    dead = torch.ones(c["cache"].shape[0], dtype=torch.bool)
    dead[used[(used >= 0) & (used < len(dead))].unique().long()] = False
    c["lens"][3] = 83                          # ends inside page 5
    clean = c["cache"].clone()
    c["cache"][dead] = math.nan
    c["cache"][int(c["table"][3, 5]), 3:] = math.nan
    clean[dead] = 0
    clean[int(c["table"][3, 5]), 3:] = 0
    scale = 144 ** -0.5
    want, slack = definition(c, scale, cache=clean)
    ref.close_out(run(c, scale), want, slack)


def test_one_sequences_nan_stays_its_own():
    c = case(45, 3, 1, 16, 512, 16, [100, 60, 200], torch.bfloat16)
    scale = 144 ** -0.5
    want, slack = definition(c, scale)
    c["q"][1] = math.nan
    got = run(c, scale)
    assert torch.isnan(got[1]).all()
    ref.close_out(got[0::2], want[0::2], slack)


def test_lengths_past_the_table_and_past_the_announced():
    c = case(51, 4, 1, 16, 256, 16, [64] * 4, torch.float16)
    c["lens"][2] = 1 << 30
    check(c, longest=64)
    check(c, longest=1 << 30)
    check(c, longest=20, want_lens=torch.tensor([32, 32, 32, 32], dtype=torch.int32))
    big = case(52, 1, 1, 16, 128, 16, [6000], torch.bfloat16)
    check(big, longest=3001, want_lens=torch.tensor([3008], dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rising_maxima(dtype):
    """Scores that rise along the context by far more than a rescale's slack, and
    ones that fall: the running maximum moves at every block."""
    c = case(61, 2, 1, 16, 512, 64, [700, 700], dtype)
    t = torch.arange(700)
    for b in range(2):
        ramp = (t if b == 0 else 699 - t).to(torch.float32) * 0.01
        for j in range(11):
            e = int(c["table"][b, j])
            n = min(64, 700 - 64 * j)
            c["cache"][e, :n, 512:] = ramp[64 * j:64 * j + n, None].to(dtype)
    c["q"][..., 512:] = 1.0
    check(c, scale=0.3)


def test_other_stream_and_torch_workspace():
    c = case(71, 3, 1, 128, 512, 64, [5000, 1, 700], torch.bfloat16)
    check(c, stream=torch.cuda.Stream(), own_workspace=False)
    check(case(72, 2, 1, 16, 512, 64, [50, 70], torch.bfloat16), drop=True)


def test_graph_replay_follows_lengths_and_tables():
    c = case(81, 4, 1, 16, 512, 64, [3000, 200, 64, 1], torch.bfloat16)
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.zeros((4, 1, 16, 512), dtype=torch.bfloat16, device=DEV)
    need = pa.workspace_size_latent(d["q"], d["cache"], 512, d["table"], 3000)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)

    def call():
        pa.decode_latent(out, d["q"], d["cache"], d["table"], d["lens"], 0.1, 3000, workspace=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c["lens"] = torch.tensor([2500, 1, 0, 9], dtype=torch.int32)
    c["table"][3, 0] = int(c["table"][1, 3])
    d["lens"].copy_(c["lens"])
    d["table"].copy_(c["table"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    want, slack = definition(c, 0.1)
    ref.close_out(out.cpu(), want, slack)


def test_equal_calls_give_equal_bits():
    c = case(91, 5, 2, 24, 512, 64, [2000, 3, 900, 64, 5000], torch.float16)
    a = run(c, 0.1)
    for _ in range(3):
        assert torch.equal(a, run(c, 0.1))
