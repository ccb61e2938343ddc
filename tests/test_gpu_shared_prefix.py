"""GPU tests of pa.decode_shared_prefix against the 64-bit definition: the
softmax over a sequence's prefix and own tokens as one (the bound is derived
in step_reference)."""
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(seed, n, Q, H, Hkv, D, bs, plens, lens, dtype):
    B = n * len(plens)
    assert len(lens) == B
    ptable, first = ref.tables(plens, bs, seed)
    table, pool = ref.tables(lens, bs, seed + 1, first=first)
    return dict(q=ref.normal((B, Q, H, D), dtype, seed + 2),
                k_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 3),
                v_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 4), ptable=ptable,
                plens=torch.tensor(plens, dtype=torch.int32), table=table,
                lens=torch.tensor(lens, dtype=torch.int32))


def run(c, scale, out_dtype=None, max_p=None, max_own=None, stream=None, own_workspace=True):
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.full(c["q"].shape, float("nan"), dtype=out_dtype or c["q"].dtype, device=DEV)
    mp = max_p if max_p is not None else max(0, int(c["plens"].max()))
    mo = max_own if max_own is not None else max(0, int(c["lens"].max()))
    ws = None
    if own_workspace:
        need = pa.workspace_size_shared_prefix(d["q"], d["k_cache"], d["ptable"], d["table"],
                                               out.dtype, mp, mo)
        ws = torch.full((need // 4 + 1,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    pa.decode_shared_prefix(out, d["q"], d["k_cache"], d["v_cache"], d["ptable"], d["plens"],
                            d["table"], d["lens"], scale, mp, mo, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu()


def check(c, scale=None, **kw):
    scale = scale or 1 / math.sqrt(c["q"].shape[-1])
    want = ref.shared_prefix(c["q"], c["k_cache"], c["v_cache"], c["ptable"], c["plens"],
                             c["table"], c["lens"], scale)
    pages = [int((c[t] >= 0).sum(1).max()) for t in ("ptable", "table")]  # attended at most
    tokens = max(1, sum(pages)) * c["k_cache"].shape[1]
    ref.close_out(run(c, scale, **kw), want,
                  ref.out_slack(c["q"], c["k_cache"], c["v_cache"], scale, tokens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,Q,H,Hkv,D,bs,plens,lens", [
    (1, 1, 1, 1, 64, 16, [1], [1]),
    (1, 1, 4, 2, 128, 16, [100], [30]),
    (3, 1, 8, 2, 128, 16, [77], [1, 50, 16]),          # up to 16 rows: the warp-level kernel
    (8, 1, 8, 2, 128, 16, [1000], [5 * b + 1 for b in range(8)]),
    (40, 1, 32, 8, 128, 16, [333], [b % 7 + 1 for b in range(40)]),   # two row tiles
    (2, 1, 16, 1, 256, 32, [500], [33, 64]),
    (1, 1, 16, 1, 256, 16, [500], [100]),              # a compact tile
    (5, 2, 4, 4, 64, 32, [65, 64, 1, 300], [2 + b for b in range(20)]),
    (3, 4, 16, 2, 256, 16, [40, 129], [4, 9, 30, 4, 100, 5]),
    (2, 70, 8, 2, 128, 16, [200], [70, 90]),
])
def test_matches_definition(n, Q, H, Hkv, D, bs, plens, lens, dtype):
    check(case(n * 100 + Q, n, Q, H, Hkv, D, bs, plens, lens, dtype))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_output_types(out_dtype):
    check(case(31, 6, 1, 8, 2, 128, 16, [400], [10 * b + 1 for b in range(6)], torch.bfloat16),
          out_dtype=out_dtype)


@pytest.mark.parametrize("Q", [1, 3, 12])
def test_empty_prefixes_empty_sequences_and_padding(Q):
    lens = [Q, 0, max(0, Q - 2), -4, 50, Q + 1, 0, 1]
    c = case(32 + Q, 4, Q, 8, 2, 128, 16, [0, 45], [max(t, 0) for t in lens], torch.bfloat16)
    c["lens"] = torch.tensor(lens, dtype=torch.int32)
    check(c)
    c["plens"][1] = -2
    check(c, max_p=45)


@pytest.mark.parametrize("n", [2, 20])
def test_masked_pages_and_nan_in_unread_places(n):
    c = case(40 + n, n, 1, 8, 2, 128, 16, [150], [40 + b for b in range(n)], torch.bfloat16)
    c["ptable"][0, 3] = -1
    c["ptable"][0, 9] = c["k_cache"].shape[0] + 5
    c["table"][0, 1] = -1
    c["table"][1, :] = -1
    used = torch.cat([c["ptable"].flatten(), c["table"].flatten()])
    dead = torch.ones(c["k_cache"].shape[0], dtype=torch.bool)
    dead[used[(used >= 0) & (used < len(dead))].unique().long()] = False
    c["plens"][0] = 135                        # ends inside page 8
    for cache in (c["k_cache"], c["v_cache"]):
        cache[dead] = float("nan")
        cache[int(c["ptable"][0, 8]), 7:] = float("nan")
    check(c, max_p=150)


def test_lengths_past_the_tables():
    c = case(51, 5, 1, 8, 2, 64, 16, [64], [32] * 5, torch.float16)
    c["plens"][0], c["lens"][2] = 1 << 30, 1 << 30
    check(c, max_p=64, max_own=32)


@pytest.mark.parametrize("n,plen,own", [(2, 30000, 5), (12, 9000, 700), (150, 600, 40)])
def test_every_split(n, plen, own):
    check(case(60 + n, n, 1, 8, 2, 64, 16, [plen], [own + b % 5 for b in range(n)], torch.bfloat16))


def test_equals_attention_over_one_table():
    """The same tokens behind one table each: decode_multi over prefix and own pages."""
    n, Q, bs = 4, 3, 16
    c = case(70, n, Q, 8, 2, 128, bs, [64], [20, 3, 33, 16], torch.bfloat16)
    d = {k: v.to(DEV) for k, v in c.items()}
    whole = torch.cat([d["ptable"].expand(n, -1), d["table"]], 1).contiguous()
    want = torch.zeros(c["q"].shape, device=DEV)
    pa.decode_multi(want, d["q"], d["k_cache"], d["v_cache"], whole, d["lens"] + 64, 0.1, 97)
    got = run(c, 0.1, out_dtype=torch.float32)
    slack = 2 * ref.out_slack(c["q"], c["k_cache"], c["v_cache"], 0.1, 97)
    assert (got - want.cpu()).abs().max().item() <= slack


def test_same_bits_twice_other_stream_one_token_form_and_graph():
    c = case(80, 20, 1, 32, 8, 128, 16, [2000], [3 * b + 1 for b in range(20)], torch.bfloat16)
    want = run(c, 0.1)
    for kw in (dict(), dict(stream=torch.cuda.Stream(DEV)),
               dict(stream=torch.cuda.Stream(DEV), own_workspace=False)):
        assert torch.equal(run(c, 0.1, **kw), want)
    d = {k: v.to(DEV) for k, v in c.items()}
    q, out = d["q"][:, 0].contiguous(), torch.zeros((20, 32, 128), dtype=torch.bfloat16, device=DEV)
    args = (out, q, d["k_cache"], d["v_cache"], d["ptable"], d["plens"], d["table"], d["lens"], 0.1,
            2000, 58)
    pa.decode_shared_prefix(*args)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[:, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_shared_prefix(*args)
    out.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[:, 0])


@pytest.mark.parametrize("kernel", ["mma", "tile"])
def test_either_kernel_forced(kernel, switches):
    switches(kernel=kernel)
    check(case(90, 5, 3, 8, 2, 128, 16, [150, 33], [3 + 7 * b for b in range(10)], torch.bfloat16))
    check(case(91, 20, 1, 16, 1, 256, 16, [100], [5 + b for b in range(20)], torch.float16))


def test_two_graphs_share_a_workspace():
    cs = [case(92, 20, 1, 8, 2, 128, 16, [700], [40] * 20, torch.bfloat16),
          case(93, 3, 4, 8, 2, 128, 16, [90], [9, 30, 70], torch.bfloat16)]
    want = [run(c, 0.1) for c in cs]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    graphs, outs, keep = [], [], []
    for c in cs:
        d = {k: v.to(DEV) for k, v in c.items()}
        out = torch.zeros(c["q"].shape, dtype=c["q"].dtype, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.decode_shared_prefix(out, d["q"], d["k_cache"], d["v_cache"], d["ptable"], d["plens"],
                                    d["table"], d["lens"], 0.1, int(c["plens"].max()),
                                    int(c["lens"].max()), workspace=ws)
        graphs.append(graph), outs.append(out), keep.append(d)
    for i in (0, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i].cpu(), want[i])


def widened(c, tokens):
    """The same prefixes in tables of `tokens` tokens: announced so long, they
    are given two tiles to a CTA from 129 rows of a kv head on."""
    bs = c["k_cache"].shape[1]
    wide = torch.full((c["ptable"].shape[0], tokens // bs), -1, dtype=torch.int32)
    wide[:, :c["ptable"].shape[1]] = c["ptable"]
    return dict(c, ptable=wide)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,Q,H,Hkv,D,bs,plens", [
    (33, 1, 32, 8, 64, 32, [1]),           # 132 rows
    (40, 1, 32, 8, 128, 16, [127]),
    (64, 1, 32, 8, 128, 32, [128]),        # 256
    (65, 1, 32, 8, 128, 16, [129]),        # 260: a third tile
    (96, 1, 32, 8, 64, 16, [333]),         # 384
    (22, 3, 16, 8, 128, 16, [500, 0, 77]),
    (11, 13, 8, 8, 64, 16, [400, 401]),    # a head to a kv head, padding
    (9, 1, 16, 1, 128, 32, [5000]),        # 144 rows of one kv head, several partitions
    (17, 2, 64, 8, 128, 16, [4999]),       # 272
])
def test_two_tiles_to_a_cta(n, Q, H, Hkv, D, bs, plens, dtype):
    B = n * len(plens)
    c = case(n * 1000 + D, n, Q, H, Hkv, D, bs, plens, [(b * 7) % 30 + 1 for b in range(B)], dtype)
    check(widened(c, 65536), max_p=65536)


def test_two_tiles_masked_pages_and_nan_in_unread_places():
    c = case(900, 40, 1, 32, 8, 128, 16, [1000], [b % 9 + 1 for b in range(40)], torch.bfloat16)
    c["ptable"][0, 3] = -1
    c["ptable"][0, 20] = c["k_cache"].shape[0] + 5
    c["ptable"][0, 24:34] = -1                 # a whole block of 8 pages among them
    used = torch.cat([c["ptable"].flatten(), c["table"].flatten()])
    dead = torch.ones(c["k_cache"].shape[0], dtype=torch.bool)
    dead[used[(used >= 0) & (used < len(dead))].unique().long()] = False
    c["plens"][0] = 985                        # ends inside a page
    last = int(c["ptable"][0, 61])
    for cache in (c["k_cache"], c["v_cache"]):
        cache[dead] = float("nan")
        cache[last, 9:] = float("nan")
    check(widened(c, 65536), max_p=65536)
    c["ptable"][0, :] = -1                     # no page at all
    check(widened(c, 65536), max_p=65536)


def test_two_tiles_scores_that_rise_and_fall():
    """Maxima that move by more than the slack, up along the prefix and down again."""
    c = case(901, 64, 1, 32, 8, 128, 16, [2000], [3] * 64, torch.float16)
    ramp = 1 + 7 * torch.sin(torch.arange(c["k_cache"].shape[0]) / 9.0).abs()
    c["k_cache"] = (c["k_cache"].float() * ramp.view(-1, 1, 1, 1)).to(torch.float16)
    check(widened(c, 65536), scale=0.2, max_p=65536)


def test_two_tiles_same_bits_twice_and_in_a_graph():
    c = widened(case(902, 70, 1, 32, 8, 128, 16, [3000], [b % 20 + 1 for b in range(70)],
                     torch.bfloat16), 65536)
    first = run(c, 0.1, max_p=65536)
    for own in (True, False):
        assert torch.equal(run(c, 0.1, max_p=65536, own_workspace=own), first)
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.empty_like(d["q"])
    mo = int(c["lens"].max())
    ws = torch.empty(pa.workspace_size_shared_prefix(d["q"], d["k_cache"], d["ptable"], d["table"],
                                                     out.dtype, 65536, mo), dtype=torch.uint8, device=DEV)
    call = lambda: pa.decode_shared_prefix(out, d["q"], d["k_cache"], d["v_cache"], d["ptable"],
                                           d["plens"], d["table"], d["lens"], 0.1, 65536, mo, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    out.zero_()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first) and pa.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Q,H,Hkv,D,bs", [(40, 32, 8, 128, 16), (150, 8, 8, 64, 32), (33, 32, 8, 64, 16)])
def test_two_tiles_of_the_sequences_own_rows(Q, H, Hkv, D, bs, dtype):
    """Own rows that go two tiles to a CTA, causal among themselves, with padding."""
    lens = [Q, Q + 1, 700, Q - 2, 129, 0, 333, Q + 128]
    c = case(Q * 10 + D, 4, Q, H, Hkv, D, bs, [60, 0], lens, dtype)
    wide = torch.full((8, 65536 // bs), -1, dtype=torch.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    check(dict(c, table=wide), max_own=65536)


APART = 1 << 20   # announced so long, a prefix is never read by each sequence itself


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,Q,H,Hkv,D,bs,plens,lens", [
    (1, 1, 4, 2, 128, 16, [100], [30]),
    (3, 1, 8, 2, 128, 16, [77], [1, 50, 16]),
    (8, 1, 8, 2, 64, 32, [1000], [5 * b + 1 for b in range(8)]),
    (2, 1, 16, 1, 256, 32, [500], [33, 64]),
    (5, 2, 4, 4, 64, 32, [65, 64, 1, 300], [2 + b for b in range(20)]),
    (3, 4, 16, 2, 256, 16, [40, 129], [4, 9, 30, 4, 100, 5]),
    (4, 3, 8, 2, 128, 16, [0, 45], [3, 0, 1, -4, 50, 4, 0, 1]),    # empty ones and padding
])
def test_in_launches_of_their_own(n, Q, H, Hkv, D, bs, plens, lens, dtype):
    """The prefix and the own pages apart, and joined, at sizes that go in one launch too."""
    c = case(n * 10 + Q, n, Q, H, Hkv, D, bs, plens, [max(t, 0) for t in lens], dtype)
    c["lens"] = torch.tensor(lens, dtype=torch.int32)
    check(c)
    check(widened(c, APART), max_p=APART)


def test_in_launches_of_their_own_masked_pages_and_nan_in_unread_places():
    c = case(950, 3, 1, 8, 2, 128, 16, [150], [40, 41, 42], torch.bfloat16)
    c["ptable"][0, 3] = -1
    c["ptable"][0, 6] = c["k_cache"].shape[0] + 5
    c["table"][0, 1] = -1
    c["table"][1, :] = -1
    used = torch.cat([c["ptable"].flatten(), c["table"].flatten()])
    dead = torch.ones(c["k_cache"].shape[0], dtype=torch.bool)
    dead[used[(used >= 0) & (used < len(dead))].unique().long()] = False
    c["plens"][0] = 135
    for cache in (c["k_cache"], c["v_cache"]):
        cache[dead] = float("nan")
        cache[int(c["ptable"][0, 8]), 7:] = float("nan")
    check(c, max_p=150)
    check(widened(c, APART), max_p=APART)


def test_contexts_longer_than_announced_stay_in_bounds():
    """Lengths past those announced: tokens are left out, nothing else is touched."""
    for n, Q in ((4, 1), (4, 3), (40, 4)):
        c = case(960 + n, n, Q, 8, 2, 128, 16, [900], [70 + b for b in range(n)], torch.bfloat16)
        out = run(c, 0.1, max_p=200, max_own=20)
        assert torch.isfinite(out.float()).all()


def test_two_graphs_share_a_workspace_of_launches_apart():
    cs = [widened(case(94, 20, 1, 8, 2, 128, 16, [700], [40] * 20, torch.bfloat16), APART),
          widened(case(95, 3, 4, 8, 2, 128, 16, [90], [9, 30, 70], torch.bfloat16), APART)]
    want = [run(c, 0.1, max_p=APART) for c in cs]
    ws = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    graphs, outs, keep = [], [], []
    for c in cs:
        d = {k: v.to(DEV) for k, v in c.items()}
        out = torch.zeros(c["q"].shape, dtype=c["q"].dtype, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.decode_shared_prefix(out, d["q"], d["k_cache"], d["v_cache"], d["ptable"], d["plens"],
                                    d["table"], d["lens"], 0.1, APART, int(c["lens"].max()), workspace=ws)
        graphs.append(graph), outs.append(out), keep.append(d)
    for i in (0, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i].cpu(), want[i])
