"""GPU tests of pa.decode_accumulate against the 64-bit definition; the bounds
are derived in step_reference (a weight's relative error; an output's error)."""
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(seed, B, Q, H, Hkv, D, bs, lens, dtype, extra_pages=1):
    width = max((max(t, 0) + bs - 1) // bs for t in lens) + extra_pages
    table, pool = ref.tables(lens, bs, seed, width=width)
    g = torch.Generator().manual_seed(seed)
    return dict(q=ref.normal((B, Q, H, D), dtype, seed + 1),
                k_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 2),
                v_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 3), table=table,
                lens=torch.tensor(lens, dtype=torch.int32),
                weights=torch.rand((B, Hkv, width * bs), generator=g))


def run(c, scale, out_dtype=None, in_place=False, max_len=None, stream=None, own_workspace=True):
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.full(c["q"].shape, float("nan"), dtype=out_dtype or c["q"].dtype, device=DEV)
    new = d["weights"] if in_place else torch.full_like(d["weights"], -5.0)
    longest = max_len if max_len is not None else max(0, int(c["lens"].max()))
    ws = None
    if own_workspace:  # NaN first, so that a read of what nothing wrote shows
        need = pa.workspace_size_accumulate(d["q"], d["k_cache"], d["table"], out.dtype, longest)
        ws = torch.full((need // 4 + 1,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    pa.decode_accumulate(out, new, d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], scale,
                         longest, weights=None if in_place else d["weights"], workspace=ws,
                         stream=stream)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu(), new.cpu()


def check(c, scale=None, **kw):
    scale = scale or 1 / math.sqrt(c["q"].shape[-1])
    out, new = run(c, scale, **kw)
    want_out, want = ref.accumulate(c["weights"], c["q"], c["k_cache"], c["v_cache"], c["table"],
                                    c["lens"], scale)
    reach = torch.clamp(c["lens"], 0, c["weights"].shape[2]).tolist()
    T = max(1, max(reach))
    ref.close_out(out, want_out, ref.out_slack(c["q"], c["k_cache"], c["v_cache"], scale, T))
    rows = c["q"].shape[1] * (c["q"].shape[2] // c["k_cache"].shape[2])
    rel = ref.weight_slack(c["q"], c["k_cache"], scale, T)
    for b, t in enumerate(reach):
        added = want[b, :, :t] - c["weights"][b, :, :t].double()
        bound = rel * added + (rows + 2) * 2.0 ** -23 * want[b, :, :t]
        err = (new[b, :, :t].double() - want[b, :, :t]).abs()
        assert (err <= bound).all(), (err - bound).max().item()
        rest = c["weights"][b, :, t:] if kw.get("in_place") else torch.full((), -5.0)
        assert (new[b, :, t:] == rest).all()      # past the tokens: as they were


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,lens", [
    (1, 1, 1, 1, 64, 16, [1]),
    (4, 1, 32, 8, 128, 16, [1, 700, 33, 16]),
    (2, 1, 16, 1, 256, 32, [300, 1025]),       # the tile kernel
    (3, 1, 8, 1, 256, 16, [300, 17, 64]),
    (2, 1, 4, 4, 64, 32, [5000, 63]),
    (3, 4, 8, 2, 128, 16, [2, 50, 333]),       # a sequence shorter than its query tokens
    (2, 5, 16, 1, 64, 16, [5, 200]),
    (2, 33, 8, 2, 128, 32, [40, 500]),
    (1, 130, 4, 4, 256, 16, [257]),
])
def test_matches_definition(B, Q, H, Hkv, D, bs, lens, dtype):
    check(case(B * 1000 + Q, B, Q, H, Hkv, D, bs, lens, dtype))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q", [1, 9])
def test_in_place_and_output_types(Q, out_dtype):
    c = case(40 + Q, 3, Q, 8, 2, 128, 16, [9, 100, 1000], torch.bfloat16)
    check(c, out_dtype=out_dtype, in_place=True)


@pytest.mark.parametrize("Q", [1, 20])
def test_masked_pages_nan_in_unread_places_and_empty_sequences(Q):
    c = case(50 + Q, 5, Q, 8, 2, 128, 16, [100, 40, 0, -3, 64], torch.bfloat16)
    c["table"][0, 2] = -1
    c["table"][0, 6] = c["k_cache"].shape[0]
    c["table"][1, :] = -1                       # a sequence whose pages are all masked
    live = c["table"][(c["table"] >= 0) & (c["table"] < c["k_cache"].shape[0])].unique().long()
    dead = torch.ones(c["k_cache"].shape[0], dtype=torch.bool)
    dead[live] = False
    for cache in (c["k_cache"], c["v_cache"]):
        cache[dead] = float("nan")              # pages of no sequence
        last = int(c["table"][0, 100 // 16]) if 0 <= int(c["table"][0, 100 // 16]) < len(cache) else -1
        if last >= 0:
            cache[last, 100 % 16:] = float("nan")   # slots past the last token
    check(c)
    check(c, in_place=True)


def test_lengths_past_the_table():
    c = case(60, 2, 1, 8, 2, 64, 16, [90, 30], torch.float16, extra_pages=0)
    c["lens"][0] = 1 << 30
    check(c, max_len=96)


@pytest.mark.parametrize("B,T", [(1, 40000), (70, 300)])
def test_every_split(B, T):
    """Long single sequences (partials through the workspace) and many short ones (one pass)."""
    check(case(70 + B, B, 1, 8, 2, 64, 16, [T - 3 * b for b in range(B)], torch.bfloat16))


def test_weights_of_each_row_sum_to_one():
    c = case(80, 3, 7, 8, 2, 128, 16, [7, 400, 90], torch.bfloat16)
    c["weights"].zero_()
    _, new = run(c, 0.09, in_place=True)
    # 7 query tokens of 4 heads on each kv head, every one with a token to see
    assert (new.double().sum(2) - 28).abs().max() < 28 * ref.weight_slack(c["q"], c["k_cache"], 0.09, 400)


def test_same_bits_twice_other_stream_allocator_workspace_and_graph():
    c = case(90, 2, 1, 32, 8, 128, 16, [3000, 5], torch.bfloat16)
    want = run(c, 0.1)
    for kw in (dict(), dict(stream=torch.cuda.Stream(DEV)), dict(own_workspace=False),
               dict(stream=torch.cuda.Stream(DEV), own_workspace=False)):
        got = run(c, 0.1, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d = {k: v.to(DEV) for k, v in c.items()}
    out, new = torch.zeros_like(d["q"]), torch.full_like(d["weights"], -5.0)
    args = (out, new, d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], 0.1, 3000)
    pa.decode_accumulate(*args, weights=d["weights"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_accumulate(*args, weights=d["weights"])
    out.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(new.cpu(), want[1])


def test_output_is_that_of_plain_decode():
    c = case(95, 3, 1, 32, 8, 128, 16, [900, 64, 1], torch.float16)
    d = {k: v.to(DEV) for k, v in c.items()}
    plain = torch.zeros((3, 32, 128), device=DEV)
    pa.decode_splitkv(plain, d["q"][:, 0].contiguous(), d["k_cache"], d["v_cache"], d["table"],
                      d["lens"], 0.1, 900)
    out = torch.zeros((3, 32, 128), device=DEV)
    pa.decode_accumulate(out, d["weights"], d["q"][:, 0].contiguous(), d["k_cache"], d["v_cache"],
                         d["table"], d["lens"], 0.1, 900)
    # the same sums, possibly split elsewhere: twice the error of either
    slack = 2 * ref.out_slack(c["q"], c["k_cache"], c["v_cache"], 0.1, 900)
    assert (out - plain).abs().max().item() <= slack


@pytest.mark.parametrize("kernel", ["mma", "tile"])
@pytest.mark.parametrize("Q,H,Hkv,D", [(1, 8, 2, 128), (3, 8, 2, 64), (12, 8, 2, 128), (2, 16, 1, 256)])
def test_either_kernel_forced(kernel, Q, H, Hkv, D, switches):
    switches(kernel=kernel)
    check(case(100 + Q, 2, Q, H, Hkv, D, 16, [50, 400], torch.float16))


@pytest.mark.parametrize("B,Q,T,limit", [(2, 1, 2000, 96), (1, 1, 30000, 9000), (40, 1, 3000, 1500),
                                         (2, 20, 3000, 1000), (40, 33, 700, 500)])
def test_contexts_longer_than_announced_drop_the_rest(B, Q, T, limit):
    """Tokens past max_context_len's pages are in neither the output nor the
    weights, which they keep; by every kernel and plan that adds weights."""
    c = case(110 + B, B, Q, 8, 2, 128, 16, [T - b for b in range(B)], torch.bfloat16)
    scale, end = 0.1, (limit + 15) // 16 * 16
    out, new = run(c, scale, max_len=limit)
    masked = {k: v.clone() for k, v in c.items()}
    masked["table"][:, end // 16:] = -1      # the same tokens, left out by their pages
    want_out, want = ref.accumulate(c["weights"], c["q"], c["k_cache"], c["v_cache"], masked["table"],
                                    c["lens"], scale)
    ref.close_out(out, want_out, ref.out_slack(c["q"], c["k_cache"], c["v_cache"], scale, T))
    rel = ref.weight_slack(c["q"], c["k_cache"], scale, T)
    for b in range(B):
        t = T - b
        added = want[b, :, :t] - c["weights"][b, :, :t].double()
        err = (new[b, :, :t].double() - want[b, :, :t]).abs()
        assert (err <= rel * added + (Q * 4 + 2) * 2.0 ** -23 * want[b, :, :t]).all()
        assert torch.equal(new[b, :, end:t], c["weights"][b, :, end:t])


@pytest.mark.parametrize("Q", [1, 20])
def test_tables_far_wider_than_the_contexts(Q):
    check(case(115 + Q, 2, Q, 8, 2, 64, 16, [200, 30], torch.float16, extra_pages=4000), max_len=200)


@pytest.mark.parametrize("B,T", [(1, 30000), (2, 9000), (4, 4096), (3, 60)])
def test_weights_by_the_attention_kernel_or_apart(B, T):
    """Cluster plans with long and short partitions, and one pass."""
    check(case(120 + T, B, 1, 8, 2, 128, 16, [T - 100 * b if T > 1000 else T - b for b in range(B)],
               torch.bfloat16))
