"""GPU tests of pa.evict_kv against the plain definition: everything is a
copy or a whole number, so every comparison is exact."""
import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(seed, B, Hkv, D, bs, dtype, lens, budget, ties=0.2, width=0):
    g = torch.Generator().manual_seed(seed)
    table, first = ref.tables(lens, bs, seed, width=width)
    new_table, pool = ref.tables([budget] * B, bs, seed + 1, first=first)
    w = torch.exp(1.5 * torch.randn((B, Hkv, table.shape[1] * bs), generator=g))
    w[torch.rand(w.shape, generator=g) < ties] = 0.25
    return dict(table=table, new_table=new_table, weights=w,
                lens=torch.tensor(lens, dtype=torch.int32),
                k_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 2),
                v_cache=ref.normal((pool, bs, Hkv, D), dtype, seed + 3))


def run(c, budget, sink, recent, in_place=False, stream=None):
    d = {k: v.to(DEV) for k, v in c.items()}
    B, Hkv = c["weights"].shape[:2]
    bs = c["k_cache"].shape[1]
    new_table = d["table"] if in_place else d["new_table"]
    new_w = d["weights"] if in_place else torch.full((B, Hkv, new_table.shape[1] * bs),
                                                     float("nan"), device=DEV)
    kept = torch.full((B, Hkv, budget), 77, dtype=torch.int32, device=DEV)
    new_lens = torch.full((B,), 77, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    pa.evict_kv(d["k_cache"], d["v_cache"], d["weights"], d["table"], d["lens"], new_table, new_w,
                new_lens, kept, sink=sink, recent=recent, stream=stream)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return d["k_cache"].cpu(), d["v_cache"].cpu(), new_w.cpu(), new_lens.cpu(), kept.cpu()


def same(got, want):
    for name, g, w in zip(("k_cache", "v_cache", "new_weights", "new_lens", "kept"), got, want):
        assert torch.equal(torch.nan_to_num(g.float(), 99.0), torch.nan_to_num(w.float(), 99.0)), name


def check(c, budget, sink, recent, in_place):
    want = ref.evict(c["k_cache"], c["v_cache"], c["weights"], c["table"], c["lens"],
                     c["table"] if in_place else c["new_table"], budget, sink, recent)
    same(run(c, budget, sink, recent, in_place), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,Hkv,D,bs,lens,budget,sink,recent", [
    (1, 1, 64, 16, [1], 1, 0, 0),
    (1, 2, 64, 16, [40], 1, 0, 1),
    (3, 8, 128, 16, [0, 1, 200], 64, 4, 16),
    (2, 1, 256, 32, [333, 64], 65, 0, 0),
    (2, 4, 128, 32, [100, 257], 100, 50, 50),
    (4, 2, 128, 16, [300, 17, 1025, 600], 130, 3, 0),
    (1, 2, 64, 16, [5000], 2049, 4, 1000),
])
def test_matches_definition(B, Hkv, D, bs, lens, budget, sink, recent, in_place):
    dtype = torch.bfloat16 if B % 2 else torch.float16
    width = (budget + bs - 1) // bs
    check(case(B + budget, B, Hkv, D, bs, dtype, lens, budget, width=width), budget, sink, recent,
          in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_weights_of_every_kind(in_place):
    """All equal; zeros of both signs; infinities and NaN; negative; the type's ends."""
    c = case(11, 6, 2, 64, 16, torch.float16, [90] * 6, 20, ties=0.0, width=2)
    inf, big = float("inf"), torch.finfo(torch.float32).max
    c["weights"][0] = 1.5
    c["weights"][1] = 0.0
    c["weights"][1, :, ::3] = -0.0
    c["weights"][2, :, ::4] = float("nan")
    c["weights"][2, :, 1::4] = inf
    c["weights"][3, :, ::2] = -inf
    c["weights"][3, :, 1::2] = float("nan")
    c["weights"][4].neg_()
    c["weights"][5, :, ::5] = big
    c["weights"][5, :, 1::5] = 1e-45
    c["weights"][5, :, 2::5] = -big
    check(c, 20, 2, 3, in_place)


def test_masked_pages_are_never_kept():
    c = case(12, 3, 2, 128, 16, torch.bfloat16, [200, 90, 160], 40)
    c["table"][0, 0] = -1                     # a masked sink page
    c["table"][0, 5] = c["k_cache"].shape[0]  # out of range
    c["table"][1, 1:] = -1                    # fewer readable tokens than the budget
    c["table"][2, 9] = -7                     # the latest tokens' page
    check(c, 40, 4, 20, False)


def test_new_entries_that_are_masked_store_nothing():
    c = case(13, 2, 2, 64, 16, torch.bfloat16, [100, 70], 40)
    c["new_table"][0, 1] = -1
    c["new_table"][1, 2] = 1 << 20
    check(c, 40, 0, 8, False)


def test_lengths_past_the_table_and_negative():
    c = case(14, 3, 1, 64, 16, torch.bfloat16, [100, 70, 50], 40)
    c["lens"][0], c["lens"][1] = 1 << 30, -3
    check(c, 40, 1, 8, False)
    check(c, 40, 1, 8, True)


def test_same_result_twice_other_stream_and_graph():
    c = case(15, 2, 4, 128, 16, torch.bfloat16, [3000, 1500], 700)
    want = run(c, 700, 4, 64)
    same(run(c, 700, 4, 64, stream=torch.cuda.Stream(DEV)), want)
    d = {k: v.to(DEV) for k, v in c.items()}
    new_w = torch.zeros((2, 4, d["new_table"].shape[1] * 16), device=DEV)
    kept = torch.zeros((2, 4, 700), dtype=torch.int32, device=DEV)
    lens = torch.zeros((2,), dtype=torch.int32, device=DEV)
    args = (d["k_cache"], d["v_cache"], d["weights"], d["table"], d["lens"], d["new_table"], new_w,
            lens, kept, 4, 64)
    pa.evict_kv(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.evict_kv(*args)
    for t in (new_w, kept, lens):
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    same((d["k_cache"].cpu(), d["v_cache"].cpu(), new_w.cpu(), lens.cpu(), kept.cpu()), want)


def test_attention_over_what_is_kept():
    """A budget that holds everything changes no attention output, in place or moved."""
    c = case(16, 2, 2, 128, 16, torch.float16, [77, 64], 80, width=5)
    d = {k: v.to(DEV) for k, v in c.items()}
    q = ref.normal((2, 8, 128), torch.float16, 3).to(DEV)
    before = pa.decode(torch.zeros((2, 8, 128), device=DEV), q, d["k_cache"], d["v_cache"],
                       d["table"], d["lens"], 0.09)
    new_w = torch.zeros((2, 2, d["new_table"].shape[1] * 16), device=DEV)
    kept = torch.zeros((2, 2, 80), dtype=torch.int32, device=DEV)
    lens = torch.zeros((2,), dtype=torch.int32, device=DEV)
    pa.evict_kv(d["k_cache"], d["v_cache"], d["weights"], d["table"], d["lens"], d["new_table"],
                new_w, lens, kept)
    after = pa.decode(torch.zeros((2, 8, 128), device=DEV), q, d["k_cache"], d["v_cache"],
                      d["new_table"], lens, 0.09)
    assert torch.equal(lens, d["lens"]) and torch.equal(before, after)


@pytest.mark.parametrize("T,kind", [(9000, "distinct"), (70000, "distinct"), (70000, "ties"),
                                    (70000, "equal"), (70000, "one digit"), (320000, "ties"),
                                    (320000, "equal")])
def test_rows_that_several_ctas_share(T, kind):
    """Long rows: a cluster of CTAs, lists of candidates that fit and that do not
    (many keys with one first digit), rows too long for the key cache."""
    c = case(20, 1, 1 if T > 100000 else 2, 64, 16, torch.float16, [T - 5], 700,
             ties=0.3 if kind == "ties" else 0.0)
    if kind == "equal":
        c["weights"].fill_(0.5)
    if kind == "one digit":   # 1 .. 1.25: the first eleven bits agree
        c["weights"] = 1 + c["weights"] / c["weights"].max() * 0.24
    check(c, 700, 4, 100, False)


@pytest.mark.parametrize("budget,T", [(513, 3000), (1500, 1501), (9000, 20000)])
def test_in_place_over_several_chunks_and_segments(budget, T):
    """Chunks of 512 rows whose sources the chunks before must not touch; a budget past one segment."""
    c = case(40 + T, 2, 2, 128, 16, torch.bfloat16, [T, T - 7], budget)
    check(c, budget, 3, 11, True)


def test_in_place_keeps_an_untouched_front():
    """Weights that fall with the index: the kept tokens are the first ones and none moves."""
    c = case(50, 1, 2, 64, 16, torch.float16, [2000], 600)
    c["weights"] = torch.arange(c["weights"].numel(), 0, -1).float().reshape(c["weights"].shape)
    check(c, 600, 0, 0, True)
