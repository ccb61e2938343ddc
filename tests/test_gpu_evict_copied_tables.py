"""GPU tests of pa.evict_kv with new tables that name old pages at their own
places: a copy of the old table, of its first columns, and mixtures with other
pages.  Everything is a copy or a whole number: exact."""
import pytest
import torch

from test_gpu_evict import case, check

pytestmark = pytest.mark.gpu

SHAPES = [
    # B, Hkv, D, bs, lens, budget, sink, recent
    (1, 2, 64, 16, [200], 100, 2, 10),
    (3, 8, 128, 16, [0, 1, 700], 333, 4, 16),
    (2, 1, 256, 32, [900, 64], 257, 0, 0),
    (4, 2, 128, 16, [3000, 17, 1025, 2600], 1030, 3, 100),
    (1, 4, 128, 32, [6000], 5000, 0, 0),
]


@pytest.mark.parametrize("columns", ["all", "first"])
@pytest.mark.parametrize("args", SHAPES)
def test_copies_of_the_table(args, columns):
    B, Hkv, D, bs, lens, budget, sink, recent = args
    c = case(B + budget, B, Hkv, D, bs, torch.bfloat16 if B % 2 else torch.float16, lens, budget,
             width=(budget + bs - 1) // bs)
    width = c["table"].shape[1] if columns == "all" else (budget + bs - 1) // bs
    c["new_table"] = c["table"][:, :width].clone()
    check(c, budget, sink, recent, False)


@pytest.mark.parametrize("keep", [1, 3, 20])
def test_some_pages_kept_and_others_new(keep):
    """The first `keep` pages stay, or the others do."""
    B, Hkv, D, bs, lens, budget = 2, 2, 128, 16, [900, 1500], 500
    c = case(5, B, Hkv, D, bs, torch.float16, lens, budget)
    fresh = c["new_table"].clone()
    c["new_table"][:, :keep] = c["table"][:, :keep]
    check(c, budget, 2, 30, False)
    c["new_table"] = torch.cat([fresh[:, :keep], c["table"][:, keep:fresh.shape[1]]], 1)
    check(c, budget, 2, 30, False)


def test_one_sequence_of_a_batch_on_its_own_pages():
    B, Hkv, D, bs, lens, budget = 4, 2, 64, 16, [700, 800, 900, 90], 300
    c = case(6, B, Hkv, D, bs, torch.bfloat16, lens, budget)
    c["new_table"][1] = c["table"][1, :c["new_table"].shape[1]]
    c["new_table"][2, 4] = -1                     # and a masked entry in another
    check(c, budget, 4, 64, False)
