"""GPU tests of pa.decode_shared_prefix with lengths past those announced, and
with announced lengths far past the tables."""
import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,Q,H,Hkv,plen,own,max_p,max_own,apart", [
    (4, 1, 8, 2, 900, 40, 200, 64, False),         # one launch, a cluster
    (4, 1, 8, 2, 900, 70, 200, 20, False),
    (4, 3, 8, 2, 900, 70, 200, 20, False),
    (60, 1, 32, 8, 120, 40, 30, 20, False),        # one launch, one pass
    (2, 5, 4, 2, 300, 300, 512, 100, False),
    (160, 1, 16, 8, 900, 70, 200, 20, True),       # launches of their own, warp-level
    (5, 5, 8, 2, 900, 400, 200, 100, True),        # the tile kernel
    (140, 1, 32, 8, 3000, 90, 2500, 33, True),     # two tiles to a CTA
])
def test_each_part_loses_its_own_tail(n, Q, H, Hkv, plen, own, max_p, max_own, apart, dtype):
    """Tokens past the announced prefix's pages are left out of the prefix, and those
    past the announced context's pages of the sequence's own; by every plan."""
    D, bs, scale = 128, 16, 0.1
    ptable, first = ref.tables([plen], bs, 1)
    lens = [own + b % 5 for b in range(n)]
    lens[0] = 1                                # (shorter than its query tokens, if several)
    table, pool = ref.tables(lens, bs, 2, first=first)
    q, kc, vc = (ref.normal(s, dtype, 3 + i) for i, s in enumerate(
        ((n, Q, H, D), (pool, bs, Hkv, D), (pool, bs, Hkv, D))))
    plens, lens = torch.tensor([plen], dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    pages = lambda t: (t + bs - 1) // bs
    seen_p, seen_own = ptable.clone(), table.clone()   # the same tokens, left out by their pages
    seen_p[:, pages(max_p):] = -1
    seen_own[:, pages(max_own):] = -1
    some = sorted({0, 1, 2, 3, 4, n // 2, n - 2, n - 1} & set(range(n)))
    want = ref.shared_prefix(q[some], kc, vc, seen_p, plens, seen_own[some], lens[some], scale)
    out = torch.empty(q.shape, device=DEV)
    args = [t.to(DEV) for t in (q, kc, vc, ptable, plens, table, lens)]
    need = pa.workspace_size_shared_prefix(args[0], args[1], args[3], args[5], out.dtype, max_p, max_own)
    assert (need > 0) == apart
    pa.decode_shared_prefix(out, *args, scale, max_p, max_own)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    assert torch.isfinite(out).all()
    ref.close_out(out.cpu()[some], want, ref.out_slack(q, kc, vc, scale, plen + own + 5))


def plan_parts(n, H, Hkv, D, bs, width, max_p, max_own):
    """Partitions of the prefix and of the own pages together (a record of each
    row and partition in the workspace: D + 2 floats)."""
    q = torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV)
    kc = torch.empty((4, bs, Hkv, D), dtype=torch.bfloat16, device=DEV)
    ptable = torch.empty((1, (max_p + bs - 1) // bs), dtype=torch.int32, device=DEV)
    table = torch.empty((n, width // bs), dtype=torch.int32, device=DEV)
    need = pa.workspace_size_shared_prefix(q, kc, ptable, table, torch.bfloat16, max_p, max_own)
    return need // (n * H * (D + 2) * 4)


def test_the_plan_goes_by_the_tables_reach():
    a = plan_parts(128, 32, 8, 128, 16, 2048, 65536, 2048)
    assert a > 4 and plan_parts(128, 32, 8, 128, 16, 2048, 65536, 1 << 30) == a


def test_a_loose_bound_does_not_serialise_the_prefix():
    """Own tables of 131,072 tokens, announced in full: 64 partitions of the own pages,
    and the prefix still in more than one (all of it by 16 CTAs took 1.5 ms)."""
    assert plan_parts(128, 32, 8, 128, 16, 131072, 65536, 131072) >= 64 + 3
