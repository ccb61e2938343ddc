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
    (128, 1, 16, 8, 900, 70, 200, 20, True),       # launches of their own, warp-level
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
    want = ref.shared_prefix(q, kc, vc, seen_p, plens, seen_own, lens, scale)
    out = torch.empty(q.shape, device=DEV)
    args = [t.to(DEV) for t in (q, kc, vc, ptable, plens, table, lens)]
    need = pa.workspace_size_shared_prefix(args[0], args[1], args[3], args[5], out.dtype, max_p, max_own)
    assert (need > 0) == apart
    pa.decode_shared_prefix(out, *args, scale, max_p, max_own)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    ref.close_out(out.cpu(), want, ref.out_slack(q, kc, vc, scale, plen + own + 5))
