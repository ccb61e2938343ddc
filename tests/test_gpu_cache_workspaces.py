"""GPU tests: one workspace, sized for the largest batch and the longest context,
serves every smaller batch and shorter announced length of the attentions over the
8-bit and the latent cache, whatever plan each takes."""
import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def batches(most):
    """The largest, ones around it, and some of every size below."""
    sizes = {most, most - 1, max(1, most // 2), max(1, most // 3), 1, 2, 3, 5, 7}
    k = 1
    while k < most:
        sizes.update((k, k + 1))
        k = k * 5 // 4 + 1
    return sorted((b for b in sizes if 1 <= b <= most), reverse=True)


@pytest.mark.parametrize("most,Q,H,Hkv,D,bs,T", [
    (600, 1, 4, 4, 64, 16, 1700),       # past 3 units a slot, down through runs to clusters
    (2200, 1, 1, 1, 64, 32, 1700),      # past the lengths that a CTA looks through
    (40, 1, 8, 8, 128, 16, 9000),
    (70, 5, 16, 8, 128, 16, 3000),
    (20, 40, 8, 1, 256, 32, 2000),
])
def test_8_bit_attention_of_shrinking_batches(most, Q, H, Hkv, D, bs, T):
    pages = (T + bs - 1) // bs
    kc, ks = cref.cache8(pages, bs, Hkv, D, 1)
    vc, vs = cref.cache8(pages, bs, Hkv, D, 2)
    kc, ks, vc, vs = (x.to(DEV) for x in (kc, ks, vc, vs))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table = table.expand(most, pages).contiguous().to(DEV)
    q = ref.normal((1, Q, H, D), torch.bfloat16, 4).expand(most, Q, H, D).contiguous().to(DEV)
    lens = torch.full((most,), T, dtype=torch.int32, device=DEV)
    scale = D ** -0.5
    # what one sequence gives, in fp32, by whatever plan it takes
    want = torch.empty((1, Q, H, D), device=DEV)
    pa.decode_kv8(want, q[:1], kc, vc, ks, vs, table[:1], lens[:1], scale, T)
    # both sides off by what their sums, exponentials and weights in two parts round
    k, v = cref.values8(kc.cpu(), ks.cpu()), cref.values8(vc.cpu(), vs.cpu())
    slack = 2 * cref.attention_slack(q[:1].cpu(), k, v, scale, T, 2.0 ** -16) + 2.0 ** -22 * 64
    most_bytes = pa.workspace_size_kv8(q, kc, table, torch.float32, T)
    ws = torch.empty(max(most_bytes, 16), dtype=torch.uint8, device=DEV)
    for b in batches(most):
        assert pa.workspace_size_kv8(q[:b], kc, table[:b], torch.float32, T) <= most_bytes
        out = torch.empty((b, Q, H, D), device=DEV)
        pa.decode_kv8(out, q[:b], kc, vc, ks, vs, table[:b], lens[:b], scale, T, workspace=ws)
        assert (out - want).abs().max().item() <= slack, b
    for t in (T - 1, T // 2, 900, 40, 0):
        short = lens.clamp(max=t)
        assert pa.workspace_size_kv8(q, kc, table, torch.float32, t) <= most_bytes
        out = torch.empty((most, Q, H, D), device=DEV)
        pa.decode_kv8(out, q, kc, vc, ks, vs, table, short, scale, t, workspace=ws)
    torch.cuda.synchronize()
    assert pa.device_error() == 0


@pytest.mark.parametrize("most,Q,H,R,bs,T", [(2200, 1, 3, 128, 16, 300), (90, 1, 16, 512, 64, 700),
                                             (20, 2, 128, 256, 32, 900)])
def test_latent_attention_of_shrinking_batches(most, Q, H, R, bs, T):
    pages = (T + bs - 1) // bs
    cache = ref.normal((pages, bs, R + 64), torch.float16, 1).to(DEV)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table = table.expand(most, pages).contiguous().to(DEV)
    q = ref.normal((1, Q, H, R + 64), torch.float16, 4).expand(most, Q, H, R + 64).contiguous().to(DEV)
    lens = torch.full((most,), T, dtype=torch.int32, device=DEV)
    want = torch.empty((1, Q, H, R), dtype=torch.float16, device=DEV)
    pa.decode_latent(want, q[:1], cache, table[:1], lens[:1], 0.1, T)
    # both sides off by what their sums, exponentials and weights round, and by their own rounding
    c = cache.cpu().double().unsqueeze(2)
    slack = 2 * cref.attention_slack(q[:1].cpu(), c, c[..., :R], 0.1, T, 2.0 ** -11)
    most_bytes = pa.workspace_size_latent(q, cache, R, table, T)
    ws = torch.empty(max(most_bytes, 16), dtype=torch.uint8, device=DEV)
    for b in batches(most):
        assert pa.workspace_size_latent(q[:b], cache, R, table[:b], T) <= most_bytes
        out = torch.empty((b, Q, H, R), dtype=torch.float16, device=DEV)
        pa.decode_latent(out, q[:b], cache, table[:b], lens[:b], 0.1, T, workspace=ws)
        off = (out.double() - want.double()).abs() - 2 * 2.0 ** -11 * want.double().abs()
        assert off.max().item() <= slack, b
    for t in (T - 1, T // 2, 40, 0):
        assert pa.workspace_size_latent(q, cache, R, table, t) <= most_bytes
        out = torch.empty((most, Q, H, R), dtype=torch.float16, device=DEV)
        pa.decode_latent(out, q, cache, table, lens.clamp(max=t), 0.1, t, workspace=ws)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
