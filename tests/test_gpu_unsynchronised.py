"""GPU tests of the serving-step operators in a loop that never waits for the
device: queries, lengths, tables and weights are rewritten by kernels between
the calls, and every call's results must be those of the same call made alone."""
import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TURNS = 24


def rotary(D):
    inv_freq = 1e4 ** (-torch.arange(D // 2).double() * 2 / D)
    return pa.rope_phases(inv_freq).to(DEV), torch.zeros(D // 2, dtype=torch.int32, device=DEV)


def variants(count, B, H, Hkv, D, bs, longest, dtype, first, Q=1):
    """Several states of one batch: tables (rows of the same pages in another
    order), lengths and new tokens."""
    g = torch.Generator().manual_seed(B * 1000 + longest)
    width = (longest + bs - 1) // bs
    pages = torch.arange(B * width, dtype=torch.int32) + first
    out = []
    for i in range(count):
        lens = torch.randint(max(Q, longest // 2), longest + 1, (B,), generator=g).to(torch.int32)
        lens[i % B] = longest
        out.append(dict(table=pages[torch.randperm(len(pages), generator=g)].reshape(B, width).to(DEV),
                        lens=lens.to(DEV), pos=(lens - 1).view(1, B, 1).repeat(1, 1, Q).contiguous().to(DEV),
                        qkv=ref.normal((B, Q, H + 2 * Hkv, D), dtype, 7 * i + 1).to(DEV)))
    return out, first + B * width


@pytest.mark.parametrize("B,H,Hkv,D,longest", [(1, 8, 2, 64, 30000), (40, 8, 2, 64, 3000),
                                               (3, 8, 2, 128, 9000)])
def test_accumulate_in_partitions(B, H, Hkv, D, longest):
    bs, dtype = 16, torch.bfloat16
    vs, pool = variants(4, B, H, Hkv, D, bs, longest, dtype, 0)
    phases, axes = rotary(D)
    k0, v0 = (ref.normal((pool, bs, Hkv, D), dtype, s).to(DEV) for s in (91, 92))
    width = vs[0]["table"].shape[1] * bs
    w0 = torch.rand((B, Hkv, width), device=DEV)
    kc, vc, weights = k0.clone(), v0.clone(), w0.clone()
    state = {n: torch.empty_like(vs[0][n]) for n in ("table", "lens", "pos", "qkv")}
    q, out = (torch.empty((B, 1, H, D), dtype=dtype, device=DEV) for _ in range(2))
    need = pa.workspace_size_accumulate(q, kc, state["table"], dtype, longest)
    ws = torch.full((need // 4 + 1,), float("nan"), device=DEV)

    def turn(i):
        for n, t in state.items():
            t.copy_(vs[i % len(vs)][n])
        qkv = state["qkv"]
        pa.rope_append_kv(q, kc, vc, qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:],
                          state["pos"], phases, axes, state["table"], state["lens"])
        weights.mul_(0.5)
        pa.decode_accumulate(out, weights, q, kc, vc, state["table"], state["lens"], D ** -0.5,
                             longest, workspace=ws)
        return out.clone(), weights.clone()

    alone = []
    for i in range(TURNS):
        alone.append(turn(i))
        torch.cuda.synchronize()
    for c, c0 in ((kc, k0), (vc, v0), (weights, w0)):
        c.copy_(c0)
    ws.fill_(float("nan"))
    torch.cuda.synchronize()
    together = [turn(i) for i in range(TURNS)]
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for a, b in zip(alone, together):
        assert torch.isfinite(a[0].float()).all()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
