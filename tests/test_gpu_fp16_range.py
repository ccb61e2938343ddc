"""GPU tests of fp16 attention weights far below the row's largest, which the
kernels hold in fp16 (in one part or two) for the product with V: tokens of no
value (a sink) that outweigh the others by 20 to 26 bits, so that the output
is made of weights near the end of fp16's range."""
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SINK = 64     # every 64th token is one: each half of a block has one


def sunk(q, k_cache, v_cache, tables, lens, bits, scale):
    """Makes every SINK-th token of these sequences a sink of `bits` bits."""
    q[..., 0] = 8
    k_cache[..., 0] = 0
    v_cache.copy_(1 + v_cache.float() / 4)
    for row, t in zip(tables, lens):
        for at in range(0, int(t), SINK):
            e, s = ref.slot(row, at, k_cache.shape[1], len(k_cache))
            k_cache[e, s] = 0
            k_cache[e, s, :, 0] = bits / (8 * scale * math.log2(math.e))
            v_cache[e, s] = 0


def some_of(n):
    return sorted({0, 1, 2, n // 2, n - 1} & set(range(n)))


def checked(got, q, groups, scale, rel):
    """groups[b][h]: keys and values of a sequence's kv head, all of its rows' tokens.
    Bound of a row's output: each weight p_t is off by rel (its score, the
    exponentials, the sums) and by its rounding to fp16, 2^-11, or where it is
    below fp16's normal range by half of 2^-24: at least 2^7 stands for the row's
    largest weight, so 2^-32 of that.  Numerator and normaliser both."""
    B, Q, H, D = q.shape
    Hkv = len(groups[0])
    G = H // Hkv
    worst = 0.0
    for b in range(B):
        for h in range(Hkv):
            k, v, seen = groups[b][h]
            x = q[b, :, h * G:(h + 1) * G].double().reshape(Q * G, D) @ k.T * scale
            p = torch.softmax(x.masked_fill(~seen, -math.inf), 1)
            want = p @ v
            off = 2 * (rel + 2.0 ** -11) * p + 2.0 ** -32 * p.amax(1, keepdim=True) * seen
            bound = off @ v.abs() + want.abs() * (2.0 ** -32 * seen.sum(1, keepdim=True) + 2.0 ** -23)
            err = (got[b, :, h * G:(h + 1) * G].double().reshape(Q * G, D) - want).abs()
            worst = max(worst, (err / bound).max().item())
    assert worst <= 1, f"{worst:.3g} times the bound"


@pytest.mark.parametrize("bits", [20, 22, 24, 26])
@pytest.mark.parametrize("n,Q,H,Hkv,D,bs,plen,own,announced", [
    (40, 1, 32, 8, 128, 16, 2000, 3, 65536),       # two tiles to a CTA
    (40, 1, 32, 8, 64, 32, 1500, 3, 65536),
    (10, 1, 32, 8, 128, 16, 2000, 3, 1 << 20),     # the tile kernel
    (9, 2, 16, 1, 256, 32, 1500, 30, 1 << 20),
    (3, 40, 8, 2, 128, 16, 300, 900, 1 << 20),     # the own rows on the tile kernel
    (2, 80, 16, 4, 64, 16, 300, 900, 1 << 20),     # or two tiles to a CTA (wide own tables)
    (4, 1, 32, 8, 128, 16, 1500, 40, 1500),        # the warp-level kernel: one launch
    (3, 3, 8, 2, 64, 32, 700, 90, 700),
    (2, 1, 8, 1, 256, 16, 900, 30, 900),
    (3, 1, 8, 2, 128, 16, 900, 500, 1 << 20),      # launches of their own
    (2, 2, 4, 4, 64, 16, 900, 500, 1 << 20),
])
def test_shared_prefix(n, Q, H, Hkv, D, bs, plen, own, announced, bits):
    dtype, scale = torch.float16, D ** -0.5
    ptable, first = ref.tables([plen], bs, 1)
    lens = [own + Q + b % 3 for b in range(n)]
    table, pool = ref.tables(lens, bs, 2, first=first)
    q, kc, vc = (ref.normal(s, dtype, 3 + i) for i, s in enumerate(
        ((n, Q, H, D), (pool, bs, Hkv, D), (pool, bs, Hkv, D))))
    sunk(q, kc, vc, list(ptable) + list(table), [plen] + lens, bits, scale)
    ends = plen + torch.tensor(lens).view(n, 1) - Q + 1 + torch.arange(Q)
    groups = []
    for b in some_of(n):
        groups.append([])
        for h in range(Hkv):
            parts = [(ref._rows(c, ptable[0], plen, h)[0], ref._rows(c, table[b], lens[b], h)[0])
                     for c in (kc, vc)]
            seen = torch.arange(plen + lens[b]) < ends[b].repeat_interleave(H // Hkv)[:, None]
            groups[-1].append((torch.cat(parts[0]), torch.cat(parts[1]), seen))
    wide = torch.full((1, (announced + bs - 1) // bs), -1, dtype=torch.int32)
    wide[:, :ptable.shape[1]] = ptable
    max_own = max(lens)
    if Q == 80:
        max_own, narrow = 65536, table
        table = torch.full((n, max_own // bs), -1, dtype=torch.int32)
        table[:, :narrow.shape[1]] = narrow
    out = torch.empty(q.shape, device=DEV)
    pa.decode_shared_prefix(out, q.to(DEV), kc.to(DEV), vc.to(DEV), wide.to(DEV),
                            torch.tensor([plen], dtype=torch.int32, device=DEV), table.to(DEV),
                            torch.tensor(lens, dtype=torch.int32, device=DEV), scale, announced, max_own)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    checked(out.cpu()[some_of(n)], q[some_of(n)], groups, scale,
            ref.weight_slack(q, kc, scale, plen + max(lens)))


@pytest.mark.parametrize("bits", [20, 22, 24, 26])
@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,lens", [
    (2, 20, 8, 2, 128, 16, [2000, 700]),
    (2, 33, 8, 2, 64, 32, [40, 1500]),
    (40, 10, 8, 2, 128, 16, [100 + 10 * b for b in range(40)]),    # one pass
    (1, 1, 16, 1, 256, 32, [3000]),                                # a compact tile
    (1, 20, 8, 1, 256, 16, [2500]),
    (1, 1, 32, 8, 128, 16, [1500]),                                # the warp-level kernel
    (3, 3, 8, 2, 64, 32, [900, 40, 300]),
    (70, 1, 8, 2, 64, 16, [200 + b for b in range(70)]),
    (1, 1, 8, 2, 128, 16, [20000]),
])
def test_accumulate(B, Q, H, Hkv, D, bs, lens, bits):
    dtype, scale = torch.float16, D ** -0.5
    table, pool = ref.tables(lens, bs, 11)
    q, kc, vc = (ref.normal(s, dtype, 13 + i) for i, s in enumerate(
        ((B, Q, H, D), (pool, bs, Hkv, D), (pool, bs, Hkv, D))))
    sunk(q, kc, vc, table, lens, bits, scale)
    ends = torch.tensor(lens).view(B, 1) - Q + 1 + torch.arange(Q)
    groups = [[(ref._rows(kc, table[b], lens[b], h)[0], ref._rows(vc, table[b], lens[b], h)[0],
                torch.arange(lens[b]) < ends[b].repeat_interleave(H // Hkv)[:, None])
               for h in range(Hkv)] for b in some_of(B)]
    out = torch.empty(q.shape, device=DEV)
    weights = torch.zeros((B, Hkv, table.shape[1] * bs), device=DEV)
    pa.decode_accumulate(out, weights, q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                         torch.tensor(lens, dtype=torch.int32, device=DEV), scale, max(lens))
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    rel = ref.weight_slack(q, kc, scale, max(lens))
    some = some_of(B)
    checked(out.cpu()[some], q[some], groups, scale, rel)
    want = ref.accumulate(torch.zeros(weights[some].shape), q[some], kc, vc, table[some],
                          torch.tensor(lens, dtype=torch.int32)[some], scale)[1]
    rows = Q * H // Hkv
    assert ((weights.cpu()[some].double() - want).abs() <= (rel + (rows + 2) * 2.0 ** -23) * want).all()
