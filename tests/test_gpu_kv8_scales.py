"""GPU tests of pa.decode_kv8 over pages whose value scales lie far apart: a page
of small values, or of none, keeps its tokens' share of the softmax's normaliser,
whatever the output's type, the plan and the order of the pages."""
import math

import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def definition(q, kc, vc, ks, vs, table, lens, scale):
    """(output, mean |value| under the weights, largest weight times value scale) in
    float64, one query token a sequence."""
    B, _, H, D = q.shape
    bs, Hkv = kc.shape[1], kc.shape[2]
    G = H // Hkv
    k, v = cref.values8(kc, ks), cref.values8(vc, vs)
    s = vs.double().view(-1, 1, Hkv, 1).expand(-1, bs, Hkv, 1).contiguous()
    want, mean, top = (torch.zeros(B, 1, H, D).double() for _ in range(3))
    for b in range(B):
        for h in range(Hkv):
            n = int(lens[b])
            rows = [ref._rows(x, table[b], n, h)[0] for x in (k, v, s)]
            heads = slice(h * G, (h + 1) * G)
            p = torch.softmax(q[b, 0, heads].double() @ rows[0].T * scale, 1)
            want[b, 0, heads] = p @ rows[1]
            mean[b, 0, heads] = p @ rows[1].abs()
            top[b, 0, heads] = (p * rows[2].T).amax(1, keepdim=True)
    return want, mean, top


def check(q, kc, vc, ks, vs, table, lens, scale, out_dtype, expect_runs=None):
    """Runs the call and holds its output against the definition, element by element:
    each weight's relative error and its exponent's (which holds the score and the
    scale's logarithm, up to 2^7 in all, three times rounded), in numerator and
    normaliser; a weight's own rounding to fp16 (in two parts for fp32 outputs); a
    weight below fp16's normal numbers rounds by 2^-25, where the row's largest
    weight times scale stands at 2^7 or higher; then the output's rounding."""
    want, mean, top = definition(q, kc, vc, ks, vs, table, lens, scale)
    tokens = int(lens.max())
    held = table[table >= 0].long()
    k = cref.values8(kc, ks)[held]
    d = [x.to(DEV) for x in (q, kc, vc, ks, vs, table, lens)]
    out = torch.full(q.shape, math.nan, dtype=out_dtype, device=DEV)
    need = pa.workspace_size_kv8(d[0], d[1], d[5], out_dtype, tokens)
    if expect_runs is not None:
        assert (need > 0) == expect_runs
    ws = torch.full((need // 4 + 4,), math.nan, device=DEV)
    pa.decode_kv8(out, *d, scale, tokens, workspace=ws)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    got = out.cpu().double()
    # two more products a score: the page's scale and the query's power of two
    two = 2 * 2.0 ** -23 * 0.6932 * 1.4427 * scale * \
        (q.double().norm(dim=-1).max() * k.norm(dim=-1).max()).item()
    one = ref.weight_slack(q, k, scale, tokens) + 2 * two + 3 * 0.6932 * 2.0 ** -17
    part = 2.0 ** -11 if out_dtype != torch.float32 else 2.0 ** -16
    bound = (2 * one + part) * mean + tokens * 2.0 ** -32 * 448 * top
    tiny = torch.finfo(out_dtype).tiny * torch.finfo(out_dtype).eps / 2
    bound += torch.finfo(out_dtype).eps / 2 * (want.abs() + bound) + tiny
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert over.max().item() <= 0, (over.max().item(), want.flatten()[over.argmax()].item(),
                                    got.flatten()[over.argmax()].item())


def uneven(seed, exponents, B, H, Hkv, D, bs, lens, dtype):
    """A case whose pages' value scales are 2^e, e in turn from `exponents`, codes of
    full range; the scores are ordinary."""
    table, pool = ref.tables(lens, bs, seed)
    kc, ks = cref.cache8(pool, bs, Hkv, D, seed + 1)
    vc, vs = cref.cache8(pool, bs, Hkv, D, seed + 2)
    vs = torch.empty(pool, Hkv)
    for b, row in enumerate(table):
        for j, e in enumerate(row[row >= 0].tolist()):
            for h in range(Hkv):
                vs[e, h] = 2.0 ** exponents[(j + h + b) % len(exponents)]
    return (ref.normal((B, 1, H, D), dtype, seed + 3), kc, vc, ks, vs, table,
            torch.tensor(lens, dtype=torch.int32), D ** -0.5)


OUTS = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
        (torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("B,H,Hkv,D,bs,lens", [
    (2, 8, 2, 128, 16, [600, 77]),
    (2, 8, 2, 128, 32, [601, 64]),
    (1, 4, 1, 64, 16, [9000]),
    (1, 16, 1, 256, 16, [3001]),
    (30, 8, 8, 64, 16, [17 * (b % 7) + 30 for b in range(30)]),
])
@pytest.mark.parametrize("exponents", [(0, -8, -16, -24, -31, -38), (-60, -60, -60, 4)])
def test_pages_of_uneven_value_scales(exponents, B, H, Hkv, D, bs, lens, dtype, out_dtype):
    check(*uneven(B + D + bs, exponents, B, H, Hkv, D, bs, lens, dtype), out_dtype)


@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("B,H,Hkv,D,bs,T,runs", [
    (30, 8, 8, 64, 16, 64, False),     # a unit to a CTA
    (30, 8, 8, 64, 32, 64, False),
    (2, 4, 2, 128, 16, 320, False),     # clusters
    (2, 4, 2, 128, 32, 320, False),
    (1, 4, 1, 128, 16, 9024, True),     # runs
    (1, 4, 1, 256, 32, 9024, True),
])
@pytest.mark.parametrize("where", ["before", "beside", "after"])
@pytest.mark.parametrize("lead", [0, 10])
def test_appended_pages_of_zero_values(lead, where, B, H, Hkv, D, bs, T, runs, dtype, out_dtype):
    """Pages of all-zero values, as the append writes them, before, between (with 16
    tokens to a page in one step of 32) and after the others, with the others' score
    or 2^10 their weight."""
    pages = T // bs
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(T)).view(B, pages)
    table = table.to(torch.int32)
    zero = {"before": torch.arange(pages) < pages // 2, "beside": torch.arange(pages) % 2 == 0,
            "after": torch.arange(pages) >= pages // 2}[where].repeat_interleave(bs)
    v = ref.normal((B, T, Hkv, D), dtype, T + 1)
    v = torch.where(zero.view(1, T, 1, 1), torch.zeros((), dtype=dtype), 1 + v.abs())
    k = zero.to(dtype).view(1, T, 1, 1).expand(B, T, Hkv, D).contiguous()
    lens = torch.full((B,), T, dtype=torch.int32)
    NB = B * pages
    kc, vc = (torch.full((NB, bs, Hkv, D), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3)
              for _ in range(2))
    ks, vs = (torch.full((NB, Hkv), math.nan, device=DEV) for _ in range(2))
    q0 = torch.zeros(B, T, H, D, dtype=dtype, device=DEV)
    pa.rope_append_kv8(q0, kc, vc, ks, vs, q0, k.to(DEV), v.to(DEV),
                       torch.zeros(1, B, T, dtype=torch.int32, device=DEV),
                       pa.rope_phases(torch.zeros(8, dtype=torch.float64, device=DEV)),
                       torch.zeros(8, dtype=torch.int32, device=DEV), table.to(DEV), lens.to(DEV))
    torch.cuda.synchronize()
    held = table[:, zero.view(pages, bs)[:, 0]].flatten().long()
    assert (vs.cpu()[held] == 2.0 ** -60).all()
    # q . k is 0 or D
    scale = (lead or 1) / (1.4426950408889634 * D)
    q = torch.full((B, 1, H, D), 1.0 if lead else 0.0, dtype=dtype)
    check(q, kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), table, lens, scale, out_dtype, expect_runs=runs)


@pytest.mark.parametrize("dtype,tiny", [(torch.bfloat16, -40), (torch.float16, -14)])
def test_weight_on_a_page_of_tiny_values(dtype, tiny):
    q, kc, vc, ks, vs, table, lens, _ = uneven(63, (0,), 1, 4, 1, 64, 16, [64], dtype)
    q = torch.ones_like(q)
    kc.view(torch.uint8)[:] = 0
    kc[int(table[0, 2])] = torch.full((16, 1, 64), 8.0).to(E4M3)   # score 512 above
    ks[:] = 1.0
    vs[int(table[0, 2])] = 2.0 ** tiny
    check(q, kc, vc, ks, vs, table, lens, 1.0, dtype)


@pytest.mark.parametrize("dtype,exponent", [(torch.bfloat16, -60), (torch.bfloat16, 60),
                                            (torch.float16, -24), (torch.float16, 6)])
def test_scales_far_from_one(dtype, exponent):
    check(*uneven(65, (exponent,), 1, 4, 1, 128, 16, [200], dtype), dtype)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,Hkv,D,bs,T,runs,drop", [
    (30, 8, 8, 64, 16, 256, False, 8),     # a unit to a CTA: warps of tiny pages only
    (30, 16, 8, 64, 32, 512, False, 8),
    (2, 4, 2, 128, 16, 1024, False, 10),    # clusters
    (1, 4, 1, 256, 32, 2048, False, 11),
    (1, 4, 1, 128, 16, 9024, True, 13),     # runs
    (1, 4, 1, 128, 32, 9024, True, 14),
    (1, 4, 1, 64, 16, 9024, True, 15),      # tiny pages beside the large one: under 2^-126 of it
])
@pytest.mark.parametrize("at", [0, 3, -1])
def test_scales_at_both_ends_at_once(at, B, H, Hkv, D, bs, T, runs, drop, out_dtype):
    """One page of values on the scale 2^60, the others on 2^-60 with scores `drop`
    binary orders lower: their values are nothing beside the large ones, their number
    is a visible share of the normaliser.  Weights times scales lie past fp32's range."""
    pages = T // bs
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(T)).view(B, pages)
    table = table.to(torch.int32)
    big = table[:, at].long()
    kc, vc = (torch.zeros(B * pages, bs, Hkv, D).to(E4M3) for _ in range(2))
    raw = torch.randint(0x58, 0x7e, vc.shape, generator=torch.Generator().manual_seed(T + 1),
                        dtype=torch.uint8)              # 16 .. 416
    vc.view(torch.uint8)[:] = raw
    kc[big] = torch.ones(1).to(E4M3)
    ks, vs = torch.ones(B * pages, Hkv), torch.full((B * pages, Hkv), 2.0 ** -60)
    vs[big] = 2.0 ** 60
    q = torch.ones(B, 1, H, D, dtype=torch.bfloat16)
    check(q, kc, vc, ks, vs, table, torch.full((B,), T, dtype=torch.int32),
          drop / (1.4426950408889634 * D), out_dtype, expect_runs=runs)
