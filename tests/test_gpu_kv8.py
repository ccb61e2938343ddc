"""GPU tests of the 8-bit cache: pa.rope_append_kv8 and pa.decode_kv8 against
their 64-bit definitions."""
import math

import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def raw(x):
    return x.view(torch.uint8)


# ---- append ----

def append_case(seed, B, Q, H, Hkv, D, bs, rot, axes, lens, dtype, fused=True):
    table, pool = ref.tables([max(t, 0) for t in lens], bs, seed)
    kc, ks = cref.cache8(pool, bs, Hkv, D, seed + 1)
    vc, vs = cref.cache8(pool, bs, Hkv, D, seed + 2)
    qkv = ref.normal((B, Q, H + 2 * Hkv, D), dtype, seed + 3)
    g = torch.Generator().manual_seed(seed + 4)
    pos = torch.randint(0, 1 << 20, (axes, B, Q), generator=g, dtype=torch.int32)
    inv = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return dict(qkv=qkv, k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, pos=pos, inv=inv,
                axis=(torch.arange(rot // 2) % axes).to(torch.int32), table=table,
                lens=torch.tensor(lens, dtype=torch.int32), H=H, Hkv=Hkv)


def check_append(c, interleaved=False, in_place=False, drop=False):
    H, Hkv = c["H"], c["Hkv"]
    q, k, v = (c["qkv"][:, :, :H], c["qkv"][:, :, H:H + Hkv], c["qkv"][:, :, H + Hkv:])
    want = cref.append8(q, c["k_cache"], c["v_cache"], c["k_scales"], c["v_scales"], k, v,
                        c["pos"], c["inv"], c["axis"], c["table"], c["lens"], interleaved)
    d = {n: x.to(DEV) for n, x in c.items() if torch.is_tensor(x)}
    dq, dk, dv = d["qkv"][:, :, :H], d["qkv"][:, :, H:H + Hkv], d["qkv"][:, :, H + Hkv:]
    q_out = dq if in_place else torch.full(q.shape, math.nan, dtype=q.dtype, device=DEV)
    phases = pa.rope_phases(d["inv"])
    args = [q_out, d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], dq, dk, dv, d["pos"]]
    if drop:  # one token a sequence, without the dimension
        args = [x.squeeze(1) if i in (0, 5, 6, 7) else x.squeeze(2) if i == 8 else x
                for i, x in enumerate(args)]
    pa.rope_append_kv8(*args, phases, d["axis"], d["table"], d["lens"], interleaved=interleaved)
    torch.cuda.synchronize()
    # a turned element: two products and a sum in fp32 with a sine and a cosine of 2^-22 each
    # (and an angle off by 2^-31 half turns, pi 2^-31), then one rounding
    half = torch.finfo(q.dtype).eps / 2
    big = 2 * q.double().abs().max().item()
    err = (q_out.cpu().double() - want[0]).abs() - half * want[0].abs() - 2.0 ** -21 * big
    assert err.max().item() <= 0
    for which, (cache, scales) in enumerate((("k_cache", "k_scales"), ("v_cache", "v_scales"))):
        got, got_s = d[cache].cpu(), d[scales].cpu()
        new, old = want[1 + which], raw(c[cache])
        assert torch.equal(got_s, want[3 + which]), scales
        rounded = want[5][which]
        assert torch.equal(raw(got)[~rounded], old[~rounded])
        s = got_s.double().view(got_s.shape[0], 1, -1, 1)
        if which == 1:  # values do not turn: their codes are the rounding itself
            exact = cref.codes_of(new, s)
            assert torch.equal(raw(got)[rounded], raw(exact)[rounded])
        err = (cref.values8(got, got_s) - new).abs()
        # half a step: 2^-4 of the value, 2^-10 scales under 2^-6 of them
        bound = torch.maximum(2.0 ** -4 * new.abs(), 2.0 ** -10 * s) + 2.0 ** -20 * big
        assert (err - bound)[rounded].max().item() <= 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,rot,axes,lens,interleaved", [
    (1, 1, 1, 1, 64, 16, 64, 1, [1], False),
    (3, 1, 8, 2, 128, 16, 128, 1, [100, 17, 16], False),
    (3, 1, 8, 2, 128, 32, 64, 3, [33, 32, 31], True),
    (2, 5, 4, 4, 64, 16, 32, 2, [20, 5], False),
    (2, 70, 8, 1, 256, 32, 256, 1, [200, 70], True),
    (1, 40, 16, 8, 128, 16, 16, 1, [47], False),
    (4, 3, 2, 1, 256, 16, 128, 2, [3, 2, 18, 1000], True),
])
def test_append_matches_definition(B, Q, H, Hkv, D, bs, rot, axes, lens, interleaved, dtype):
    check_append(append_case(B * 10 + Q, B, Q, H, Hkv, D, bs, rot, axes, lens, dtype), interleaved)


def test_append_padding_masked_and_far_entries():
    c = append_case(5, 6, 3, 4, 2, 64, 16, 64, 1, [2, 0, -7, 40, 33, 1], torch.bfloat16)
    c["table"][3, 2] = -1
    c["table"][4, 2] = c["k_cache"].shape[0] + 3
    c["pos"][0, 2] = -(1 << 31)
    check_append(c)
    c["lens"][3] = 1 << 30   # past the table
    check_append(c, in_place=True)


def test_append_raises_scales_and_keeps_older_tokens():
    """A page filled token by token with ever larger values: the scale rises with
    them, and each token stays within half a step of its own rounding plus what
    falls under e4m3's smallest normal number."""
    B, Hkv, D, bs = 1, 2, 64, 16
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    kc, vc = (torch.full((2, bs, Hkv, D), 7, dtype=torch.uint8, device=DEV).view(E4M3)
              for _ in range(2))
    ks, vs = (torch.full((2, Hkv), 3.0, device=DEV) for _ in range(2))
    x = ref.normal((bs, Hkv, D), torch.float32, 9) * 2.0 ** torch.arange(bs).view(bs, 1, 1)
    x = x.to(torch.bfloat16)
    phases = pa.rope_phases(torch.zeros(8, dtype=torch.float64, device=DEV))
    axes = torch.zeros(8, dtype=torch.int32, device=DEV)
    pos = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    want = torch.zeros(bs, Hkv, D).double()
    scale = [0.0] * Hkv
    for t in range(bs):
        new = x[t:t + 1].to(DEV)
        q = torch.zeros(1, Hkv, D, dtype=torch.bfloat16, device=DEV)
        pa.rope_append_kv8(q, kc, vc, ks, vs, q, new, new, pos, phases, axes, table,
                           torch.tensor([t + 1], dtype=torch.int32, device=DEV))
        for h in range(Hkv):
            s = max(scale[h], cref.scale_for(x[t, h].double().abs().max().item()))
            if s > scale[h]:
                want[:t, h] = cref.codes_of(want[:t, h], s).double() * s
            scale[h] = s
            want[t, h] = cref.codes_of(x[t, h], s).double() * s
    torch.cuda.synchronize()
    for cache, scales in ((kc, ks), (vc, vs)):
        assert torch.equal(scales[1].cpu().double(), torch.tensor(scale).double())
        assert torch.equal(cref.values8(cache.cpu(), scales.cpu())[1], want)
        assert (scales[0] == 3).all() and (raw(cache)[0] == 7).all()   # the other page


def test_append_extremes():
    """Zeros, infinities, NaN and the ends of the scales' range."""
    c = append_case(6, 4, 1, 2, 2, 64, 16, 16, 1, [17, 17, 17, 5], torch.bfloat16)
    c["pos"].zero_()
    kv = c["qkv"][:, 0, 2:]
    kv[0] = 0.0
    kv[1, :, 5] = math.inf
    kv[1, :, 6] = math.nan
    kv[2, 0] = 2.0 ** 120
    kv[2, 2] = -2.0 ** -100
    check_finite = append_case(6, 4, 1, 2, 2, 64, 16, 16, 1, [17, 17, 17, 5], torch.bfloat16)
    check_finite["pos"].zero_()
    check_finite["qkv"][0, 0, 2:] = 0.0
    check_append(check_finite, drop=True)
    d = {n: x.to(DEV) for n, x in c.items() if torch.is_tensor(x)}
    q = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    pa.rope_append_kv8(q, d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], q,
                       d["qkv"][:, :, 2:4], d["qkv"][:, :, 4:], d["pos"],
                       pa.rope_phases(d["inv"]), d["axis"], d["table"], d["lens"])
    torch.cuda.synchronize()
    for which, (cache, scales) in enumerate((("k_cache", "k_scales"), ("v_cache", "v_scales"))):
        got, s = d[cache].cpu(), d[scales].cpu()
        for b in range(3):  # a page of their own
            e = int(c["table"][b, 1])
            for h in range(2):
                x = kv[b, 2 * which + h].double()
                if which == 0:  # (an infinite element's partner is inf * sin 0 + y: NaN)
                    x = cref.turned(x[None], torch.zeros(8).double(), False)[0]
                finite = x[torch.isfinite(x)].abs().max().item()
                assert s[e, h].item() == cref.scale_for(finite)
                want = cref.codes_of(x, s[e, h].double())
                have = got[e, 0, h].float()
                assert torch.equal(torch.isnan(have), torch.isnan(want.float()))
                fine = ~torch.isnan(have)
                assert torch.equal(have[fine], want.float()[fine])


# ---- attention ----

def case(seed, B, Q, H, Hkv, D, bs, lens, dtype, spread=0.5):
    table, pool = ref.tables(lens, bs, seed)
    kc, ks = cref.cache8(pool, bs, Hkv, D, seed + 1, spread)
    vc, vs = cref.cache8(pool, bs, Hkv, D, seed + 2, spread)
    return dict(q=ref.normal((B, Q, H, D), dtype, seed + 3), k_cache=kc, v_cache=vc, k_scales=ks,
                v_scales=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32))


def run(c, scale, out_dtype=None, longest=None, stream=None, own_workspace=True, drop=False):
    d = {k: v.to(DEV) for k, v in c.items()}
    if drop:
        d["q"] = d["q"].squeeze(1)
    out = torch.full(d["q"].shape, math.nan, dtype=out_dtype or c["q"].dtype, device=DEV)
    longest = max(0, int(c["lens"].max())) if longest is None else longest
    ws = None
    if own_workspace:
        need = pa.workspace_size_kv8(d["q"], d["k_cache"], d["table"], out.dtype, longest)
        ws = torch.full((need // 4 + 4,), math.nan, device=DEV)
    torch.cuda.synchronize()
    pa.decode_kv8(out, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"],
                  d["table"], d["lens"], scale, longest, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu().reshape(c["q"].shape)


def check(c, scale=None, want_lens=None, **kw):
    D = c["q"].shape[-1]
    scale = scale or 1 / math.sqrt(D)
    k, v = cref.values8(c["k_cache"], c["k_scales"]), cref.values8(c["v_cache"], c["v_scales"])
    lens = c["lens"] if want_lens is None else want_lens
    want = cref.attention(c["q"], k, v, c["table"], lens, scale)
    tokens = max(1, int((c["table"] >= 0).sum(1).max())) * k.shape[1]
    held = c["table"][(c["table"] >= 0) & (c["table"] < len(k))].long()
    got = run(c, scale, **kw)
    ref.close_out(got, want, cref.attention_slack(c["q"], k[held], v[held], scale, tokens, weights(got.dtype)))


def weights(out_dtype):
    """Rounding of a weight on the way to the values: fp32 outputs in two fp16
    parts (2^-22, and under 2^-16 whatever the lift), 16-bit ones once to fp16."""
    return 2.0 ** -16 if out_dtype == torch.float32 else 2.0 ** -11


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,lens", [
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 1, 4, 2, 128, 16, [100]),
    (3, 1, 8, 2, 128, 16, [1, 50, 16]),
    (8, 1, 32, 8, 128, 16, [37 * b + 1 for b in range(8)]),
    (2, 1, 16, 1, 256, 32, [33, 640]),
    (2, 1, 8, 8, 64, 32, [300, 31]),
    (1, 1, 16, 2, 256, 16, [900]),
    (2, 3, 4, 4, 64, 32, [65, 3]),
    (2, 4, 16, 2, 256, 16, [40, 129]),
    (2, 4, 16, 4, 128, 16, [77, 400]),
    (3, 5, 8, 2, 128, 32, [5, 9, 200]),
    (1, 40, 8, 2, 128, 16, [90]),
    (1, 17, 16, 1, 64, 16, [100]),
])
def test_matches_definition(B, Q, H, Hkv, D, bs, lens, dtype):
    check(case(B * 100 + Q, B, Q, H, Hkv, D, bs, lens, dtype))


@pytest.mark.parametrize("T,H,Hkv,D", [(3000, 32, 8, 128), (9000, 8, 1, 128), (5000, 4, 1, 64),
                                       (4100, 16, 1, 256)])
def test_split_contexts(T, H, Hkv, D):
    check(case(T, 1, 1, H, Hkv, D, 16, [T], torch.bfloat16))
    check(case(T + 1, 2, 2, H, Hkv, D, 32, [T, 7], torch.float16), out_dtype=torch.float32)


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float32)])
def test_output_types(dtype, out_dtype):
    check(case(31, 6, 1, 8, 2, 128, 16, [10 * b + 1 for b in range(6)], dtype), out_dtype=out_dtype)
    check(case(32, 6, 1, 8, 2, 128, 16, [10 * b + 1 for b in range(6)], dtype), drop=True)


@pytest.mark.parametrize("Q", [1, 3, 12])
def test_empty_sequences_and_padding(Q):
    lens = [Q, 0, max(0, Q - 2), -4, 50, Q + 1, 0, 1]
    c = case(32 + Q, 8, Q, 8, 2, 128, 16, [max(t, 0) for t in lens], torch.bfloat16)
    c["lens"] = torch.tensor(lens, dtype=torch.int32)
    check(c)


@pytest.mark.parametrize("Q", [1, 6])
def test_masked_pages_and_nan_in_unread_places(Q):
    c = case(40 + Q, 4, Q, 8, 2, 128, 16, [150, 40, 41, 90], torch.bfloat16)
    c["table"][0, 3] = -1
    c["table"][0, 9] = c["k_cache"].shape[0] + 5
    c["table"][1, 1] = -1
    c["table"][2, :] = -1
    used = c["table"].flatten()
    dead = torch.ones(c["k_cache"].shape[0], dtype=torch.bool)
    dead[used[(used >= 0) & (used < len(dead))].unique().long()] = False
    c["lens"][3] = 83                          # ends inside page 5
    for cache, scales in (("k_cache", "k_scales"), ("v_cache", "v_scales")):
        raw(c[cache])[dead] = 0x7f             # NaN
        c[scales][dead] = math.nan
        raw(c[cache])[int(c["table"][3, 5]), 3:] = 0x7f
        raw(c[cache])[int(c["table"][0, 9 - 1]), :] = raw(c[cache])[int(c["table"][0, 0]), :]
    clean = {k: v.clone() for k, v in c.items()}
    for cache, scales in (("k_cache", "k_scales"), ("v_cache", "v_scales")):
        raw(clean[cache])[dead] = 0
        clean[scales][dead] = 1
        raw(clean[cache])[int(c["table"][3, 5]), 3:] = 0
    scale = 128 ** -0.5
    k, v = cref.values8(clean["k_cache"], clean["k_scales"]), cref.values8(clean["v_cache"], clean["v_scales"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], scale)
    ref.close_out(run(c, scale), want,
                  cref.attention_slack(c["q"], k, v, scale, 160, weights(torch.bfloat16)))


def test_lengths_past_the_table_and_past_the_announced():
    c = case(51, 4, 1, 8, 2, 64, 16, [64] * 4, torch.float16)
    c["lens"][2] = 1 << 30
    check(c, longest=64)
    check(c, longest=1 << 30)
    # what lies past the announced length's last page is left out
    check(c, longest=20, want_lens=torch.tensor([32, 32, 32, 32], dtype=torch.int32))
    big = case(52, 1, 1, 8, 1, 128, 16, [6000], torch.bfloat16)
    check(big, longest=3001, want_lens=torch.tensor([3008], dtype=torch.int32))


@pytest.mark.parametrize("spread", [4.0, 12.0])
def test_pages_of_very_different_scales(spread):
    """Pages whose values differ by many powers of two: the small ones count where
    the softmax gives them the weight."""
    c = case(61, 2, 1, 8, 2, 128, 16, [600, 77], torch.bfloat16, spread)
    c["k_scales"] = cref.cache8(len(c["k_scales"]), 16, 2, 128, 62)[1]  # scores stay ordinary
    check(c, out_dtype=torch.float32)


def test_weight_on_a_page_of_tiny_values():
    """All weight on a page whose scale is far below the others': its values are
    the output, to the relative precision of any other page."""
    c = case(63, 1, 1, 4, 1, 64, 16, [64], torch.float16, 0.0)
    q = torch.ones(1, 1, 4, 64, dtype=torch.float16)
    c["q"] = q
    raw(c["k_cache"])[:] = 0
    c["k_cache"][int(c["table"][0, 2])] = torch.full((16, 1, 64), 8.0).to(E4M3)  # score 64 above
    c["k_scales"][:] = 1.0
    c["v_scales"][:] = 1.0
    c["v_scales"][int(c["table"][0, 2])] = 2.0 ** -40
    k, v = cref.values8(c["k_cache"], c["k_scales"]), cref.values8(c["v_cache"], c["v_scales"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], 1.0)
    got = run(c, 1.0, out_dtype=torch.float32)
    # the other pages' weights are e^-512: their values do not show
    assert ((got.double() - want).abs() <= 2.0 ** -16 * 2.0 ** -40 * 448).all()
    assert got.abs().max() > 0


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 60])
def test_scales_at_the_ends_of_their_range(scale):
    c = case(65, 1, 1, 4, 1, 128, 16, [200], torch.bfloat16)
    c["v_scales"][:] = scale
    k, v = cref.values8(c["k_cache"], c["k_scales"]), cref.values8(c["v_cache"], c["v_scales"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], 128 ** -0.5)
    got = run(c, 128 ** -0.5, out_dtype=torch.float32)
    ref.close_out(got, want, cref.attention_slack(c["q"], k, v, 128 ** -0.5, 208, 2.0 ** -16))


@pytest.mark.parametrize("magnitude", [2.0 ** 100, 2.0 ** -100])
def test_queries_of_any_magnitude(magnitude):
    c = case(66, 2, 1, 8, 2, 128, 16, [200, 9], torch.bfloat16)
    c["q"] = (c["q"].float() * magnitude).to(torch.bfloat16)
    check(c, scale=128 ** -0.5 / magnitude, out_dtype=torch.float32)


def test_other_stream_and_torch_workspace():
    c = case(71, 3, 1, 8, 2, 128, 16, [5000, 1, 700], torch.bfloat16)
    check(c, stream=torch.cuda.Stream(), own_workspace=False)


def test_graph_replay_follows_lengths_and_tables():
    c = case(81, 4, 1, 8, 2, 128, 16, [3000, 200, 64, 1], torch.bfloat16)
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.zeros(c["q"].shape, dtype=torch.bfloat16, device=DEV)
    need = pa.workspace_size_kv8(d["q"], d["k_cache"], d["table"], out.dtype, 3000)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)

    def call():
        pa.decode_kv8(out, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"],
                      d["table"], d["lens"], 128 ** -0.5, 3000, workspace=ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c["lens"] = torch.tensor([2500, 1, 0, 9], dtype=torch.int32)
    c["table"][3, 0] = int(c["table"][1, 3])
    d["lens"].copy_(c["lens"])
    d["table"].copy_(c["table"])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    k, v = cref.values8(c["k_cache"], c["k_scales"]), cref.values8(c["v_cache"], c["v_scales"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], 128 ** -0.5)
    ref.close_out(out.cpu(), want, cref.attention_slack(
        c["q"], k, v, 128 ** -0.5, 3000, weights(torch.bfloat16)))


def test_equal_calls_give_equal_bits():
    c = case(91, 5, 2, 8, 2, 128, 16, [2000, 3, 900, 64, 5000], torch.float16)
    a = run(c, 0.1, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(a, run(c, 0.1, out_dtype=torch.float32))


def test_one_sequences_nan_stays_its_own():
    c = case(95, 3, 1, 8, 2, 128, 16, [100, 60, 200], torch.bfloat16)
    k, v = cref.values8(c["k_cache"], c["k_scales"]), cref.values8(c["v_cache"], c["v_scales"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], 0.1)
    c["q"][1] = math.nan
    got = run(c, 0.1)
    assert torch.isnan(got[1]).all()
    ref.close_out(got[0::2], want[0::2], cref.attention_slack(
        torch.nan_to_num(c["q"]), k, v, 0.1, 208, weights(torch.bfloat16)))
