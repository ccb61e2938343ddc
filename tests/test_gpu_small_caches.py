"""GPU tests of the operators on the 8-bit and the latent cache as they are used
together: prompts and steps appended and attended to, captured, on shared
workspaces, from several threads, on caches past 2^32 bytes, and every plan of
the attentions by shapes that take it."""
import math
import os
import re
import threading

import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def weights(out_dtype):
    """See test_gpu_kv8: how a weight is rounded on the way to the values."""
    return 2.0 ** -16 if out_dtype == torch.float32 else 2.0 ** -11


class Loop8:
    """A serving loop over an 8-bit cache: q, k, v of a step come in one tensor."""

    def __init__(self, B, H, Hkv, D, bs, longest, seed):
        self.H, self.Hkv, self.D, self.longest = H, Hkv, D, longest
        table, pool = ref.tables([longest] * B, bs, seed)
        self.table = table.to(DEV)
        self.kc, self.vc = (torch.full((pool, bs, Hkv, D), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3)
                            for _ in range(2))
        self.ks, self.vs = (torch.full((pool, Hkv), math.nan, device=DEV) for _ in range(2))
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.phases = pa.rope_phases(1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) * 2 / D))
        self.axes = torch.zeros(D // 2, dtype=torch.int32, device=DEV)
        self.ws = None

    def step(self, qkv):
        B, Q = qkv.shape[:2]
        H, Hkv = self.H, self.Hkv
        self.lens += Q
        pos = (self.lens.view(1, B, 1) - Q + torch.arange(Q, device=DEV, dtype=torch.int32)).contiguous()
        q = torch.empty((B, Q, H, self.D), dtype=qkv.dtype, device=DEV)
        pa.rope_append_kv8(q, self.kc, self.vc, self.ks, self.vs, qkv[:, :, :H], qkv[:, :, H:H + Hkv],
                           qkv[:, :, H + Hkv:], pos, self.phases, self.axes, self.table, self.lens)
        if self.ws is None:
            need = max(pa.workspace_size_kv8(q, self.kc, self.table, qkv.dtype, self.longest), 16)
            self.ws = torch.empty(need + (1 << 20), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(q)
        pa.decode_kv8(out, q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens,
                      self.D ** -0.5, self.longest, workspace=self.ws)
        return q, out


def check8(loop, q, out, lens):
    k, v = (cref.values8(c.cpu(), torch.nan_to_num(s.cpu()))
            for c, s in ((loop.kc, loop.ks), (loop.vc, loop.vs)))
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)   # (slots not written so far)
    scale = loop.D ** -0.5
    want = cref.attention(q.cpu(), k, v, loop.table.cpu(), lens, scale)
    ref.close_out(out.cpu(), want, cref.attention_slack(q.cpu(), k, v, scale, loop.longest,
                                                        weights(out.dtype)))


def test_serving_steps_over_the_8_bit_cache():
    B, H, Hkv, D, bs = 3, 8, 2, 128, 16
    loop = Loop8(B, H, Hkv, D, bs, 96, 1)
    lens = 0
    for i, Q in enumerate((40, 1, 1, 4, 1, 20, 1)):
        qkv = ref.normal((B, Q, H + 2 * Hkv, D), torch.bfloat16, 10 + i).to(DEV) * (1 + i)
        q, out = loop.step(qkv)
        torch.cuda.synchronize()
        lens += Q
        check8(loop, q, out, torch.full((B,), lens))
    assert pa.device_error() == 0


def test_a_captured_step_of_the_8_bit_cache_goes_on():
    B, H, Hkv, D, bs = 2, 8, 2, 64, 16
    eager, graph = (Loop8(B, H, Hkv, D, bs, 64, 2) for _ in range(2))
    prompt = ref.normal((B, 9, H + 2 * Hkv, D), torch.float16, 3).to(DEV)
    qkv = torch.zeros((B, 1, H + 2 * Hkv, D), dtype=torch.float16, device=DEV)
    for x in (eager, graph):
        x.step(prompt)
    torch.cuda.synchronize()
    saved = [t.clone() for t in (graph.kc.view(torch.uint8), graph.vc.view(torch.uint8), graph.ks, graph.vs,
                                 graph.lens)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.step(qkv)
    torch.cuda.synchronize()
    for t, s in zip((graph.kc.view(torch.uint8), graph.vc.view(torch.uint8), graph.ks, graph.vs, graph.lens),
                    saved):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, got = graph.step(qkv)
    for i in range(20):
        qkv.copy_(ref.normal(tuple(qkv.shape), torch.float16, 20 + i) * (1.0 + i))
        _, want = eager.step(qkv)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        assert torch.equal(graph.ks.nan_to_num(), eager.ks.nan_to_num())
    assert torch.equal(graph.kc.view(torch.uint8), eager.kc.view(torch.uint8))


def test_serving_steps_over_the_latent_cache():
    B, H, R, P, bs, longest = 3, 20, 256, 64, 16, 96
    table, pool = ref.tables([longest] * B, bs, 4)
    cache = torch.full((pool, bs, R + P), math.nan, dtype=torch.bfloat16, device=DEV)
    phases = pa.rope_phases(1e4 ** (-torch.arange(32, dtype=torch.float64, device=DEV) / 32))
    norm = ref.normal((R,), torch.bfloat16, 5).to(DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    total = 0
    for i, Q in enumerate((50, 1, 3, 1, 1)):
        total += Q
        lens += Q
        new = ref.normal((B, Q, R + P), torch.bfloat16, 30 + i).to(DEV)
        proj = ref.normal((B, Q, H, 128 + P), torch.bfloat16, 40 + i).to(DEV)
        query = ref.normal((B, Q, H, R + P), torch.bfloat16, 50 + i).to(DEV)   # (its first part absorbed)
        pos = (lens.view(B, 1) - Q + torch.arange(Q, device=DEV, dtype=torch.int32)).contiguous()
        pa.rope_append_latent(query[..., R:], cache, proj[..., 128:], new, norm, pos, phases,
                              table.to(DEV), lens)
        out = torch.empty((B, Q, H, R), dtype=torch.bfloat16, device=DEV)
        pa.decode_latent(out, query, cache, table.to(DEV), lens, 0.1, longest)
        torch.cuda.synchronize()
        c = torch.nan_to_num(cache.cpu().double()).unsqueeze(2)
        want = cref.attention(query.cpu(), c, c[..., :R], table, torch.full((B,), total), 0.1)
        ref.close_out(out.cpu(), want, cref.attention_slack(query.cpu(), c, c[..., :R], 0.1, longest,
                                                            2.0 ** -8))
    assert pa.device_error() == 0


# ---- every plan of the two attentions ----

def case8(seed, B, Q, H, Hkv, D, bs, lens, dtype):
    table, pool = ref.tables(lens, bs, seed)
    kc, ks = cref.cache8(pool, bs, Hkv, D, seed + 1)
    vc, vs = cref.cache8(pool, bs, Hkv, D, seed + 2)
    return dict(q=ref.normal((B, Q, H, D), dtype, seed + 3), kc=kc, vc=vc, ks=ks, vs=vs, table=table,
                lens=torch.tensor(lens, dtype=torch.int32))


def run8(c, out_dtype=None, ws=None):
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.full(c["q"].shape, math.nan, dtype=out_dtype or c["q"].dtype, device=DEV)
    pa.decode_kv8(out, d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"],
                  c["q"].shape[-1] ** -0.5, int(c["lens"].max()), workspace=ws)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu()


@pytest.mark.parametrize("B,Q,H,Hkv,D,bs,T", [
    (1, 40, 32, 8, 64, 16, 600),     # 5 chunks of 8 kv heads: two groups of units a sequence
    (3, 40, 16, 2, 64, 16, 700),     # chunks of 32 rows, clusters
    (5, 4, 64, 8, 64, 16, 4200),     # clusters that fill the GPU, 33 steps a CTA
    (2, 3, 16, 1, 256, 32, 1500),    # 48 rows at head_dim 256
    (2, 8, 4, 1, 128, 32, 1500),     # 32 rows at head_dim 128
    (1, 1, 8, 1, 128, 16, 20000),    # a unit over many runs
    (1, 1, 8, 1, 64, 16, 9000),      # runs over each head_dim and row tile
    (1, 2, 8, 1, 64, 32, 9000),
    (2, 4, 8, 1, 64, 16, 9100),
    (2, 2, 8, 1, 128, 32, 9000),
    (1, 4, 8, 1, 128, 16, 9000),
    (2, 1, 4, 1, 256, 16, 9000),
    (1, 5, 8, 2, 256, 32, 9000),
    (130, 1, 8, 8, 64, 16, 40),      # short contexts, a unit to a CTA
])
def test_plans_of_the_8_bit_attention(B, Q, H, Hkv, D, bs, T):
    lens = [max(1, T - 37 * (b % 5)) for b in range(B)]
    c = case8(B + Q + D, B, Q, H, Hkv, D, bs, lens, torch.bfloat16)
    k, v = cref.values8(c["kc"], c["ks"]), cref.values8(c["vc"], c["vs"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], D ** -0.5)
    for dt in (torch.bfloat16, torch.float32):
        ref.close_out(run8(c, dt), want, cref.attention_slack(c["q"], k, v, D ** -0.5, T, weights(dt)))


def test_many_sequences_over_the_8_bit_cache():
    """More units than runs hold, more lengths than a CTA looks through: each
    sequence as alone."""
    B, T = 2100, 600
    one = case8(5, 1, 1, 2, 1, 64, 16, [T], torch.float16)
    lens = torch.tensor([1 + (b * 7919) % T for b in range(B)], dtype=torch.int32)
    c = dict(one, q=one["q"].expand(B, 1, 2, 64).contiguous(), lens=lens,
             table=one["table"].expand(B, -1).contiguous())
    got = run8(c)
    k, v = cref.values8(c["kc"], c["ks"]), cref.values8(c["vc"], c["vs"])
    for b in list(range(0, B, 97)) + [B - 1]:
        want = cref.attention(one["q"], k, v, one["table"], lens[b:b + 1], 0.125)
        ref.close_out(got[b:b + 1], want, cref.attention_slack(one["q"], k, v, 0.125, T, 2.0 ** -11))


def run_latent(q, cache, table, lens, scale, ws=None, out=None):
    R = cache.shape[2] - 64
    if out is None:
        out = torch.full((*q.shape[:-1], R), math.nan, dtype=q.dtype, device=DEV)
    pa.decode_latent(out, q.to(DEV), cache.to(DEV), table.to(DEV), lens.to(DEV), scale,
                     int(lens.max()), workspace=ws)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    return out.cpu()


@pytest.mark.parametrize("B,Q,H,R,T", [
    (1, 11, 128, 128, 300),    # 22 row tiles: three groups of 8, 8 and 6, CTAs without a row tile
    (2, 9, 128, 128, 200),     # 18 row tiles
    (80, 1, 64, 128, 70),      # sequences of one length in turn
    (170, 1, 16, 128, 70),     # more of them than groups
    (3, 1, 16, 128, 9000),     # cut by many runs
])
def test_plans_of_the_latent_attention(B, Q, H, R, T):
    one = ref.tables([T] * min(B, 4), 16, B + Q)
    table, pool = one[0].repeat((B + 3) // min(B, 4), 1)[:B].contiguous(), one[1]
    cache = ref.normal((pool, 16, R + 64), torch.bfloat16, B)
    q = ref.normal((B, Q, H, R + 64), torch.bfloat16, B + 1)
    lens = torch.full((B,), T, dtype=torch.int32)
    got = run_latent(q, cache, table, lens, 0.1)
    c = cache.double().unsqueeze(2)
    for b in sorted({0, 1 % B, B // 2, B - 1}):
        want = cref.attention(q[b:b + 1], c, c[..., :R], table[b:b + 1], lens[b:b + 1], 0.1)
        ref.close_out(got[b:b + 1], want, cref.attention_slack(q[b:b + 1], c, c[..., :R], 0.1, T, 2.0 ** -8))


def test_many_sequences_over_the_latent_cache():
    B, T, R = 2100, 200, 128
    table, pool = ref.tables([T], 32, 7)
    cache = ref.normal((pool, 32, R + 64), torch.float16, 8)
    q = ref.normal((1, 1, 3, R + 64), torch.float16, 9)
    lens = torch.tensor([(b * 7919) % (T + 1) for b in range(B)], dtype=torch.int32)
    got = run_latent(q.expand(B, 1, 3, R + 64).contiguous(), cache, table.expand(B, -1).contiguous(), lens, 0.1)
    c = cache.double().unsqueeze(2)
    for b in list(range(0, B, 97)) + [B - 1]:
        want = cref.attention(q, c, c[..., :R], table, lens[b:b + 1], 0.1)
        ref.close_out(got[b:b + 1], want, cref.attention_slack(q, c, c[..., :R], 0.1, T, 2.0 ** -11))


# ---- workspaces, rows behind the batch, graphs, threads, large caches ----

def test_workspaces_that_do_not_fit():
    c = case8(11, 1, 1, 4, 1, 128, 16, [9000], torch.bfloat16)
    d = {k: v.to(DEV) for k, v in c.items()}
    need = pa.workspace_size_kv8(d["q"], d["kc"], d["table"], torch.bfloat16, 9000)
    assert need > 0
    out = torch.zeros(c["q"].shape, dtype=torch.bfloat16, device=DEV)
    args = (out, d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], 0.1, 9000)
    buf = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    for ws in (buf[:need - 1], buf[1:]):
        with pytest.raises(pa.PaError) as e:
            pa.decode_kv8(*args, workspace=ws)
        assert e.value.code == 3
    pa.decode_kv8(*args, workspace=buf[:need])
    q = torch.zeros((1, 1, 16, 192), dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros((600, 16, 192), dtype=torch.bfloat16, device=DEV)
    table = torch.arange(600, dtype=torch.int32, device=DEV).view(1, 600)
    lens = torch.tensor([9000], dtype=torch.int32, device=DEV)
    need = pa.workspace_size_latent(q, cache, 128, table, 9000)
    assert need > 0
    out = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
    buf = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    for ws in (buf[:need - 1], buf[1:]):
        with pytest.raises(pa.PaError) as e:
            pa.decode_latent(out, q, cache, table, lens, 0.1, 9000, workspace=ws)
        assert e.value.code == 3
    with pytest.raises(pa.PaError) as e:   # the output inside the workspace
        pa.decode_latent(buf[:4096].view(torch.bfloat16).view(1, 1, 16, 128), q, cache, table, lens, 0.1,
                         9000, workspace=buf[:need])
    assert e.value.code == 1
    pa.decode_latent(out, q, cache, table, lens, 0.1, 9000, workspace=buf[:need])
    torch.cuda.synchronize()


def test_rows_behind_the_batch_stay_and_calls_share_a_workspace():
    """Calls of several shapes in turn on one workspace full of NaN, each into the
    first rows of a larger output."""
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for i, (B, H, R, T) in enumerate([(2, 128, 512, 900), (5, 16, 512, 3000), (1, 40, 256, 5000), (2, 128, 512, 900)]):
        table, pool = ref.tables([T - 11 * b for b in range(B)], 32, 60 + i)
        cache = ref.normal((pool, 32, R + 64), torch.bfloat16, 61)
        q = ref.normal((B, 1, H, R + 64), torch.bfloat16, 62)
        lens = torch.tensor([T - 11 * b for b in range(B)], dtype=torch.int32)
        big = torch.full((B + 3, 1, H, R), 7.0, dtype=torch.bfloat16, device=DEV)
        got = run_latent(q, cache, table, lens, 0.1, ws=ws, out=big[:B])
        assert (big[B:] == 7).all()
        c = cache.double().unsqueeze(2)
        want = cref.attention(q, c, c[..., :R], table, lens, 0.1)
        ref.close_out(got, want, cref.attention_slack(q, c, c[..., :R], 0.1, T, 2.0 ** -8))
    c = case8(13, 2, 1, 8, 2, 128, 16, [5000, 4000], torch.float16)
    k, v = cref.values8(c["kc"], c["ks"]), cref.values8(c["vc"], c["vs"])
    want = cref.attention(c["q"], k, v, c["table"], c["lens"], 128 ** -0.5)
    ref.close_out(run8(c, ws=ws), want, cref.attention_slack(c["q"], k, v, 128 ** -0.5, 5000, 2.0 ** -11))


def test_two_graphs_on_one_workspace():
    q = ref.normal((2, 1, 16, 576), torch.bfloat16, 70).to(DEV)
    cache = ref.normal((200, 64, 576), torch.bfloat16, 71).to(DEV)
    table = torch.arange(200, dtype=torch.int32, device=DEV).view(2, 100)
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([6400, 100], [3, 6000])]
    ws = torch.empty(max(pa.workspace_size_latent(q, cache, 512, table, 6400), 16), dtype=torch.uint8, device=DEV)
    outs, wants, graphs = [], [], []
    for n in lens:
        want = torch.empty((2, 1, 16, 512), dtype=torch.bfloat16, device=DEV)
        pa.decode_latent(want, q, cache, table, n, 0.05, 6400, workspace=ws)
        torch.cuda.synchronize()
        wants.append(want)
        outs.append(torch.zeros_like(want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.decode_latent(outs[-1], q, cache, table, n, 0.05, 6400, workspace=ws)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)


def test_threads_on_streams_of_their_own():
    c8 = [case8(80 + i, 2, 1, 8, 2, 128, 16, [4000, 500 + i], torch.bfloat16) for i in range(2)]
    lat = []
    for i in range(2):
        table, pool = ref.tables([3000, 200], 64, 90 + i)
        lat.append((ref.normal((2, 1, 64, 576), torch.bfloat16, 91 + i), ref.normal((pool, 64, 576), torch.bfloat16, 92),
                    table, torch.tensor([3000, 200], dtype=torch.int32)))
    want = [run8(c) for c in c8] + [run_latent(*x, 0.1) for x in lat]
    dev8 = [{k: v.to(DEV) for k, v in c.items()} for c in c8]
    devl = [tuple(t.to(DEV) for t in x) for x in lat]
    torch.cuda.synchronize()
    errors = []

    def worker():
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                outs = []
                with torch.cuda.stream(s):
                    for d in dev8:
                        out = torch.empty_like(d["q"])
                        pa.decode_kv8(out, d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"],
                                      128 ** -0.5, 4000)
                        outs.append(out)
                    for q, cache, table, lens in devl:
                        out = torch.empty((2, 1, 64, 512), dtype=torch.bfloat16, device=DEV)
                        pa.decode_latent(out, q, cache, table, lens, 0.1, 3000)
                        outs.append(out)
                s.synchronize()
                for w, o in zip(want, outs):
                    assert torch.equal(o.cpu(), w)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=worker) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_caches_past_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32: the same bits as on a small cache."""
    big_n, bs, Hkv, D = 300000, 16, 8, 128           # 4.9e9 codes
    small = case8(100, 2, 1, 16, Hkv, D, bs, [100, 37], torch.bfloat16)
    first = big_n - len(small["kc"])
    assert first * bs * Hkv * D > 2 ** 32
    want = run8(small)
    kc, vc = (torch.empty((big_n, bs, Hkv, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty((big_n, Hkv), device=DEV) for _ in range(2))
    for b, s in ((kc, "kc"), (vc, "vc")):
        b[first:] = small[s].view(torch.uint8).to(DEV)
    for b, s in ((ks, "ks"), (vs, "vs")):
        b[first:] = small[s].to(DEV)
    table = torch.where(small["table"] >= 0, small["table"] + first, -1).to(torch.int32).to(DEV)
    lens = small["lens"].to(DEV)
    q = small["q"].to(DEV)
    out = torch.empty_like(q)
    pa.decode_kv8(out, q, kc.view(E4M3), vc.view(E4M3), ks, vs, table, lens, D ** -0.5, 100)
    assert torch.equal(out.cpu(), want)
    qkv = ref.normal((2, 5, 16 + 2 * Hkv, D), torch.bfloat16, 101).to(DEV)
    phases = pa.rope_phases(torch.ones(64, dtype=torch.float64, device=DEV))
    axes = torch.zeros(64, dtype=torch.int32, device=DEV)
    pos = torch.zeros((1, 2, 5), dtype=torch.int32, device=DEV)
    sk, sv = (small[x].to(DEV) for x in ("kc", "vc"))
    ssk, ssv = (small[x].to(DEV) for x in ("ks", "vs"))
    for k_, v_, s1, s2, t in ((kc.view(E4M3), vc.view(E4M3), ks, vs, table),
                              (sk, sv, ssk, ssv, small["table"].to(DEV))):
        q5 = torch.empty((2, 5, 16, D), dtype=torch.bfloat16, device=DEV)
        pa.rope_append_kv8(q5, k_, v_, s1, s2, qkv[:, :, :16], qkv[:, :, 16:24], qkv[:, :, 24:], pos, phases,
                           axes, t, lens)
    assert torch.equal(kc[first:], sk.view(torch.uint8)) and torch.equal(vc[first:], sv.view(torch.uint8))
    assert torch.equal(ks[first:], ssk) and torch.equal(vs[first:], ssv)
    del kc, vc, ks, vs
    # the latent cache: 2.4e9 elements
    pages, W = 65000, 576
    q = ref.normal((2, 1, 16, W), torch.bfloat16, 102).to(DEV)
    table, pool = ref.tables([150, 70], 64, 103)
    part = ref.normal((pool, 64, W), torch.bfloat16, 104).to(DEV)
    cache = torch.empty((pages, 64, W), dtype=torch.bfloat16, device=DEV)
    first = pages - pool
    cache[first:] = part
    lens = torch.tensor([150, 70], dtype=torch.int32, device=DEV)
    far = torch.where(table >= 0, table + first, -1).to(torch.int32).to(DEV)
    assert first * 64 * W > 2 ** 31
    a, b = (torch.empty((2, 1, 16, 512), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pa.decode_latent(a, q, cache, far, lens, 0.1, 150)
    pa.decode_latent(b, q, part, table.to(DEV), lens, 0.1, 150)
    assert torch.equal(a, b)
    new = ref.normal((2, 3, W), torch.bfloat16, 105).to(DEV)
    rq = ref.normal((2, 3, 4, 64), torch.bfloat16, 106).to(DEV)
    p2 = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    phases = pa.rope_phases(torch.ones(32, dtype=torch.float64, device=DEV))
    for c, t in ((cache, far), (part, table.to(DEV))):
        pa.rope_append_latent(torch.empty_like(rq), c, rq, new, None, p2, phases, t, lens)
    assert torch.equal(cache[first:], part)


def test_the_readme_example_of_the_small_caches_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    code = next(b for b in blocks if "decode_kv8" in b)
    space = {}
    exec(compile(code, "README.md", "exec"), space)
    torch.cuda.synchronize()
    assert torch.isfinite(space["out8"]).all() and torch.isfinite(space["out"]).all()
    assert pa.device_error() == 0
