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


APART = 1 << 20   # announced so long, a prefix is read in a launch of its own


def prefix_loop(n, Q, H, Hkv, D, own, prefix, wide=0):
    """(turn(i), reset()) of samples behind one prefix, everything rewritten before each call."""
    bs, dtype = 16, torch.bfloat16
    vs, first = variants(4, n, H, Hkv, D, bs, own, dtype, 0, Q)
    if wide:
        for v in vs:
            table = torch.full((n, wide // bs), -1, dtype=torch.int32, device=DEV)
            table[:, :v["table"].shape[1]] = v["table"]
            v["table"] = table
    pages = (prefix + bs - 1) // bs
    for i, v in enumerate(vs):
        g = torch.Generator().manual_seed(i)
        v["ptable"] = torch.full((1, APART // bs), -1, dtype=torch.int32)
        v["ptable"][0, :pages] = (torch.randperm(pages, generator=g) + first).to(torch.int32)
        v["ptable"] = v["ptable"].to(DEV)
        v["plens"] = torch.tensor([prefix - 37 * i], dtype=torch.int32, device=DEV)
    phases, axes = rotary(D)
    k0, v0 = (ref.normal((first + pages, bs, Hkv, D), dtype, s).to(DEV) for s in (93, 94))
    kc, vc = k0.clone(), v0.clone()
    state = {x: torch.empty_like(vs[0][x]) for x in vs[0]}
    q, out = (torch.empty((n, Q, H, D), dtype=dtype, device=DEV) for _ in range(2))
    max_own = wide or own
    need = pa.workspace_size_shared_prefix(q, kc, state["ptable"], state["table"], dtype, APART, max_own)
    assert need > 0                                  # launches of their own
    ws = torch.empty((need // 4 + 1,), device=DEV)

    def reset():
        kc.copy_(k0)
        vc.copy_(v0)
        ws.fill_(float("nan"))

    def turn(i):
        for x, t in state.items():
            t.copy_(vs[i % len(vs)][x])
        qkv = state["qkv"]
        pa.rope_append_kv(q, kc, vc, qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:],
                          state["pos"], phases, axes, state["table"], state["lens"])
        pa.decode_shared_prefix(out, q, kc, vc, state["ptable"], state["plens"], state["table"],
                                state["lens"], D ** -0.5, APART, max_own, workspace=ws)
        return out.clone()

    return turn, reset


# own pages on the warp-level kernel, on the tile kernel, and two tiles to a CTA
LOOPS = [(20, 1, 32, 8, 128, 300, 3000, 0), (4, 40, 8, 2, 128, 200, 3000, 0),
         (4, 40, 32, 8, 128, 200, 3000, 65536), (3, 8, 16, 1, 256, 100, 500, 0)]


@pytest.mark.parametrize("args", LOOPS)
def test_shared_prefix_in_launches_of_their_own(args):
    turn, reset = prefix_loop(*args)
    reset()
    alone = []
    for i in range(TURNS):
        alone.append(turn(i))
        torch.cuda.synchronize()
    reset()
    torch.cuda.synchronize()
    together = [turn(i) for i in range(TURNS)]
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for a, b in zip(alone, together):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_shared_prefix_captured_with_what_surrounds_it():
    """Several calls and their inputs' copies in one graph, replayed without a wait."""
    turn, reset = prefix_loop(*LOOPS[0])
    reset()
    for _ in range(5):     # (a round appends to slots that the next one reads)
        want = [turn(i) for i in range(4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [turn(i) for i in range(4)]
    reset()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_shared_prefix_eager_while_another_stream_is_captured():
    (ta, ra), (tb, rb) = prefix_loop(*LOOPS[0]), prefix_loop(*LOOPS[1])
    ra(), rb()
    want_a, want_b = ta(0), tb(0)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    got_b = []
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        got_a = ta(0)
        with torch.cuda.stream(side):
            got_b.append(tb(0))
        again = ta(0)
    torch.cuda.synchronize()
    assert torch.equal(got_b[0], want_b)
    ra()
    for _ in range(2):
        graph.replay()
    assert torch.equal(tb(0), want_b)                # eager after the capture
    torch.cuda.synchronize()
    assert torch.equal(got_a, want_a) and torch.equal(again, want_a)
    assert pa.device_error() == 0


def test_shared_prefix_on_one_stream_does_not_wait_for_another():
    (ta, ra), (tb, rb) = prefix_loop(*LOOPS[0]), prefix_loop(*LOOPS[1])
    ra(), rb()
    want_a, want_b = ta(0), tb(0)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    done = torch.cuda.Event()
    with torch.cuda.stream(sa):
        torch.cuda._sleep(int(4e8))                  # some 0.2 s
        got_a = ta(0)
        done.record()
    with torch.cuda.stream(sb):
        got_b = tb(0)
    sb.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(got_a, want_a) and torch.equal(got_b, want_b)


def test_shared_prefix_from_several_threads():
    import threading

    loops = [prefix_loop(*LOOPS[i % 2]) for i in range(4)]
    want = []
    for turn, reset in loops:
        reset()
        want.append([turn(i) for i in range(8)])
    torch.cuda.synchronize()
    got = [None] * len(loops)

    def work(x):
        with torch.cuda.stream(torch.cuda.Stream(DEV)):
            loops[x][1]()
            got[x] = [loops[x][0](i) for i in range(8)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(x,)) for x in range(len(loops))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert pa.device_error() == 0
