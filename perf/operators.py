"""What is measured of the serving-step operators around paged attention.

Four operators on one paged KV cache, in the order in which a long-context
serving loop calls them:

  rope        multi-axis rotary positions for the new tokens' queries and keys
              (text, image and video tokens: an axis of its own for time, height
              and width), the keys and values written into their cache slots;
  prefix      attention of sequences that share a long prefix, whose pages are
              read once for all of them, joined with each sequence's own pages;
  accumulate  paged attention that also adds each cached token's attention
              weight to a running sum per kv head;
  evict       the cache cut down to a budget of tokens per kv head: the first
              and the latest tokens and those of the largest running sums.

A case names its operator in "op".  ``run`` computes the plain form, or with
``own`` set makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


def listed():
    return [
        # one decode step of a small chat batch: every sequence's new token, text and image axes
        dict(name="rope_step", op="rope", B=8, Q=1, H=32, Hkv=8, D=128, rot=128, axes=3,
             interleaved=False, dtype="bf16", bs=16, past=100),
        # a prompt of two videos: tens of thousands of tokens with (time, height, width)
        dict(name="rope_video", op="rope", B=2, Q=12001, H=16, Hkv=4, D=64, rot=64, axes=3,
             interleaved=True, dtype="fp16", bs=16, past=37),
        # a few users of one short system prompt, latency bound
        dict(name="prefix_step", op="prefix", P=1, n=4, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", prefix=1001, suffix=64),
        # a full batch behind one system prompt with its documents
        dict(name="prefix_system", op="prefix", P=1, n=64, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", prefix=8191, suffix=1024),
        # eight prompts, eight samples each, four drafted tokens to verify, one kv head
        dict(name="prefix_samples", op="prefix", P=8, n=8, Q=4, H=16, Hkv=1, D=256, bs=32,
             dtype="bf16", prefix=4100, suffix=300),
        # many questions about one book
        dict(name="prefix_book", op="prefix", P=1, n=128, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", prefix=65536, suffix=2048),
        # one short conversation, latency bound
        dict(name="accumulate_step", op="accumulate", B=1, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", lo=700, hi=700),
        # a batch of very different lengths
        dict(name="accumulate_ragged", op="accumulate", B=32, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="fp16", lo=1, hi=8192),
        # long contexts, one token each
        dict(name="accumulate_long", op="accumulate", B=4, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", lo=65536, hi=65536),
        # the last window of a prompt, whose queries judge the prompt's tokens
        dict(name="accumulate_window", op="accumulate", B=2, Q=64, H=32, Hkv=8, D=128, bs=16,
             dtype="bf16", lo=8001, hi=8001),
        # one conversation past its budget
        dict(name="evict_one", op="evict", B=1, Hkv=8, D=128, bs=16, dtype="bf16", lo=2000,
             hi=2000, budget=1024, sink=4, recent=256),
        # long documents cut down after their prompt
        dict(name="evict_long", op="evict", B=4, Hkv=8, D=128, bs=16, dtype="bf16", lo=65000,
             hi=131072, budget=8192, sink=4, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["rope", "prefix", "accumulate", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    while Hkv * G > 64:
        G //= 2
    bs = rng.choice([16, 32])
    c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, bs=bs)
    if op == "rope":
        Q = 1 if rng.random() < 0.4 else _log_int(rng, 2, 16000)
        c.update(B=_log_int(rng, 1, 128), Q=Q, H=Hkv * G, axes=rng.choice([1, 2, 3, 4]),
                 interleaved=rng.random() < 0.5, past=_log_int(rng, 1, 300),
                 rot=rng.choice([D, D, D // 2, D // 4]))
    elif op == "prefix":
        c.update(P=rng.choice([1, 1, 1, 2, 5, 8]), n=_log_int(rng, 1, 128),
                 Q=rng.choice([1, 1, 1, 2, 4, 7]), H=Hkv * G,
                 prefix=_log_int(rng, 100, 65536), suffix=_log_int(rng, 1, 2048))
    elif op == "accumulate":
        hi = _log_int(rng, 300, 65536)
        c.update(B=_log_int(rng, 1, 64), Q=rng.choice([1, 1, 1, 2, 5, 16, 33, 64]), H=Hkv * G,
                 lo=hi if rng.random() < 0.3 else 1 + hi // 10, hi=hi)
    else:
        hi = _log_int(rng, 1000, 131072)
        budget = _log_int(rng, 64, 8192)
        c.update(B=_log_int(rng, 1, 16), lo=1 + hi // 2, hi=hi, budget=budget,
                 sink=rng.randint(0, 8), recent=rng.randint(0, budget // 4))
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), max(w["bytes"], w["flops"] / 280))
    while True:
        c = _draw_once(rng)
        w = work(c)
        if max(w["bytes"], w["flops"] / 280) > most[c["op"]]:
            continue
        # scores of the plain form and pages of the state, kept to a few GB
        if c["op"] == "prefix" and c["P"] * c["n"] * c["Q"] * c["H"] * (c["prefix"] + c["suffix"]) > 6e8:
            continue
        if c["op"] == "accumulate" and (c["B"] * c["Q"] * c["H"] * c["hi"] > 6e8 or
                                        c["B"] * c["hi"] * c["Hkv"] * c["D"] > 4e8):
            continue
        return c


def _lens(case):
    """Context lengths of a case, the same for every seed (the work depends on
    them): spread evenly over [lo, hi], in a scattered order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * ((b * 7919) % B) // (B - 1) for b in range(B)]


def _suffix_lens(case):
    n, Q = case["P"] * case["n"], case["Q"]
    lo, hi = Q, max(Q, case["suffix"])
    return [hi if n == 1 else lo + (hi - lo) * ((b * 7919) % n) // (n - 1) for b in range(n)]


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        tokens = case["B"] * case["Q"]
        return {"bytes": tokens * D * 2 * 2 * (case["H"] + 2 * case["Hkv"])
                + tokens * 4 * case["axes"] + case["rot"] // 2 * 12 + case["B"] * 4,
                "flops": tokens * case["rot"] * 3 * (case["H"] + case["Hkv"])}
    if case["op"] == "prefix":
        rows, own_tokens = case["n"] * case["Q"] * case["H"], sum(_suffix_lens(case))
        tokens = case["P"] * case["prefix"] + own_tokens
        return {"bytes": tokens * case["Hkv"] * D * 4 + case["P"] * rows * D * 4
                + 4 * (tokens // case["bs"]),
                "flops": 4 * D * (case["P"] * rows * case["prefix"]
                                  + case["Q"] * case["H"] * own_tokens)}
    tokens = sum(_lens(case))
    if case["op"] == "accumulate":
        rows = case["Q"] * case["H"]
        return {"bytes": tokens * case["Hkv"] * (D * 4 + 8) + case["B"] * rows * D * 4
                + 4 * (tokens // case["bs"]),
                "flops": 4 * D * rows * tokens}
    kept = sum(min(t, case["budget"]) for t in _lens(case)) * case["Hkv"]
    slots = case["B"] * case["Hkv"] * _pages(case["budget"], case["bs"]) * case["bs"]
    return {"bytes": tokens * case["Hkv"] * 4 + kept * (D * 8 + 4) + slots * 4, "flops": 0}


def _pages(tokens, bs):
    return (tokens + bs - 1) // bs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _tables(lens, bs, g, first=0, width=None):
    """Block tables (-1 padded) of sequences of these lengths over scattered
    pages first, first + 1, ... and the next free page."""
    pages = [_pages(t, bs) for t in lens]
    total = sum(pages)
    order = (torch.randperm(total, generator=g, device=DEV) + first).to(torch.int32)
    width = width or max(1, max(pages))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    return table, first + total


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    dt, bs, D, Hkv = DTYPES[case["dtype"]], case["bs"], case["D"], case["Hkv"]
    s = {"case": case}
    if case["op"] == "rope":
        B, Q, H, A = case["B"], case["Q"], case["H"], case["axes"]
        # the last sequence of a batch is padded: its first tokens lie before its start
        lens = [case["past"] + Q + 3 * b for b in range(B)]
        if B > 1:
            lens[-1] = max(1, Q // 2)
        table, pool = _tables(lens, bs, g)
        qkv = _normal((B, Q, H + 2 * Hkv, D), dt, g)  # one projection's output
        half = case["rot"] // 2
        inv_freq = 1e4 ** (-torch.arange(half, dtype=torch.float64, device=DEV) * 2 / case["rot"])
        axis = (torch.arange(half, device=DEV) % A).to(torch.int32)
        at = torch.tensor(lens, device=DEV).view(B, 1) - Q + torch.arange(Q, device=DEV)
        # time runs with the token, the other axes with a frame's rows and columns
        pos = torch.stack([at if a == 0 else (at // (7 * a)) % 97 + 1000 * a for a in range(A)])
        s.update(q=qkv[:, :, :H], k=qkv[:, :, H:H + Hkv], v=qkv[:, :, H + Hkv:],
                 q_out=torch.zeros((B, Q, H, D), dtype=dt, device=DEV),
                 k_cache=_normal((pool + 1, bs, Hkv, D), dt, g),
                 v_cache=_normal((pool + 1, bs, Hkv, D), dt, g),
                 pos=pos.to(torch.int32).contiguous(), inv_freq=inv_freq, axis=axis, table=table,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        if own:
            import paged_kv_attention_08_gb300 as pa
            s["phases"] = pa.rope_phases(inv_freq)
    elif case["op"] == "prefix":
        P, n, Q, H = case["P"], case["n"], case["Q"], case["H"]
        plens = [case["prefix"] - 5 * i for i in range(P)]
        slens = _suffix_lens(case)
        ptable, first = _tables(plens, bs, g)
        table, pool = _tables(slens, bs, g, first)
        s.update(q=_normal((P * n, Q, H, D), dt, g),
                 out=torch.zeros((P * n, Q, H, D), dtype=dt, device=DEV),
                 k_cache=_normal((pool, bs, Hkv, D), dt, g),
                 v_cache=_normal((pool, bs, Hkv, D), dt, g), ptable=ptable, table=table,
                 plens=torch.tensor(plens, dtype=torch.int32, device=DEV),
                 lens=torch.tensor(slens, dtype=torch.int32, device=DEV), scale=D ** -0.5)
        if own:
            import paged_kv_attention_08_gb300 as pa
            need = pa.workspace_size_shared_prefix(s["q"], s["k_cache"], ptable, table, dt,
                                                   case["prefix"], max(slens))
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    elif case["op"] == "accumulate":
        B, Q, H = case["B"], case["Q"], case["H"]
        lens = _lens(case)
        table, pool = _tables(lens, bs, g)
        width = table.shape[1] * bs
        # what some tens of earlier queries have left, as uneven as attention is
        w = torch.exp(torch.randn((B, Hkv, width), generator=g, device=DEV)) * (20.0 / max(lens))
        s.update(q=_normal((B, Q, H, D), dt, g),
                 out=torch.zeros((B, Q, H, D), dtype=dt, device=DEV),
                 k_cache=_normal((pool, bs, Hkv, D), dt, g),
                 v_cache=_normal((pool, bs, Hkv, D), dt, g), table=table, weights=w,
                 new_weights=torch.zeros_like(w),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scale=D ** -0.5)
        if own:
            import paged_kv_attention_08_gb300 as pa
            need = pa.workspace_size_accumulate(s["q"], s["k_cache"], table, dt, max(lens))
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    else:
        B, budget = case["B"], case["budget"]
        lens = _lens(case)
        table, first = _tables(lens, bs, g)
        new_table, pool = _tables([budget] * B, bs, g, first)
        width = table.shape[1] * bs
        w = torch.exp(1.5 * torch.randn((B, Hkv, width), generator=g, device=DEV)) / max(lens)
        # some tokens have never had a weight that shows: ties
        w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, 0.0, w)
        t = torch.arange(width, device=DEV)
        w = torch.where(t < torch.tensor(lens, device=DEV).view(B, 1, 1), w, 0.0)
        s.update(k_cache=_normal((pool, bs, Hkv, D), dt, g),
                 v_cache=_normal((pool, bs, Hkv, D), dt, g), table=table, weights=w,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), new_table=new_table,
                 new_weights=torch.zeros((B, Hkv, new_table.shape[1] * bs), device=DEV),
                 new_lens=torch.zeros((B,), dtype=torch.int32, device=DEV),
                 kept=torch.zeros((B, Hkv, budget), dtype=torch.int32, device=DEV))
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import paged_kv_attention_08_gb300 as pa
    c = s["case"]
    if c["op"] == "rope":
        pa.rope_append_kv(s["q_out"], s["k_cache"], s["v_cache"], s["q"], s["k"], s["v"], s["pos"],
                          s["phases"], s["axis"], s["table"], s["lens"],
                          interleaved=c["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "prefix":
        longest = max(c["Q"], c["suffix"])
        pa.decode_shared_prefix(s["out"], s["q"], s["k_cache"], s["v_cache"], s["ptable"],
                                s["plens"], s["table"], s["lens"], s["scale"], c["prefix"], longest,
                                workspace=s["workspace"])
        return s["out"]
    if c["op"] == "accumulate":
        pa.decode_accumulate(s["out"], s["new_weights"], s["q"], s["k_cache"], s["v_cache"],
                             s["table"], s["lens"], s["scale"], c["hi"], weights=s["weights"],
                             workspace=s["workspace"])
        return s["out"], s["new_weights"]
    pa.evict_kv(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["lens"], s["new_table"],
                s["new_weights"], s["new_lens"], s["kept"], sink=c["sink"], recent=c["recent"])
    return s["kept"], s["new_lens"], s["new_weights"], s["k_cache"], s["v_cache"]


def _gather(cache, table):
    """[S, Hkv, tokens, D] in 32 bits of the pages that a table names."""
    x = cache[table.clamp(min=0).long()]
    S, m, bs, Hkv, D = x.shape
    return x.reshape(S, m * bs, Hkv, D).permute(0, 2, 1, 3).float()


def _in_table(table, bs):
    return (table >= 0).repeat_interleave(bs, dim=1)


def _run_plain(s):
    c = s["case"]
    bs = c["bs"]
    if c["op"] == "rope":
        B, Q, H, half = c["B"], c["Q"], c["H"], c["rot"] // 2
        # angles in 64 bits: far positions
        ang = s["pos"].double()[s["axis"].long()].permute(1, 2, 0) * s["inv_freq"]
        cos, sin = ang.cos().float().unsqueeze(2), ang.sin().float().unsqueeze(2)

        def turn(x):
            x = x.float()
            if c["interleaved"]:
                a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
                r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
            else:
                a, b = x[..., :half], x[..., half:2 * half]
                r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
            return torch.cat([r, x[..., 2 * half:]], -1)

        dt = s["q"].dtype
        s["q_out"].copy_(turn(s["q"]))
        k = turn(s["k"]).to(dt).reshape(B * Q, c["Hkv"], c["D"])
        at = s["lens"].long().view(B, 1) - Q + torch.arange(Q, device=DEV)
        page = s["table"].long().gather(1, at.clamp(min=0) // bs)
        # tokens before a sequence's start go to the spare last block, which keeps its values
        spare = (s["k_cache"].shape[0] - 1) * bs
        valid = ((at >= 0) & (page >= 0)).reshape(-1)
        slot = torch.where(valid, (page * bs + at.clamp(min=0) % bs).reshape(-1), spare)
        for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].reshape(B * Q, c["Hkv"], c["D"]))):
            flat = cache.view(-1, c["Hkv"], c["D"])
            flat[slot] = torch.where(valid.view(-1, 1, 1), new, flat[spare])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "prefix":
        P, n, Q, H, Hkv, D = c["P"], c["n"], c["Q"], c["H"], c["Hkv"], c["D"]
        G, B = H // Hkv, P * n
        kp, vp = _gather(s["k_cache"], s["ptable"]), _gather(s["v_cache"], s["ptable"])
        ks, vs = _gather(s["k_cache"], s["table"]), _gather(s["v_cache"], s["table"])
        q = s["q"].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4) * s["scale"]
        qp = q.reshape(P, n, Hkv, Q * G, D).transpose(1, 2).reshape(P, Hkv, n * Q * G, D)
        tp, ts = torch.arange(kp.shape[2], device=DEV), torch.arange(ks.shape[2], device=DEV)
        seen = (tp < s["plens"].view(P, 1)) & _in_table(s["ptable"], bs)
        sp = (qp @ kp.transpose(2, 3)).masked_fill(~seen.view(P, 1, 1, -1), -math.inf)
        sp = sp.reshape(P, Hkv, n, Q, G, -1).transpose(1, 2).reshape(B, Hkv, Q, G, -1)
        last = s["lens"].view(B, 1) - Q + torch.arange(Q, device=DEV)
        seen = (ts <= last.unsqueeze(2)) & _in_table(s["table"], bs).unsqueeze(1)
        ss = (q.reshape(B, Hkv, Q * G, D) @ ks.transpose(2, 3)).reshape(B, Hkv, Q, G, -1)
        ss = ss.masked_fill(~seen.view(B, 1, Q, 1, -1), -math.inf)
        m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
        m = torch.where(m == -math.inf, 0.0, m)
        sp, ss = torch.exp(sp - m), torch.exp(ss - m)
        total = sp.sum(-1, keepdim=True) + ss.sum(-1, keepdim=True)
        op = sp.reshape(P, n, Hkv, Q * G, -1).transpose(1, 2).reshape(P, Hkv, n * Q * G, -1) @ vp
        op = op.reshape(P, Hkv, n, Q, G, D).transpose(1, 2).reshape(B, Hkv, Q, G, D)
        o = op + (ss.reshape(B, Hkv, Q * G, -1) @ vs).reshape(B, Hkv, Q, G, D)
        o = o / torch.where(total == 0, 1.0, total)
        s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, Q, H, D))
        return s["out"]
    if c["op"] == "accumulate":
        B, Q, H, Hkv, D = c["B"], c["Q"], c["H"], c["Hkv"], c["D"]
        G = H // Hkv
        k = _gather(s["k_cache"], s["table"])
        q = s["q"].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
        p = ((q * s["scale"]) @ k.transpose(2, 3)).reshape(B, Hkv, Q, G, -1)
        t = torch.arange(k.shape[2], device=DEV)
        last = s["lens"].view(B, 1) - Q + torch.arange(Q, device=DEV)
        seen = (t <= last.unsqueeze(2)) & _in_table(s["table"], bs).unsqueeze(1)
        p = p.masked_fill(~seen.view(B, 1, Q, 1, -1), -math.inf)
        m = p.amax(-1, keepdim=True)
        p = torch.exp(p - torch.where(m == -math.inf, 0.0, m))
        total = p.sum(-1, keepdim=True)
        p = (p / torch.where(total == 0, 1.0, total)).reshape(B, Hkv, Q * G, -1)
        o = (p @ _gather(s["v_cache"], s["table"])).reshape(B, Hkv, Q, G, D)
        s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, Q, H, D))
        w = s["weights"] + p.sum(2)
        s["new_weights"].copy_(torch.where(t < s["lens"].view(B, 1, 1), w, s["new_weights"]))
        return s["out"], s["new_weights"]
    B, Hkv, D, budget = c["B"], c["Hkv"], c["D"], c["budget"]
    w, lens = s["weights"], s["lens"].view(B, 1, 1)
    t = torch.arange(w.shape[2], device=DEV)
    held = (t < lens) & _in_table(s["table"], bs).unsqueeze(1)
    rank = torch.where((t < c["sink"]) | (t >= lens - c["recent"]), math.inf, w)
    rank = torch.where(held, rank, -math.inf)
    best = torch.sort(rank, dim=2, descending=True, stable=True).indices
    width = min(budget, w.shape[2])
    n = held.sum(2).clamp(max=budget)                       # [B, 1]
    j = torch.arange(budget, device=DEV)
    first = torch.full((B, Hkv, budget), 1 << 30, dtype=torch.long, device=DEV)
    first[:, :, :width] = best[:, :, :width]
    kept = torch.where(j < n.unsqueeze(2), first, 1 << 30).sort(2).values
    there = kept < (1 << 30)
    s["kept"].copy_(torch.where(there, kept, -1))
    s["new_lens"].copy_(n[:, 0])
    src = torch.where(there, kept, 0)
    slots = s["new_weights"].shape[2]
    s["new_weights"].zero_()
    s["new_weights"][:, :, :budget] = torch.where(there, w.gather(2, src), 0.0)[:, :, :slots]
    # the kept rows of each kv head, in order, into the new pages
    head = torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
    table = s["table"].long().unsqueeze(1).expand(B, Hkv, -1)
    old = table.gather(2, src // bs) * bs + src % bs
    new = s["new_table"].long()[:, j // bs].unsqueeze(1) * bs + j % bs
    new = new.expand(B, Hkv, budget)
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.view(-1, Hkv, D)
        flat[new, head] = torch.where(there.unsqueeze(3), flat[old.clamp(min=0), head],
                                      flat[new, head])
    return s["kept"], s["new_lens"], s["new_weights"], s["k_cache"], s["v_cache"]


# ---- the operators' definitions in 64 bits, one row or token at a time ----

def _tokens_of(cache, row, upto, bs, head):
    """Keys or values [tokens, D] of one kv head at positions 0 .. upto - 1."""
    pages = row[:_pages(upto, bs)].long()
    return cache[pages, :, head].reshape(-1, cache.shape[3])[:upto].double()


def exact(case, seed):
    s = prepare(case, seed)
    bs = case["bs"]
    if case["op"] == "rope":
        H, Q, half = case["H"], case["Q"], case["rot"] // 2
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        first = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        for b, length in enumerate(s["lens"].tolist()):
            angle = torch.stack([s["pos"][a, b].double()[:, None] * s["inv_freq"]
                                 for a in range(case["axes"])])
            angle = angle.gather(0, s["axis"].long().expand(1, Q, half))[0]
            z = torch.polar(torch.ones_like(angle), angle)[:, None]
            y = torch.cat([s["q"][b], s["k"][b]], 1).double()
            turned = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = turned.real, turned.imag
            out[b], k_new = y[:, :H], y[:, H:]
            i = torch.arange(max(0, Q - length), Q, device=DEV)
            at = length - Q + i
            page = s["table"][b].long()[at // bs]
            kc[page, at % bs] = k_new[i]
            vc[page, at % bs] = s["v"][b, i].double()
        return out, kc, vc
    if case["op"] == "prefix":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        G, Q = case["H"] // case["Hkv"], case["Q"]
        slens, plens = s["lens"].tolist(), s["plens"].tolist()
        for h in range(case["Hkv"]):
            for i in range(case["P"]):
                kp = _tokens_of(s["k_cache"], s["ptable"][i], plens[i], bs, h)
                vp = _tokens_of(s["v_cache"], s["ptable"][i], plens[i], bs, h)
                for b in range(i * case["n"], (i + 1) * case["n"]):
                    k = torch.cat([kp, _tokens_of(s["k_cache"], s["table"][b], slens[b], bs, h)])
                    v = torch.cat([vp, _tokens_of(s["v_cache"], s["table"][b], slens[b], bs, h)])
                    q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(Q * G, -1)
                    x = q @ k.T * s["scale"]
                    end = plens[i] + slens[b] - Q + 1 + torch.arange(Q, device=DEV)
                    blind = torch.arange(len(k), device=DEV) >= end.repeat_interleave(G)[:, None]
                    x[blind] = -math.inf
                    out[b, :, h * G:(h + 1) * G] = (torch.softmax(x, 1) @ v).reshape(Q, G, -1)
        return out
    if case["op"] == "accumulate":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        w = s["new_weights"].double()
        G, Q = case["H"] // case["Hkv"], case["Q"]
        for b, length in enumerate(s["lens"].tolist()):
            for h in range(case["Hkv"]):
                k = _tokens_of(s["k_cache"], s["table"][b], length, bs, h)
                v = _tokens_of(s["v_cache"], s["table"][b], length, bs, h)
                q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(Q * G, -1)
                x = q @ k.T * s["scale"]
                end = length - Q + 1 + torch.arange(Q, device=DEV).repeat_interleave(G)
                blind = torch.arange(length, device=DEV) >= end[:, None]
                p = torch.softmax(x.masked_fill(blind, -math.inf), 1).nan_to_num(0.0)
                out[b, :, h * G:(h + 1) * G] = (p @ v).reshape(Q, G, -1)
                w[b, h, :length] = s["weights"][b, h, :length].double() + p.sum(0)
        return out, w
    w64, kept, budget = s["new_weights"].double(), s["kept"], case["budget"]
    kept.fill_(-1)
    for b, length in enumerate(s["lens"].tolist()):
        n = s["new_lens"][b] = min(length, budget)
        for h in range(case["Hkv"]):
            value = s["weights"][b, h, :length].double()
            value[:case["sink"]] = math.inf
            value[max(0, length - case["recent"]):] = math.inf
            take = torch.argsort(-value, stable=True)[:n].sort().values
            kept[b, h, :n] = take.to(torch.int32)
            w64[b, h, :n] = s["weights"][b, h, take].double()
    # (keys and values are copied, not computed)
    return kept, s["new_lens"], w64, None, None
