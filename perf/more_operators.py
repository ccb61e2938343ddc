"""What is measured of attention over the smaller forms of the paged cache.

Two caches, each with the step that fills it and the attention that reads it:

  append8   rotary positions for the new tokens' queries and keys, the keys and
            values written into a cache of 8-bit floats (e4m3) with a scale for
            each page and kv head: a power of two, raised (and the page's older
            tokens with it) when a larger value arrives;
  decode8   paged attention over that cache;
  append_latent  the normalised latent vector of each new token and its turned
            positional part, written into a cache that all heads share, and
            the positional part of every head's query turned;
  decode_latent  paged attention over that cache in its absorbed form: one key a
            token for all heads, whose first part is the value too.

A case names its operator in "op".  ``run`` computes the plain form, or with
``own`` set makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"
E4M3_MAX = 448.0


def listed():
    return [
        # one decode step of a small chat batch: pages partly filled, scales that may rise
        dict(name="append8_step", op="append8", B=8, Q=1, H=32, Hkv=8, D=128, rot=128, axes=1,
             interleaved=False, dtype="bf16", bs=16, past=100),
        # prompts going into the cache
        dict(name="append8_prompt", op="append8", B=4, Q=4001, H=32, Hkv=8, D=128, rot=64, axes=3,
             interleaved=True, dtype="fp16", bs=16, past=37),
        # one short conversation, latency bound
        dict(name="decode8_step", op="decode8", B=1, Q=1, H=32, Hkv=8, D=128, bs=16, dtype="bf16",
             lo=700, hi=700),
        # a batch of very different lengths
        dict(name="decode8_ragged", op="decode8", B=64, Q=1, H=32, Hkv=8, D=128, bs=16,
             dtype="fp16", lo=1, hi=4096),
        # four drafted tokens to verify, one wide kv head
        dict(name="decode8_verify", op="decode8", B=16, Q=4, H=16, Hkv=1, D=256, bs=32,
             dtype="bf16", lo=8001, hi=8192),
        # long contexts, one token each
        dict(name="decode8_long", op="decode8", B=4, Q=1, H=32, Hkv=8, D=128, bs=16, dtype="bf16",
             lo=131072, hi=131072),
        # one decode step of a small batch, a share of the heads on this GPU
        dict(name="append_latent_step", op="append_latent", B=8, Q=1, H=16, R=512, P=64,
             interleaved=True, dtype="bf16", bs=64, past=100),
        # prompts going into the cache
        dict(name="append_latent_prompt", op="append_latent", B=2, Q=8001, H=32, R=512, P=64,
             interleaved=False, dtype="bf16", bs=32, past=37),
        # a few short conversations, latency bound
        dict(name="latent_step", op="decode_latent", B=4, Q=1, H=16, R=512, P=64, bs=64,
             dtype="bf16", lo=300, hi=700),
        # a batch of very different lengths, a share of the heads on this GPU
        dict(name="latent_ragged", op="decode_latent", B=64, Q=1, H=16, R=512, P=64, bs=32,
             dtype="bf16", lo=1, hi=8192),
        # long contexts, every head on this GPU
        dict(name="latent_long", op="decode_latent", B=4, Q=1, H=128, R=512, P=64, bs=64,
             dtype="bf16", lo=65536, hi=65536),
        # two drafted tokens to verify with every head
        dict(name="latent_verify", op="decode_latent", B=32, Q=2, H=128, R=512, P=64, bs=64,
             dtype="fp16", lo=4001, hi=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(["append8", "decode8", "decode8", "append_latent", "decode_latent",
                     "decode_latent"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op in ("append8", "decode8"):
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 8, 16])
        while Hkv * G > 64:
            G //= 2
        c.update(H=Hkv * G, Hkv=Hkv, D=D, bs=rng.choice([16, 32]))
    else:
        c.update(H=_log_int(rng, 1, 128), R=rng.choice([128, 256, 512, 512]), P=64,
                 bs=rng.choice([16, 32, 64, 64]))
    if op == "append8":
        c.update(axes=rng.choice([1, 1, 2, 3]), rot=rng.choice([D, D, D // 2, D // 4]))
    if op in ("append8", "append_latent"):
        c.update(B=_log_int(rng, 1, 128), Q=1 if rng.random() < 0.4 else _log_int(rng, 2, 8000),
                 interleaved=rng.random() < 0.5, past=_log_int(rng, 1, 300))
    else:
        hi = _log_int(rng, 100, 131072)
        c.update(B=_log_int(rng, 1, 128), Q=rng.choice([1, 1, 1, 2, 3, 4, 7]),
                 lo=hi if rng.random() < 0.3 else 1 + hi // 10, hi=hi)
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
        if c["op"] in ("decode8", "decode_latent"):
            width = c["Hkv"] * c["D"] if c["op"] == "decode8" else c["R"]
            if c["B"] * c["Q"] * c["H"] * c["hi"] > 3e8 or c["B"] * c["hi"] * width > 6e8:
                continue
        return c


def _lens(case):
    """Context lengths of a case, the same for every seed (the work depends on
    them): spread evenly over [lo, hi], in a scattered order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * ((b * 7919) % B) // (B - 1) for b in range(B)]


def work(case):
    if case["op"] == "append8":
        tokens, D, H, Hkv = case["B"] * case["Q"], case["D"], case["H"], case["Hkv"]
        pages = case["B"] * _pages(case["Q"], case["bs"])
        return {"bytes": tokens * D * (4 * H + 6 * Hkv) + tokens * 4 * case["axes"]
                + case["rot"] // 2 * 12 + case["B"] * 4 + pages * (8 * Hkv + 4),
                "flops": tokens * case["rot"] * 3 * (H + Hkv)}
    if case["op"] == "append_latent":
        tokens, W = case["B"] * case["Q"], case["R"] + case["P"]
        return {"bytes": tokens * (4 * W + 4 * case["H"] * case["P"] + 4) + case["R"] * 2
                + case["P"] * 4 + case["B"] * 4 + 4 * _pages(tokens, case["bs"]),
                "flops": tokens * (4 * case["R"] + 3 * case["P"] * (case["H"] + 1))}
    tokens, rows = sum(_lens(case)), case["Q"] * case["H"]
    if case["op"] == "decode8":
        D, Hkv = case["D"], case["Hkv"]
        return {"bytes": tokens * Hkv * D * 2 + case["B"] * rows * D * 4
                + tokens // case["bs"] * (4 + 8 * Hkv),
                "flops": 4 * D * rows * tokens}
    R, P = case["R"], case["P"]
    return {"bytes": tokens * (R + P) * 2 + case["B"] * rows * (2 * R + P) * 2
            + 4 * (tokens // case["bs"]),
            "flops": 2 * (2 * R + P) * rows * tokens}


def _pages(tokens, bs):
    return (tokens + bs - 1) // bs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _tables(lens, bs, g):
    """Block tables (-1 padded) of sequences of these lengths over scattered
    pages, and how many pages there are."""
    pages = [_pages(t, bs) for t in lens]
    total = sum(pages)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _scale_of(amax):
    """The smallest power of two that brings amax to 448 or below, in [2^-60, 2^60]."""
    mantissa, exponent = torch.frexp(amax / E4M3_MAX)
    exponent = torch.where(mantissa == 0.5, exponent - 1, exponent)
    exponent = torch.where(amax == 0, -60, exponent).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), exponent)


def _cache8(blocks, bs, Hkv, D, g):
    """A filled 8-bit cache: pages of uneven magnitude, codes and scales."""
    x = torch.randn((blocks, bs, Hkv, D), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((blocks, 1, Hkv, 1), generator=g, device=DEV))
    scale = _scale_of(x.abs().amax((1, 3)))
    return (x / scale.view(blocks, 1, Hkv, 1)).to(torch.float8_e4m3fn), scale


def _positions(case, g):
    """Lengths (with the new tokens; the last sequence of a batch is padded: its
    first tokens lie before its start) and tables of an append."""
    B, Q = case["B"], case["Q"]
    lens = [case["past"] + Q + 3 * b for b in range(B)]
    if B > 1:
        lens[-1] = max(1, Q // 2)
    table, pool = _tables(lens, case["bs"], g)
    at = torch.tensor(lens, device=DEV).view(B, 1) - Q + torch.arange(Q, device=DEV)
    return torch.tensor(lens, dtype=torch.int32, device=DEV), table, pool, at


def prepare(case, seed):
    g = _gen(seed)
    dt, bs, B, Q, H = DTYPES[case["dtype"]], case["bs"], case["B"], case["Q"], case["H"]
    s = {"case": case}
    if case["op"] == "append8":
        D, Hkv, A = case["D"], case["Hkv"], case["axes"]
        lens, table, pool, at = _positions(case, g)
        qkv = _normal((B, Q, H + 2 * Hkv, D), dt, g)  # one projection's output
        half = case["rot"] // 2
        inv_freq = 1e4 ** (-torch.arange(half, dtype=torch.float64, device=DEV) * 2 / case["rot"])
        axis = (torch.arange(half, device=DEV) % A).to(torch.int32)
        pos = torch.stack([at if a == 0 else (at // (7 * a)) % 97 + 1000 * a for a in range(A)])
        kc, ks = _cache8(pool + 1, bs, Hkv, D, g)
        vc, vs = _cache8(pool + 1, bs, Hkv, D, g)
        s.update(q=qkv[:, :, :H], k=qkv[:, :, H:H + Hkv], v=qkv[:, :, H + Hkv:],
                 q_out=torch.zeros((B, Q, H, D), dtype=dt, device=DEV), k_cache=kc, v_cache=vc,
                 k_scales=ks, v_scales=vs, pos=pos.to(torch.int32).contiguous(),
                 inv_freq=inv_freq, axis=axis, table=table, lens=lens)
    elif case["op"] == "append_latent":
        R, P = case["R"], case["P"]
        lens, table, pool, at = _positions(case, g)
        # the outputs of two projections: the rest of a row goes elsewhere
        new = _normal((B, Q, R + P + 256), dt, g)[:, :, :R + P]
        q = _normal((B, Q, H, 128 + P), dt, g)[..., 128:]
        q_all = torch.zeros((B, Q, H, R + P), dtype=dt, device=DEV)
        inv_freq = 1e4 ** (-torch.arange(P // 2, dtype=torch.float64, device=DEV) * 2 / P)
        s.update(q=q, new=new, q_out=q_all[..., R:], cache=_normal((pool + 1, bs, R + P), dt, g),
                 norm=(1 + 0.2 * torch.randn(R, generator=g, device=DEV)).to(dt), eps=1e-6,
                 pos=at.to(torch.int32).contiguous(), inv_freq=inv_freq, table=table, lens=lens)
    elif case["op"] == "decode8":
        D, Hkv = case["D"], case["Hkv"]
        lens = _lens(case)
        table, pool = _tables(lens, bs, g)
        kc, ks = _cache8(pool, bs, Hkv, D, g)
        vc, vs = _cache8(pool, bs, Hkv, D, g)
        s.update(q=_normal((B, Q, H, D), dt, g),
                 out=torch.zeros((B, Q, H, D), dtype=dt, device=DEV), k_cache=kc, v_cache=vc,
                 k_scales=ks, v_scales=vs, table=table, scale=D ** -0.5,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    else:
        R, P = case["R"], case["P"]
        lens = _lens(case)
        table, pool = _tables(lens, bs, g)
        s.update(q=_normal((B, Q, H, R + P), dt, g),
                 out=torch.zeros((B, Q, H, R), dtype=dt, device=DEV),
                 cache=_normal((pool, bs, R + P), dt, g), table=table, scale=(R // 4 + P) ** -0.5,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if own:
        import paged_kv_attention_08_gb300 as pa
        if "inv_freq" in s:
            s["phases"] = pa.rope_phases(s["inv_freq"])
        elif case["op"] == "decode8":
            need = pa.workspace_size_kv8(s["q"], s["k_cache"], s["table"], dt, case["hi"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        else:
            need = pa.workspace_size_latent(s["q"], s["cache"], case["R"], s["table"], case["hi"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import paged_kv_attention_08_gb300 as pa
    c = s["case"]
    if c["op"] == "append8":
        pa.rope_append_kv8(s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                           s["q"], s["k"], s["v"], s["pos"], s["phases"], s["axis"], s["table"],
                           s["lens"], interleaved=c["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if c["op"] == "append_latent":
        pa.rope_append_latent(s["q_out"], s["cache"], s["q"], s["new"], s["norm"], s["pos"],
                              s["phases"], s["table"], s["lens"], eps=s["eps"],
                              interleaved=c["interleaved"])
        return s["q_out"], s["cache"]
    if c["op"] == "decode8":
        pa.decode_kv8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                      s["table"], s["lens"], s["scale"], c["hi"], workspace=s["workspace"])
        return s["out"]
    pa.decode_latent(s["out"], s["q"], s["cache"], s["table"], s["lens"], s["scale"], c["hi"],
                     workspace=s["workspace"])
    return s["out"]


def _turn(x, cos, sin, interleaved):
    """The first 2 * half elements of each head turned (cos, sin: [..., half])."""
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _slots(s, Q, bs, blocks):
    """Flat cache slot of each new token [B * Q] and whether it has one; those
    that have none name the spare last block."""
    at = s["lens"].long().view(-1, 1) - Q + torch.arange(Q, device=DEV)
    page = s["table"].long().gather(1, at.clamp(min=0) // bs)
    valid = ((at >= 0) & (page >= 0)).reshape(-1)
    spare = (blocks - 1) * bs
    return torch.where(valid, (page * bs + at.clamp(min=0) % bs).reshape(-1), spare), valid


def _append8_plain(s, cache, scales, x, slot, valid, Q, bs):
    """New tokens x [B * Q, Hkv, D] (32 bits) into the codes and scales."""
    blocks, _, Hkv, D = cache.shape
    page = slot // bs
    amax = torch.where(valid.view(-1, 1), x.abs().amax(2), 0.0)
    new = torch.zeros((blocks, Hkv), device=DEV).scatter_reduce_(
        0, page.view(-1, 1).expand(-1, Hkv), amax, "amax")
    first = torch.full((blocks,), bs, device=DEV).scatter_reduce_(
        0, page, torch.where(valid, slot % bs, bs), "amin")
    scale = torch.where((first == 0).view(-1, 1), _scale_of(new),
                        torch.maximum(scales, _scale_of(new)))
    scale = torch.where((first == bs).view(-1, 1), scales, scale)
    # the older tokens of each sequence's first page, on the scale that it has now
    head = slot.view(-1, Q)[torch.arange(slot.numel() // Q, device=DEV),
                            valid.view(-1, Q).long().argmax(1)] // bs
    old = cache[head].float() * (scales[head] / scale[head]).unsqueeze(1).unsqueeze(3)
    keep = (torch.arange(bs, device=DEV) < first[head].view(-1, 1)) & (first[head] < bs).view(-1, 1)
    codes = cache.view(torch.uint8)
    codes[head] = torch.where(keep.view(-1, bs, 1, 1), old.to(torch.float8_e4m3fn).view(torch.uint8),
                              codes[head])
    flat = codes.view(-1, Hkv, D)
    q = (x / scale[page].unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
    flat[slot] = torch.where(valid.view(-1, 1, 1), q, flat[(blocks - 1) * bs])
    scales.copy_(scale)


def _softmax_rows(p):
    """Softmax over the last dimension of scores with -inf where masked; a row
    that is masked whole has no weight."""
    m = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _seen(s, Q, tokens, bs):
    """[B, Q, tokens]: which tokens each query token attends to."""
    last = s["lens"].view(-1, 1) - Q + torch.arange(Q, device=DEV)
    held = (s["table"] >= 0).repeat_interleave(bs, dim=1)
    return (torch.arange(tokens, device=DEV) <= last.unsqueeze(2)) & held.unsqueeze(1)


def _gather8(cache, scales, table):
    """[B, Hkv, tokens, D]: the values that the pages of a table hold."""
    t = table.clamp(min=0).long()
    x = cache.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
    x *= scales[t].unsqueeze(2).unsqueeze(4)
    B, m, bs, Hkv, D = x.shape
    return x.reshape(B, m * bs, Hkv, D).permute(0, 2, 1, 3)


def _run_plain(s):
    c = s["case"]
    B, Q, H, bs = c["B"], c["Q"], c["H"], c["bs"]
    if c["op"] == "append8":
        # angles in 64 bits: far positions
        ang = s["pos"].double()[s["axis"].long()].permute(1, 2, 0) * s["inv_freq"]
        cos, sin = ang.cos().float().unsqueeze(2), ang.sin().float().unsqueeze(2)
        s["q_out"].copy_(_turn(s["q"].float(), cos, sin, c["interleaved"]))
        k = _turn(s["k"].float(), cos, sin, c["interleaved"]).reshape(B * Q, c["Hkv"], c["D"])
        slot, valid = _slots(s, Q, bs, s["k_cache"].shape[0])
        _append8_plain(s, s["k_cache"], s["k_scales"], k, slot, valid, Q, bs)
        _append8_plain(s, s["v_cache"], s["v_scales"],
                       s["v"].float().reshape(B * Q, c["Hkv"], c["D"]), slot, valid, Q, bs)
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if c["op"] == "append_latent":
        R, P = c["R"], c["P"]
        ang = s["pos"].double().unsqueeze(2) * s["inv_freq"]
        cos, sin = ang.cos().float(), ang.sin().float()
        s["q_out"].copy_(_turn(s["q"].float(), cos.unsqueeze(2), sin.unsqueeze(2), c["interleaved"]))
        x = s["new"][..., :R].float()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["norm"].float()
        k = _turn(s["new"][..., R:].float(), cos, sin, c["interleaved"])
        row = torch.cat([x, k], -1).to(s["cache"].dtype).reshape(B * Q, R + P)
        slot, valid = _slots(s, Q, bs, s["cache"].shape[0])
        flat = s["cache"].view(-1, R + P)
        flat[slot] = torch.where(valid.view(-1, 1), row, flat[(s["cache"].shape[0] - 1) * bs])
        return s["q_out"], s["cache"]
    if c["op"] == "decode8":
        Hkv, D = c["Hkv"], c["D"]
        G = H // Hkv
        k = _gather8(s["k_cache"], s["k_scales"], s["table"])
        q = s["q"].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
        p = ((q * s["scale"]) @ k.transpose(2, 3)).reshape(B, Hkv, Q, G, -1)
        seen = _seen(s, Q, k.shape[2], bs)
        p = _softmax_rows(p.masked_fill(~seen.view(B, 1, Q, 1, -1), -math.inf))
        o = p.reshape(B, Hkv, Q * G, -1) @ _gather8(s["v_cache"], s["v_scales"], s["table"])
        s["out"].copy_(o.reshape(B, Hkv, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, H, D))
        return s["out"]
    R, W = c["R"], c["R"] + c["P"]
    k = s["cache"][s["table"].clamp(min=0).long()].reshape(B, -1, W).float()
    p = (s["q"].float().reshape(B, Q * H, W) * s["scale"]) @ k.transpose(1, 2)
    seen = _seen(s, Q, k.shape[1], bs)
    p = _softmax_rows(p.reshape(B, Q, H, -1).masked_fill(~seen.unsqueeze(2), -math.inf))
    s["out"].copy_((p.reshape(B, Q * H, -1) @ k[..., :R]).reshape(B, Q, H, R))
    return s["out"]


# ---- the operators' definitions in 64 bits, one sequence or page at a time ----

def _exact_turn(x, angle, interleaved):
    """x [tokens, heads, width] turned in place by angle [tokens, pairs], as complex numbers."""
    half = angle.shape[1]
    first = torch.arange(half, device=DEV) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    turned = torch.complex(x[..., first], x[..., second]) * z
    x[..., first], x[..., second] = turned.real, turned.imag
    return x


def _exact_append8(codes, scales, row, x, start, bs):
    """x [tokens, Hkv, D] from position `start` on into values / scale and scales."""
    at = 0
    while at < len(x):
        slot = (start + at) % bs
        n = min(bs - slot, len(x) - at)
        page = int(row[(start + at) // bs])
        top = x[at:at + n].abs().amax((0, 2)) / E4M3_MAX
        scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -60)))).clamp(max=2.0 ** 60)
        if slot:
            scale = torch.maximum(scale, scales[page])
            codes[page, :slot] *= (scales[page] / scale).view(1, -1, 1)
        codes[page, slot:slot + n] = x[at:at + n] / scale.view(1, -1, 1)
        scales[page] = scale
        at += n


def _exact_attention(q, k, v, scale, length, rows_per_token):
    """Rows (query token, head) of one sequence over its tokens, causal over the query tokens."""
    Q = q.shape[0] // rows_per_token
    x = q @ k.T * scale
    end = length - Q + 1 + torch.arange(Q, device=DEV).repeat_interleave(rows_per_token)
    blind = torch.arange(length, device=DEV) >= end[:, None]
    return torch.softmax(x.masked_fill(blind, -math.inf), 1).nan_to_num(0.0) @ v


def exact(case, seed):
    s = prepare(case, seed)
    Q, H, bs = case["Q"], case["H"], case["bs"]
    lens = s["lens"].tolist()
    if case["op"] == "append8":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        ks, vs = s["k_scales"].double(), s["v_scales"].double()
        table = s["table"].cpu()
        for b, length in enumerate(lens):
            angle = s["pos"][:, b].double()[s["axis"].long()].T * s["inv_freq"]
            y = _exact_turn(torch.cat([s["q"][b], s["k"][b]], 1).double(), angle,
                            case["interleaved"])
            out[b] = y[:, :H]
            skip = max(0, Q - length)
            _exact_append8(kc, ks, table[b], y[skip:, H:], length - Q + skip, bs)
            _exact_append8(vc, vs, table[b], s["v"][b, skip:].double(), length - Q + skip, bs)
        return out, kc, vc, ks, vs
    if case["op"] == "append_latent":
        R = case["R"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        cache = s["cache"].double()
        for b, length in enumerate(lens):
            angle = s["pos"][b].double()[:, None] * s["inv_freq"]
            out[b] = _exact_turn(s["q"][b].double(), angle, case["interleaved"])
            x = s["new"][b].double()
            norm = torch.linalg.vector_norm(x[:, :R], dim=1, keepdim=True) ** 2 / R + s["eps"]
            x[:, :R] *= s["norm"].double() / norm.sqrt()
            x[:, R:] = _exact_turn(x[:, None, R:].clone(), angle, case["interleaved"])[:, 0]
            i = torch.arange(max(0, Q - length), Q, device=DEV)
            at = length - Q + i
            cache[s["table"][b].long()[at // bs], at % bs] = x[i]
        return out, cache
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b, length in enumerate(lens):
        pages = s["table"][b, :_pages(length, bs)].long()
        if case["op"] == "decode_latent":
            c = s["cache"][pages].flatten(0, 1)[:length].double()
            out[b] = _exact_attention(s["q"][b].double().flatten(0, 1), c, c[:, :case["R"]],
                                      s["scale"], length, H).reshape(Q, H, -1)
            continue
        G, D = H // case["Hkv"], case["D"]
        for h in range(case["Hkv"]):
            kv = [(x.view(torch.uint8)[pages, :, h].view(torch.float8_e4m3fn).double()
                   * y[pages, h].double().view(-1, 1, 1)).flatten(0, 1)[:length]
                  for x, y in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"]))]
            q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(Q * G, D)
            out[b, :, h * G:(h + 1) * G] = _exact_attention(q, *kv, s["scale"], length,
                                                            G).reshape(Q, G, D)
    return out
