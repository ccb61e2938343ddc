"""Plain 64-bit definitions of the operators on the 8-bit and the latent cache,
on the CPU, and the seeded inputs that their tests share."""
import math

import torch

import step_reference as ref

E4M3 = torch.float8_e4m3fn


def scale_for(amax):
    """The smallest power of two s with amax <= 448 s, in [2^-60, 2^60]."""
    if amax == 0:
        return 2.0 ** -60
    k = math.ceil(math.log2(amax / 448)) - 1
    while amax > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** max(-60, min(60, k))


def codes_of(x, scale):
    """e4m3 codes of x / scale, NaN for what they cannot hold."""
    y = x.double() / scale
    y = torch.where(y.abs() <= 448, y, torch.full_like(y, math.nan))
    return y.float().to(E4M3)


def cache8(blocks, bs, Hkv, D, seed, spread=0.5):
    """(codes, scales) of a filled 8-bit cache whose pages differ in magnitude."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((blocks, bs, Hkv, D), generator=g)
    x = x * torch.exp(spread * torch.randn((blocks, 1, Hkv, 1), generator=g))
    scales = torch.empty((blocks, Hkv))
    for e in range(blocks):
        for h in range(Hkv):
            scales[e, h] = scale_for(x[e, :, h].abs().max().item())
    return (x / scales.view(blocks, 1, Hkv, 1)).to(E4M3), scales


def values8(codes, scales):
    return codes.double() * scales.double().view(scales.shape[0], 1, scales.shape[1], 1)


def turned(x, angle, interleaved):
    """x [heads, width] in float64 with its first 2 * len(angle) elements turned."""
    y, half = x.double().clone(), len(angle)
    j = torch.arange(half)
    first, second = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    u, v = x[:, first].double(), x[:, second].double()
    y[:, first] = u * angle.cos() - v * angle.sin()
    y[:, second] = u * angle.sin() + v * angle.cos()
    return y


def append8(q, k_cache, v_cache, k_scales, v_scales, k_new, v_new, positions, inv_freq, axes,
            table, lens, interleaved):
    """What pa.rope_append_kv8 is to leave: q_out (float64), the caches' codes as
    float64 values of code * scale before their rounding, the scales, and which
    codes the call rounds."""
    B, Q, H, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    out = torch.empty(q.shape).double()
    res = [values8(k_cache, k_scales), values8(v_cache, v_scales), k_scales.clone(),
           v_scales.clone()]
    rounded = [torch.zeros(k_cache.shape, dtype=torch.bool) for _ in range(2)]
    ok = (axes >= 0) & (axes < positions.shape[0])
    for b in range(B):
        pages = {}
        for i in range(Q):
            pos = positions[axes.clamp(0, positions.shape[0] - 1).long(), b, i].double()
            angle = torch.where(ok, pos * inv_freq, torch.zeros(()).double())
            out[b, i] = turned(q[b, i], angle, interleaved)
            at = ref.slot(table[b], max(int(lens[b]), 0) - Q + i, bs, NB)
            if at is not None:
                pages.setdefault(at[0], []).append(
                    (at[1], turned(k_new[b, i], angle, interleaved), v_new[b, i].double()))
        for e, new in pages.items():
            first = min(s for s, _, _ in new)
            for which in range(2):
                for h in range(Hkv):
                    x = torch.stack([n[1 + which][h] for n in new])
                    finite = x[torch.isfinite(x)].abs()
                    s = scale_for(finite.max().item() if finite.numel() else 0.0)
                    old = float((k_scales, v_scales)[which][e, h])
                    if first > 0:
                        s = max(s, old)
                        if s > old:
                            rounded[which][e, :first, h] = True
                    res[2 + which][e, h] = s
                for slot, *kv in new:
                    res[which][e, slot] = kv[which]
                    rounded[which][e, slot] = True
    return (out, *res, rounded)


def append_latent(q, cache, latent_new, norm_weight, eps, positions, inv_freq, table, lens,
                  interleaved):
    """(q_out, cache) in float64 of pa.rope_append_latent's arguments."""
    B, Q, H, P = q.shape
    NB, bs, W = cache.shape
    R = W - P
    out, c = torch.empty(q.shape).double(), cache.double().clone()
    for b in range(B):
        for i in range(Q):
            angle = positions[b, i].double() * inv_freq
            out[b, i] = turned(q[b, i], angle, interleaved)
            at = ref.slot(table[b], max(int(lens[b]), 0) - Q + i, bs, NB)
            if at is None:
                continue
            x = latent_new[b, i].double()
            y = x[:R]
            if norm_weight is not None:
                y = y / torch.sqrt((y * y).mean() + eps) * norm_weight.double()
            c[at] = torch.cat([y, turned(x[None, R:], angle, interleaved)[0]])
    return out, c


def attention(q, k, v, table, lens, scale):
    """Attention of pa.decode_multi in float64 over caches k, v [NB, bs, Hkv, *]
    of values (q [B, Q, H, D])."""
    B, Q, H, D = q.shape
    Hkv, bs = k.shape[2], k.shape[1]
    G = H // Hkv
    out = torch.zeros((B, Q, H, v.shape[3])).double()
    for b in range(B):
        ctx = max(int(lens[b]), 0)
        for h in range(Hkv):
            kk, ts = ref._rows(k, table[b], ctx, h)
            vv, _ = ref._rows(v, table[b], ctx, h)
            x = q[b, :, h * G:(h + 1) * G].double().reshape(Q * G, D) @ kk.T * scale
            end = ctx - Q + 1 + torch.arange(Q).repeat_interleave(G)
            p = ref._softmax(x, ts < end[:, None])
            out[b, :, h * G:(h + 1) * G] = (p @ vv).reshape(Q, G, -1)
    return out


def attention_slack(q, k, v, scale, tokens, rounding):
    """Absolute error of an attention output before its own rounding: every
    weight's relative error (step_reference.weight_slack, with two more products
    a score for the page's scale and the query's), twice (numerator and
    normaliser), of the largest value; and the weights' `rounding` on the way
    into the second product, twice likewise."""
    two = 2 * 2 * 2.0 ** -23 * 0.6932 * 1.4427 * scale * \
        (q.double().norm(dim=-1).max() * torch.nan_to_num(k.double()).norm(dim=-1).max()).item()
    return (2 * (ref.weight_slack(q, k, scale, tokens) + two) + 2 * rounding) * \
        torch.nan_to_num(v.double()).abs().max().item()
