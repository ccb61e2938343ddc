"""Plain 64-bit definitions of the serving-step operators, on the CPU, one
token or row at a time, and the seeded inputs that their tests share."""
import math

import torch


def tables(lens, bs, seed, width=0, first=0, spare=2):
    """Scattered block tables (-1 padded) of sequences of these lengths, on
    pages first, first + 1, ...; returns (table, pool size)."""
    g = torch.Generator().manual_seed(seed)
    pages = [(max(t, 0) + bs - 1) // bs for t in lens]
    order = torch.randperm(sum(pages) + spare, generator=g) + first
    table = torch.full((len(lens), max(1, width, max(pages))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return table, first + sum(pages) + spare


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def slot(table_row, t, bs, num_blocks):
    """(block, slot in block) of cache position t, or None."""
    if t < 0 or t >= len(table_row) * bs:
        return None
    e = int(table_row[t // bs])
    return (e, t % bs) if 0 <= e < num_blocks else None


def rope_append(q, k_cache, v_cache, k_new, v_new, positions, inv_freq, axes, table, lens,
                interleaved):
    """(q_out, k_cache, v_cache) in float64 of pa.rope_append_kv's arguments."""
    B, Q, H, D = q.shape
    half, bs = len(inv_freq), k_cache.shape[1]
    kc, vc = k_cache.double().clone(), v_cache.double().clone()
    out = q.double().clone()
    j = torch.arange(half)
    first, second = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    ok = (axes >= 0) & (axes < positions.shape[0])

    def turn(x, b, i):
        y = x.double().clone()
        pos = positions[axes.clamp(0, positions.shape[0] - 1).long(), b, i].double()
        a = torch.where(ok, pos * inv_freq, torch.zeros(()).double())
        u, v = x[:, first].double(), x[:, second].double()
        y[:, first] = u * a.cos() - v * a.sin()
        y[:, second] = u * a.sin() + v * a.cos()
        return y

    for b in range(B):
        for i in range(Q):
            out[b, i] = turn(q[b, i], b, i)
            at = slot(table[b], max(int(lens[b]), 0) - Q + i, bs, len(k_cache))
            if at is not None:
                kc[at] = turn(k_new[b, i], b, i)
                vc[at] = v_new[b, i].double()
    return out, kc, vc


def evict(k_cache, v_cache, weights, table, lens, new_table, budget, sink, recent):
    """(k_cache, v_cache, new_weights, new_lens, kept) of pa.evict_kv."""
    B, Hkv, _ = weights.shape
    NB, bs = k_cache.shape[:2]
    kc, vc = k_cache.clone(), v_cache.clone()
    nw = torch.zeros((B, Hkv, new_table.shape[1] * bs))
    nl = torch.zeros((B,), dtype=torch.int32)
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    for b in range(B):
        T = min(max(int(lens[b]), 0), table.shape[1] * bs)
        held = [t for t in range(T) if slot(table[b], t, bs, NB) is not None]
        must = [t for t in held if t < sink or t >= T - recent]
        free = [t for t in held if not (t < sink or t >= T - recent)]
        nl[b] = min(len(held), budget)
        for h in range(Hkv):
            w = weights[b, h].double().tolist()
            free.sort(key=lambda t: (0, -w[t], t) if w[t] == w[t] else (1, 0.0, t))
            take = sorted(must + free[:int(nl[b]) - len(must)])
            for j, t in enumerate(take):
                kept[b, h, j] = t
                nw[b, h, j] = weights[b, h, t]
                src, dst = slot(table[b], t, bs, NB), slot(new_table[b], j, bs, NB)
                if dst is not None:
                    kc[dst][h] = k_cache[src][h]
                    vc[dst][h] = v_cache[src][h]
    return kc, vc, nw, nl, kept


def _rows(cache, table_row, T, h):
    """Values [tokens, D] of one kv head and the positions they are at."""
    bs = cache.shape[1]
    ts = [t for t in range(min(T, len(table_row) * bs)) if slot(table_row, t, bs, len(cache))]
    idx = [slot(table_row, t, bs, len(cache)) for t in ts]
    x = torch.stack([cache[e, s, h] for e, s in idx]).double() if idx else \
        torch.zeros((0, cache.shape[3])).double()
    return x, torch.tensor(ts, dtype=torch.long)


def _softmax(x, seen):
    """Rows of probabilities over the seen columns; zeros where there are none."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(1, keepdim=True) if x.shape[1] else torch.full((len(x), 1), -math.inf).double()
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros(()).double(), m))
    p = torch.where(seen, p, torch.zeros(()).double())
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, torch.ones(()).double(), total)


def accumulate(weights, q, k_cache, v_cache, table, lens, scale):
    """(out, new weights) in float64 of pa.decode_accumulate (q [B, Q, H, D]);
    entries from the reachable length on are those of `weights`."""
    B, Q, H, D = q.shape
    Hkv, bs = k_cache.shape[2], k_cache.shape[1]
    G = H // Hkv
    out, w = torch.zeros(q.shape).double(), weights.double().clone()
    for b in range(B):
        ctx = max(int(lens[b]), 0)
        for h in range(Hkv):
            k, ts = _rows(k_cache, table[b], ctx, h)
            v, _ = _rows(v_cache, table[b], ctx, h)
            x = q[b, :, h * G:(h + 1) * G].double().reshape(Q * G, D) @ k.T * scale
            end = ctx - Q + 1 + torch.arange(Q).repeat_interleave(G)
            p = _softmax(x, ts < end[:, None])
            out[b, :, h * G:(h + 1) * G] = (p @ v).reshape(Q, G, D)
            w[b, h, ts] += p.sum(0)
    return out, w


def shared_prefix(q, k_cache, v_cache, prefix_tables, prefix_lens, table, lens, scale):
    """Attention of pa.decode_shared_prefix in float64: the prefix and the own
    tokens of a sequence, one after the other (q [B, Q, H, D])."""
    B, Q, H, D = q.shape
    Hkv, bs = k_cache.shape[2], k_cache.shape[1]
    G, n = H // Hkv, B // len(prefix_tables)
    out = torch.zeros(q.shape).double()
    for b in range(B):
        i = b // n
        plen = min(max(int(prefix_lens[i]), 0), prefix_tables.shape[1] * bs)
        ctx = max(int(lens[b]), 0)
        for h in range(Hkv):
            kp, tp = _rows(k_cache, prefix_tables[i], plen, h)
            vp, _ = _rows(v_cache, prefix_tables[i], plen, h)
            ks, ts = _rows(k_cache, table[b], ctx, h)
            vs, _ = _rows(v_cache, table[b], ctx, h)
            x = q[b, :, h * G:(h + 1) * G].double().reshape(Q * G, D) @ torch.cat([kp, ks]).T * scale
            end = plen + ctx - Q + 1 + torch.arange(Q).repeat_interleave(G)
            p = _softmax(x, torch.cat([tp, plen + ts]) < end[:, None])
            out[b, :, h * G:(h + 1) * G] = (p @ torch.cat([vp, vs])).reshape(Q, G, D)
    return out


def score_error(q, k_cache, scale):
    """Bound on the error, in log2 units, of one score formed from these 16-bit
    values in fp32: exact products, D sums and two scalings of 2^-23 each, of
    terms of at most |q| |k| in all."""
    D = q.shape[-1]
    biggest = q.double().norm(dim=-1).max() * torch.nan_to_num(k_cache.double()).norm(dim=-1).max()
    return (D + 4) * 2.0 ** -23 * biggest.item() * scale * 1.4427


def weight_slack(q, k_cache, scale, tokens):
    """Relative error of one softmax weight 2^(s - m) / l: the score's and the
    normaliser's scores' errors (times ln 2), the normaliser's sum over the
    tokens, and the exponentials (2^-22 each, of the weight and of l)."""
    return 2 * 0.6932 * score_error(q, k_cache, scale) + (tokens + 8) * 2.0 ** -23


def out_slack(q, k_cache, v_cache, scale, tokens):
    """Absolute error of an attention output before its own rounding: every
    weight's relative error, twice (numerator and normaliser), of the largest
    value; the weights' own rounding on the way into the second product: fp16
    once (2^-11), bf16 as a high and a low part (2^-16)."""
    rounding = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -16
    return (2 * weight_slack(q, k_cache, scale, tokens) + 2 * rounding) * \
        torch.nan_to_num(v_cache.double()).abs().max().item()


def close_out(got, want, slack):
    assert torch.isfinite(got).all(), "non-finite output"
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs() - half * want.abs() - slack
    assert err.max().item() <= 0, f"{err.max().item():.3e} over the bound, slack {slack:.3e}"
