"""Plain 64-bit references of the serving-step operators (tests only)."""
import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn


def values(codes, scales):
    """The values a block-scaled cache stands for, in binary64: [num_blocks, H_kv, block_size, D]."""
    return codes.view(FP8).double() * scales.double()[:, :, None, None]


def attention(q, kc, vc, ks, vs, table, lens, start, scale, window=0, sinks=None):
    """(out, lse, weighted, reach): binary64 attention of each request's tokens;
    `weighted` is sum p |V| (what the weights' rounding is relative to) and
    `reach` the largest scale * sum |q| |K| of a row's visible keys. Rows that
    no request has are NaN."""
    T, H, D = q.shape
    nb, hk, bs, _ = kc.shape
    G = H // hk
    out = torch.full((T, H, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    wsum = torch.zeros((T, H, D), dtype=torch.float64)
    reach = torch.zeros((T, H), dtype=torch.float64)
    kval, vval = values(kc, ks), values(vc, vs)
    qd = q.double()
    for b in range(len(lens)):
        q0, q1 = int(start[b]), int(start[b + 1])
        n = min(max(int(lens[b]), 0), table.shape[1] * bs)
        if q1 <= q0:
            continue
        pages = table[b, :(n + bs - 1) // bs].long()
        good = (pages >= 0) & (pages < nb)
        safe = pages.clamp(0, max(nb - 1, 0))
        there = good.repeat_interleave(bs)[:n]
        for t in range(q0, q1):
            p = n - (q1 - q0) + (t - q0)
            j = torch.arange(n)
            see = (j <= p) & there
            if window > 0:
                see &= j > p - window
            for h in range(H):
                kk = kval[safe, h // G].reshape(-1, D)[:n][see]
                vv = vval[safe, h // G].reshape(-1, D)[:n][see]
                s = (kk @ qd[t, h]) * scale
                if sinks is not None:
                    z = torch.logsumexp(torch.cat([s, sinks[h].double().reshape(1)]), 0)
                elif len(s):
                    z = torch.logsumexp(s, 0)
                else:
                    z = torch.tensor(-math.inf, dtype=torch.float64)
                lse[t, h] = z
                if len(s):
                    w = torch.exp(s - z)
                    out[t, h] = w @ vv
                    wsum[t, h] = w @ vv.abs()
                    reach[t, h] = (kk.abs() @ qd[t, h].abs()).max() * scale
                else:
                    out[t, h] = 0.0
    return out, lse, wsum, reach


def block_tables(lens, ql, held, table, ring, state, bs, T):
    """smla_build_block_tables, one entry at a time."""
    table, ring = table.copy(), ring.copy()
    head, count = int(state[0]), int(state[1])
    cap, B, width = len(ring), len(lens), table.shape[1]
    need = [-(-max(int(n), 0) // bs) for n in lens]
    lacking = sum(max(0, n - width) for n in need)
    taken = sum(max(0, n - int(h)) for n, h in zip(need, held))
    lacking += max(0, taken - count)
    given, k = 0, 0
    held_out = [int(h) for h in held]
    if lacking == 0:
        behind = []
        for b in range(B):
            for j in range(held_out[b], need[b]):
                table[b, j] = ring[(head + k) % cap]
                k += 1
            behind += [int(table[b, j]) for j in range(need[b], held_out[b])]
            held_out[b] = need[b]
        for x in behind:
            ring[(head + count + given) % cap] = x
            given += 1
    pos = np.zeros(T, np.int64)
    slots = np.full(T, -1, np.int64)
    req = np.full(T, -1, np.int32)
    start = [0]
    for b in range(B):
        n = max(int(lens[b]), 0)
        q = min(max(int(ql[b]), 0), n)
        for i in range(q):
            t = start[-1] + i
            if t < T:
                p = n - q + i
                pos[t], req[t] = p, b
                if p // bs < held_out[b]:
                    slots[t] = int(table[b, p // bs]) * bs + p % bs
        start.append(start[-1] + q)
    return dict(query_start=np.array(start), positions=pos, slot_mapping=slots, token_request=req, table=table,
                ring=ring, blocks_held=np.array(held_out),
                ring_state=np.array([(head + k) % cap, count - k + given]),
                counts=np.array([start[-1], k, given, lacking]))


def frequencies(rot, base, scaling, factor, orig, fast, slow):
    """Radians per position of each pair, and the scaling's own attention factor."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        c = [rot * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
        lo, hi = max(math.floor(c[0]), 0), min(math.ceil(c[1]), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        f = f / factor * r + f * (1 - r)
        return f, 0.1 * math.log(factor) + 1
    return f, 1.0


def append(k, slots, cache, scale):
    """smla_kv8_append of one cache, run by run, in binary32 (torch's IEEE operations): updates cache, scale."""
    nb, hk, bs, D = cache.shape
    T = k.shape[0]
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= nb * bs:
            t += 1
            continue
        e = t
        while e < T and 0 <= int(slots[e]) < nb * bs and int(slots[e]) // bs == s // bs:
            e += 1
        blk = s // bs
        offs = slots[t:e] % bs
        rows = k[t:e].float()                                  # [n, H_kv, D]
        a = rows.abs()
        amax = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax((0, 2))
        new = (amax / 448.0).clamp(min=2.0 ** -60)
        low = int(offs.min())
        for h in range(hk):
            now = new[h]
            if low > 0:
                old = scale[blk, h].clone()
                if now > old:
                    was = cache[blk, h, :low].view(FP8).float()
                    cache[blk, h, :low] = (was * old / now).clamp(-448, 448).to(FP8).view(torch.uint8)
                else:
                    now = old
            scale[blk, h] = now
            cache[blk, h, offs] = (rows[:, h] / now).clamp(-448, 448).to(FP8).view(torch.uint8)
        t = e
