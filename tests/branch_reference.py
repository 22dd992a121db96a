"""Plain references of the operators of a step that drafts and branches (tests only): 64 bits, or one entry at a time."""
import math

import numpy as np
import torch

import kv8_reference as ref

FP8 = torch.float8_e4m3fn


def norm_rope(x, w, plus, eps, pos, cs, off, neox):
    """(y, size): y in binary64, and what its roundings are relative to (of a turned element its pair's |a cos| + |b sin|)."""
    n = cs.shape[1] // 2
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * (w.double() + plus)
    size = y.abs().clone()
    row = cs.double()[pos]
    c, s = row[:, None, :n], row[:, None, n:]
    part = y[..., off:off + 2 * n].clone()
    a, b = (part[..., :n], part[..., n:]) if neox else (part[..., 0::2], part[..., 1::2])

    def put(to, p, q):
        to[..., off:off + 2 * n] = torch.cat([p, q], -1) if neox else torch.stack([p, q], -1).flatten(-2)

    put(y, a * c - b * s, b * c + a * s)
    put(size, (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())
    return y, size


def tree_masks(parents, lens, start, words, window):
    """(mask [T, 64 words] of truth values, positions), a token at a time."""
    T = len(parents)
    mask, pos = np.zeros((T, 64 * words), bool), np.zeros(T, np.int64)
    for b in range(len(lens)):
        q0, q1 = int(start[b]), int(start[b + 1])
        ctx = max(int(lens[b]), 0) - (q1 - q0)
        for i in range(q1 - q0):
            depth, at = 0, i
            if i < 64 * words:
                while True:
                    if window <= 0 or depth < window:
                        mask[q0 + i, at] = True
                    up = int(parents[q0 + at])
                    if up < 0 or up >= at:
                        break
                    at, depth = up, depth + 1
            pos[q0 + i] = max(0, ctx + depth)
    return mask, pos


def words_of(mask):
    """Truth values [T, 64 words] as int64 words."""
    return torch.from_numpy(np.packbits(np.asarray(mask), axis=1, bitorder="little").view(np.int64).copy())


def random_tree(n, r, chain=False):
    """Parents of n nodes, each before its children."""
    return np.array([i - 1 if chain else int(r.randint(-1, i)) if i else -1 for i in range(n)], np.int32)


def tree_attention(q, kc, vc, ks, vs, table, lens, start, mask, scale, window=0, positions=None, sinks=None):
    """As kv8_reference.attention, for tokens that see the context and the new tokens of their mask (truth values)."""
    T, H, D = q.shape
    nb, hk, bs, _ = kc.shape
    G = H // hk
    out = torch.full((T, H, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    wsum = torch.zeros((T, H, D), dtype=torch.float64)
    reach = torch.zeros((T, H), dtype=torch.float64)
    kval, vval = ref.values(kc, ks), ref.values(vc, vs)
    qd = q.double()
    for b in range(len(lens)):
        q0, q1 = int(start[b]), int(start[b + 1])
        n = min(max(int(lens[b]), 0), table.shape[1] * bs)
        pages = table[b, :(n + bs - 1) // bs].long()
        good = (pages >= 0) & (pages < nb)
        safe = pages.clamp(0, max(nb - 1, 0))
        there = good.repeat_interleave(bs)[:n]
        ctx = n - (q1 - q0)
        j = torch.arange(n)
        for t in range(q0, q1):
            see = (j < ctx) & there
            if window > 0:
                see &= j > min(max(int(positions[t]), ctx), n - 1) - window
            node = j - ctx
            bits = torch.as_tensor(np.asarray(mask[t]))
            inside = (node >= 0) & (node < len(bits))
            see |= inside & bits[node.clamp(0, len(bits) - 1)] & there
            for h in range(H):
                kk = kval[safe, h // G].reshape(-1, D)[:n][see]
                vv = vval[safe, h // G].reshape(-1, D)[:n][see]
                s = (kk @ qd[t, h]) * scale
                z = s if sinks is None else torch.cat([s, sinks[h].double().reshape(1)])
                z = torch.logsumexp(z, 0) if len(z) else torch.tensor(-math.inf, dtype=torch.float64)
                lse[t, h] = z
                out[t, h] = 0.0
                if len(s):
                    w = torch.exp(s - z)
                    out[t, h] = w @ vv
                    wsum[t, h] = w @ vv.abs()
                    reach[t, h] = (kk.abs() @ qd[t, h].abs()).max() * scale
    return out, lse, wsum, reach


def kept_list(kept, count, n, width):
    """The valid start of a list of kept tokens, and whether something was wrong with it."""
    want = max(int(count), 0)
    k, bad = min(want, n, width), want > min(n, width)
    got, before = [], -1
    for i in range(k):
        x = int(kept[i])
        if x <= before or x >= n:
            bad = True
            break
        got.append(x)
        before = x
    return got, bad


def keep_scaled(codes, scale, table, lens, ql, kept, counts):
    """smla_keep_tokens of one pool, a block at a time, in binary32 (torch's IEEE operations): updates codes, scale."""
    nb, hk, bs, D = codes.shape

    def block(b, pos):
        j = pos // bs
        e = int(table[b, j]) if j < table.shape[1] else -1
        return e if 0 <= e < nb else -1

    def rounded(code, old, now):
        return (code.view(FP8).float() * old / now).clamp(-448, 448).to(FP8).view(torch.uint8)

    for b in range(len(lens)):
        n = min(max(int(ql[b]), 0), max(int(lens[b]), 0))
        ctx = max(int(lens[b]), 0) - n
        nodes, _ = kept_list(kept[b], counts[b], n, kept.shape[1])
        i = 0
        while i < len(nodes):
            first = i
            j = (ctx + i) // bs
            mine = []
            while i < len(nodes) and (ctx + i) // bs == j:
                mine.append((ctx + nodes[i], ctx + i))
                i += 1
            to = block(b, ctx + first)
            if to < 0:
                continue
            mine = [(block(b, s), s % bs, d % bs) for s, d in mine]
            low = (ctx + first) % bs
            for h in range(hk):
                old = scale[to, h].clone()
                now = max([old] + [scale[f, h].clone() for f, _, _ in mine if f >= 0])
                rows = {}
                for f, so, do in mine:
                    if f >= 0:
                        was = scale[f, h].clone() if f != to else old
                        c = codes[f, h, so].clone()
                        rows[do] = c if was == now else rounded(c, was, now)
                if now > old:
                    codes[to, h, :low] = rounded(codes[to, h, :low], old, now)
                for do, c in rows.items():
                    codes[to, h, do] = c
                scale[to, h] = now


def keep_rows(pool, bs, table, lens, ql, kept, counts):
    """The same of plain rows: pool [num_slots, D]."""
    nb = pool.shape[0] // bs
    for b in range(len(lens)):
        n = min(max(int(ql[b]), 0), max(int(lens[b]), 0))
        ctx = max(int(lens[b]), 0) - n
        nodes, _ = kept_list(kept[b], counts[b], n, kept.shape[1])
        moved = []
        for i, x in enumerate(nodes):
            slots = []
            for pos in (ctx + x, ctx + i):
                e = int(table[b, pos // bs]) if pos // bs < table.shape[1] else -1
                slots.append(e * bs + pos % bs if 0 <= e < nb else -1)
            if min(slots) >= 0:
                moved.append((slots[1], pool[slots[0]].clone()))
        for d, row in moved:
            pool[d] = row


def fork(source, keep, held, table, ring, state, bs, nb, table_out):
    """smla_fork_block_tables, one entry at a time."""
    B, (B_old, width) = len(source), table.shape
    ring, table_out = ring.copy(), table_out.copy()
    cap = len(ring)
    head, count = int(state[0]) % cap, min(max(int(state[1]), 0), cap)
    rows, tokens = [], 0
    for b in range(B):
        r = int(source[b])
        n = 0
        if 0 <= r < B_old:
            n = min(max(int(keep[b]), 0), min(max(int(held[r]), 0), width) * bs)
        tokens += n
        rows.append([int(x) for x in table[r, :-(-n // bs)]] if n else [])
        rows[-1] = (rows[-1], n % bs != 0)
    full, tails = set(), {}
    for b, (row, tail) in enumerate(rows):
        full.update(row[:-1] if tail else row)
        if tail:
            tails.setdefault(row[-1], b)
    copies = [b for b, (row, tail) in enumerate(rows)
              if tail and 0 <= row[-1] < nb and (row[-1] in full or tails[row[-1]] != b)]
    lacking = max(0, len(copies) - count)
    frm, to = np.full(B, -1, np.int32), np.full(B, -1, np.int32)
    out = dict(copy_from=frm, copy_to=to)
    if lacking:
        return dict(out, counts=np.array([tokens, 0, 0, lacking]), ring=ring, ring_state=np.array([head, count]), block_table=table_out, blocks_held=None)
    live = set()
    for row, _ in rows:
        live.update(row)
    gone, seen = [], set()
    for r in range(B_old):
        for e in table[r, :min(max(int(held[r]), 0), width)]:
            e = int(e)
            if 0 <= e < nb and e not in live and e not in seen:
                seen.add(e)
                gone.append(e)
    for k, b in enumerate(copies):
        frm[b], to[b] = rows[b][0][-1], ring[(head + k) % cap]
        rows[b][0][-1] = int(to[b])
    for k, e in enumerate(gone):
        ring[(head + count + k) % cap] = e
    for b, (row, _) in enumerate(rows):
        table_out[b, :len(row)] = row
    return dict(out, counts=np.array([tokens, len(copies), len(gone), 0]), ring=ring, block_table=table_out,
                ring_state=np.array([(head + len(copies)) % cap, min(count - len(copies) + len(gone), cap)]),
                blocks_held=np.array([len(row) for row, _ in rows]))
