"""The operators of a serving step that drafts and branches, as they are measured: norms and rotation of queries and keys in one
pass, masks of drafted trees, attention of such trees over the block-scaled cache, the move of accepted tokens' rows, forked
block tables, and copies of blocks. `run` holds their plain form in elementary torch operations and, where `own` is set, the
calls of the framework's own operators; `exact` holds the definitions in 64 bits of those that compute numbers."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short chat whose draft has eight nodes: latency counts
        dict(name="tree attend one short", op="attend", B=1, H=16, Hkv=2, D=128, bs=64, ctx=509, nodes=8, window=0, mix=1),
        # a verification step of a ragged batch with long contexts, up to 32 nodes to a request
        dict(name="tree attend 64", op="attend", B=64, H=32, Hkv=8, D=128, bs=64, ctx=8192, nodes=32, window=0, mix=2),
        # the masks and positions of that step
        dict(name="tree masks 64", op="masks", B=64, nodes=32, ctx=8192, window=0, mix=4),
        # those of a large batch with large trees, under a sliding window
        dict(name="tree masks 1000", op="masks", B=1000, nodes=200, ctx=8192, window=64, mix=5),
        # a verification step's queries and keys: two drafted tokens for each of 32 requests
        dict(name="norm rope 64", op="norm", T=64, H=32, Hk=8, D=128, rot=128, off=0, half=True, dtype="bf16", wide=False, per_head=False, plus=0.0, far=131072),
        # a prompt's, the last quarter of each head rotated in interleaved pairs, a weight to each head
        dict(name="norm rope prompt 8192", op="norm", T=8192, H=32, Hk=8, D=128, rot=32, off=96, half=False, dtype="bf16", wide=True, per_head=True, plus=1.0, far=131072),
        # the accepted tokens of one request, in the latent cache of two layers
        dict(name="keep latent one", op="keep", B=1, Hkv=1, D=576, bs=64, ctx=300, nodes=32, layers=2, latent=2, mix=6),
        # those of a whole step, in every layer's block-scaled cache
        dict(name="keep 64", op="keep", B=64, Hkv=8, D=128, bs=64, ctx=300, nodes=32, layers=8, latent=0, mix=7),
        # one prompt that is sampled four times
        dict(name="fork one by 4", op="fork", B=1, beams=4, bs=16, ctx=509, mix=8),
        # the beams of 64 requests, four to each, that go on from one another
        dict(name="fork 64 by 4", op="fork", B=64, beams=4, bs=64, ctx=16384, mix=9),
        # the last blocks of three samples, in two layers
        dict(name="copy 3", op="copy", n=3, Hkv=2, D=64, bs=16, blocks=100, layers=2, mix=10),
        # those of all beams of a large batch, in 16 layers
        dict(name="copy 192", op="copy", n=192, Hkv=8, D=128, bs=64, blocks=500, layers=16, mix=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend"] * 5 + ["masks", "norm", "norm", "keep", "keep", "fork", "fork", "copy"])
    mix = rng.randrange(1000, 1 << 20)
    bs = rng.choice([16, 32, 64, 128])
    if op == "attend":
        while True:
            Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
            H = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
            B, nodes, ctx = _log(rng, 1, 64), _log(rng, 1, 200), _log(rng, 1, 32768)
            ctx = max(ctx, nodes)
            if H <= 64 and B * H * nodes * ctx <= 1 << 29 and B * Hkv * ctx * D <= 1 << 29:
                break
        return dict(op=op, B=B, H=H, Hkv=Hkv, D=D, bs=bs, ctx=ctx, nodes=nodes, window=rng.choice([0, 0, 0, _log(rng, 4, 4096)]), mix=mix)
    if op == "masks":
        B = _log(rng, 1, 1000)
        nodes = _log(rng, 1, 200)
        return dict(op=op, B=B, nodes=nodes, ctx=max(nodes, _log(rng, 1, 131072)), window=rng.choice([0, 0, _log(rng, 1, 64)]), mix=mix)
    if op == "norm":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([r for r in (32, 64, 80, 96, 128, 256) if r <= D])
        H = _log(rng, 1, 128)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        T = _log(rng, 1, min(8192, (8192 * 40 * 128) // ((H + 8) * D * (2 if dtype == "f32" else 1))))
        return dict(op=op, T=T, H=H, Hk=rng.choice([1, 2, 8]), D=D, rot=rot, off=rng.choice([0, D - rot]), half=rng.random() < 0.5, dtype=dtype,
                    wide=rng.random() < 0.5, per_head=rng.random() < 0.3, plus=rng.choice([0.0, 0.0, 1.0]), far=_log(rng, 64, 131072))
    if op == "keep":
        latent = rng.choice([0, 0, 1, 2])
        B, layers = _log(rng, 1, 64), _log(rng, 1, 8)
        nodes = _log(rng, 1, 100)
        return dict(op=op, B=B, Hkv=1 if latent else rng.choice([1, 2, 4, 8]), D=rng.choice([512, 576]) if latent else rng.choice([64, 128]), bs=bs, ctx=max(nodes, rng.randint(1, 300)),
                    nodes=nodes, layers=layers, latent=latent, mix=mix)
    if op == "fork":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, beams=rng.randint(2, 4), bs=bs, ctx=_log(rng, 1, 16384 * bs // 64), mix=mix)
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    n = _log(rng, 1, 192)
    return dict(op=op, n=n, Hkv=Hkv, D=D, bs=bs if bs < 128 else 64, blocks=2 * n + rng.randint(1, 116), layers=_log(rng, 1, 16), mix=mix)


def _lens(c):
    """Lengths with the drafted tokens, and how many those are, of each request (ragged, the first the largest), from the case alone."""
    r = np.random.RandomState(c["mix"])
    B, ctx, n = c["B"], c["ctx"], c["nodes"]
    lens = np.exp(r.uniform(math.log(max(1, ctx // 32)), math.log(ctx + 1), B)).astype(np.int64).clip(1, ctx)
    ql = r.randint(1, n + 1, B)
    lens[0], ql[0] = ctx, n
    return np.maximum(lens, ql), ql


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _start(ql):
    return _up(np.concatenate([[0], np.cumsum(ql)]))


def _pages(lens, bs, gen, spare=0):
    """A random block table over a pool that just holds the requests (and `spare` more blocks), and its number of blocks."""
    nb = -(-lens // bs)
    total = int(nb.sum())
    perm = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
    j = torch.arange(int(nb.max()), device=DEV)
    at = torch.from_numpy(np.cumsum(nb) - nb).to(DEV)[:, None] + j[None, :]
    keep = j[None, :] < torch.from_numpy(nb).to(DEV)[:, None]
    return torch.where(keep, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).contiguous(), total + spare


def _cache(total, c, gen):
    """Codes and scales of one side of a cache: heads of different size, each block with its own largest value."""
    size = torch.rand((total, c["Hkv"], 1, 1), generator=gen, device=DEV) * 1.5 + 0.25
    x = torch.randn((total, c["Hkv"], c["bs"], c["D"]), generator=gen, device=DEV) * size
    s = x.abs().amax((2, 3)) / 448.0
    return (x / s[:, :, None, None]).to(FP8).view(torch.uint8), s


def _parents(ql, r):
    """Drafted trees, a parent before its children: mostly short branches that hang on early nodes, some long chains."""
    i = np.concatenate([np.arange(n) for n in ql])
    chain = np.repeat(r.rand(len(ql)) < 0.2, ql)
    near = np.repeat(r.rand(len(ql)) * 0.7, ql)
    u = r.rand(len(i))
    some = np.floor(i * np.maximum(u, near * r.rand(len(i)))).astype(np.int64)
    p = np.where(chain, i - 1, np.where(r.rand(len(i)) < 0.1, -1, np.minimum(some, i - 1)))
    return np.where(i == 0, -1, p)


def _ancestors(parents, start):
    """[T, n] whether a token sees each node of its tree (itself and those that it descends from), and the tokens' depths; on the host."""
    T, n = len(parents), int(np.diff(start).max())
    own_i = np.arange(T) - np.repeat(start[:-1], np.diff(start))
    first = np.repeat(start[:-1], np.diff(start))
    see = np.zeros((T, n), bool)
    depth = np.zeros(T, np.int64)
    for i in range(n):  # node i of every tree at once
        t = np.nonzero(own_i == i)[0]
        up = parents[t]
        q = first[t] + np.maximum(up, 0)
        see[t] = see[q] & (up >= 0)[:, None]
        depth[t] = np.where(up >= 0, depth[q] + 1, 0)
        see[t, i] = True
    return see, depth


def _bits(see):
    """Truth values [T, n] as 64-bit words [T, ceil(n / 64)], the first the lowest bit."""
    T, n = see.shape
    words = -(-n // 64)
    b = np.packbits(np.pad(see, ((0, 0), (0, words * 64 - n))), axis=1, bitorder="little")
    return torch.from_numpy(b.view(np.int64).reshape(T, words)).to(DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    r = np.random.RandomState(int(seed) % (1 << 31))
    s = dict(c=c)
    if c["op"] == "attend":
        lens, ql = _lens(c)
        table, total = _pages(lens, c["bs"], g)
        s["kc"], s["ks"] = _cache(total, c, g)
        s["vc"], s["vs"] = _cache(total, c, g)
        s["q"] = torch.randn((int(ql.sum()), c["H"], c["D"]), generator=g, device=DEV).to(torch.bfloat16)
        see, depth = _ancestors(_parents(ql, r), np.concatenate([[0], np.cumsum(ql)]))
        pos = np.repeat(lens - ql, ql) + depth
        s.update(table=table, lens=_up(lens), start=_start(ql), mask=_bits(see), pos=torch.from_numpy(pos).to(DEV), scale=1.0 / math.sqrt(c["D"]))
    elif c["op"] == "masks":
        lens, ql = _lens(c)
        s.update(parents=_up(_parents(ql, r)), lens=_up(lens), start=_start(ql))
    elif c["op"] == "norm":
        dt = TYPES[c["dtype"]]
        wt = torch.float32 if c["wide"] else dt
        for x, h in (("q", c["H"]), ("k", c["Hk"])):
            # tokens and heads of different size
            size = torch.exp(torch.randn((c["T"], h, 1), generator=g, device=DEV))
            s[x] = (torch.randn((c["T"], h, c["D"]), generator=g, device=DEV) * size).to(dt)
            shape = (h, c["D"]) if c["per_head"] else (c["D"],)
            s["w" + x] = (1.0 - c["plus"] + 0.2 * torch.randn(shape, generator=g, device=DEV)).to(wt)
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=g, device=DEV)
        f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        a = torch.arange(c["far"], device=DEV, dtype=torch.float64)[:, None] * f[None, :]
        s["cs"] = torch.cat([a.cos(), a.sin()], 1).float()
    elif c["op"] == "keep":
        lens, ql = _lens(c)
        table, total = _pages(lens, c["bs"], g)
        if c["latent"]:
            x = torch.randn((c["layers"], total * c["bs"], c["D"]), generator=g, device=DEV)
            s["caches"] = [y.to(torch.bfloat16) if c["latent"] == 2 else y.to(FP8).view(torch.uint8) for y in x]
        else:
            s["caches"] = []
            for _ in range(c["layers"]):
                (kc, ks), (vc, vs) = _cache(total, c, g), _cache(total, c, g)
                s["caches"].append((kc, vc, ks, vs))
        # the accepted nodes: a path down the tree, so ascending; often short
        W = int(min(c["nodes"], 16))
        kept = np.full((c["B"], W), -1, np.int64)
        count = np.minimum(np.minimum(ql, W), 1 + r.geometric(0.3, c["B"]))
        count = np.where(r.rand(c["B"]) < 0.05, 0, count)
        for b in range(c["B"]):
            kept[b, :count[b]] = np.sort(r.choice(int(ql[b]), int(count[b]), replace=False))
        if own:  # what a program keeps beside its caches
            from sparse_mla_attention_04_gb300 import binding
            s["handle"] = binding.TokenPools(s["caches"], c["bs"])
        s.update(table=table, lens=_up(lens), ql=_up(ql), kept=_up(kept), count=_up(count), lens_out=torch.empty(c["B"], dtype=torch.int32, device=DEV))
    elif c["op"] == "fork":
        s.update(_fork_inputs(c, r))
    else:
        s["pools"] = []
        for _ in range(c["layers"]):
            for _ in range(2):
                s["pools"] += list(_cache(c["blocks"], c, g))
        perm = r.permutation(c["blocks"])
        src, dst = perm[:c["n"]].copy(), perm[c["n"]: 2 * c["n"]].copy()
        none = r.rand(c["n"]) < 0.1  # rows that need no copy
        none[0] = False
        src[none] = dst[none] = -1
        same = r.rand(c["n"]) < 0.3  # one block is often copied several times
        src = np.where(same & ~none, perm[0], src)
        s.update(src=_up(src), dst=_up(dst))
        if own:
            from sparse_mla_attention_04_gb300 import binding
            s["handle"] = binding.BlockPools(s["pools"])
    return s


def _fork_inputs(c, r):
    """Rows of B requests with up to `beams` beams each, which share their first blocks, as an earlier step left them; and which row each goes on from."""
    B, n, bs = c["B"], c["beams"], c["bs"]
    rows = B * n
    width = -(-c["ctx"] // bs) + 1
    top = np.exp(r.uniform(math.log(max(1, c["ctx"] // 32)), math.log(c["ctx"] + 1), B)).astype(np.int64).clip(1, c["ctx"])
    top[0] = c["ctx"]
    table = np.full((rows, width), -1, np.int64)
    held = np.zeros(rows, np.int64)
    lens = np.zeros(rows, np.int64)
    used = 0
    for b in range(B):
        first = r.rand() < 0.2 or (B == 1 and n > 1)  # a prompt that is forked now: its other rows are empty
        nb = -(-top[b] // bs)
        shared = r.randint(0, nb)  # blocks before the beams went apart
        base = used + np.arange(shared)
        used += shared
        for i in range(n):
            row = b * n + i
            if first and i:
                continue
            table[row, :shared] = base
            table[row, shared:nb] = used + np.arange(nb - shared)
            used += nb - shared
            held[row], lens[row] = nb, top[b]
    source = np.repeat(np.arange(B) * n, n) + r.randint(0, n, rows)
    source = np.where(held[source] > 0, source, np.repeat(np.arange(B) * n, n))
    ends = np.repeat(r.rand(B) < 0.05, n)  # requests that have ended give their blocks back
    ends[:n] = False
    source = np.where(ends, -1, source)
    keep = lens[source]
    short = r.rand(rows) < 0.1  # rows that go back to an earlier token
    keep = np.where(source < 0, 0, np.where(short, np.ceil(keep * r.rand(rows)), keep)).astype(np.int64)
    cap = rows * (width + 1) + 100  # blocks of the pool, from the case alone
    perm = r.permutation(cap)
    table = np.where(table >= 0, perm[table.clip(min=0)], -1)
    head, count = int(r.randint(cap)), cap - used
    ring = np.full(cap, -1, np.int64)
    ring[(head + np.arange(count)) % cap] = perm[used:]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(source=_up(source), keep=_up(keep), held=_up(held), table=_up(table), ring=_up(ring), state=_up([head, count]), cap=cap, rows=rows, table_out=torch.full((rows, width), -1, **i32),
                held_out=torch.empty(rows, **i32), state_out=torch.empty(2, **i32), src=torch.empty(rows, **i32), dst=torch.empty(rows, **i32), counts=torch.empty(4, **i32))


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "masks": _masks, "norm": _norm, "keep": _keep, "fork": _fork, "copy": _copy}[s["c"]["op"]](s)


def _own(s):
    from sparse_mla_attention_04_gb300 import binding as b
    c = s["c"]
    if c["op"] == "attend":
        out, lse = b.smla_kv8_tree_attn_fwd(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["start"], s["mask"], s["scale"], max_query_len=c["nodes"], window=c["window"],
                                            positions=s["pos"] if c["window"] else None)
        return {"out": out, "lse": lse}
    if c["op"] == "masks":
        m = b.smla_build_tree_masks(s["parents"], s["lens"], s["start"], max_query_len=c["nodes"], window=c["window"])
        return {"mask": m.tree_mask, "pos": m.positions}
    if c["op"] == "norm":
        q, k = b.smla_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["cs"], eps=1e-6, weight_offset=c["plus"], rot_offset=c["off"], is_neox=c["half"])
        return {"q": q, "k": k}
    if c["op"] == "keep":
        b.smla_keep_tokens(s["handle"], s["table"], s["lens"], s["ql"], s["kept"], s["count"], seq_lens_out=s["lens_out"])
        return _kept(s, s["lens_out"])
    if c["op"] == "fork":
        f = b.smla_fork_block_tables(s["source"], s["keep"], s["held"], s["table"], s["ring"], s["state"], block_size=c["bs"], num_blocks=s["cap"], block_table_out=s["table_out"],
                                     blocks_held_out=s["held_out"], ring_state_out=s["state_out"], copy_from=s["src"], copy_to=s["dst"], counts=s["counts"])
        return {"table": f.block_table, "held": f.blocks_held, "ring": s["ring"], "state": f.ring_state, "src": f.copy_from, "dst": f.copy_to, "counts": f.counts}
    b.smla_copy_blocks(s["handle"], s["src"], s["dst"])
    return _copied(s)


def _unpack(mask, n):
    i = torch.arange(n, device=DEV)
    return (mask[:, i // 64] >> (i % 64)) & 1 == 1


def _attend(s):
    """Every request padded to the longest: gather, dequantise, scores, softmax, values."""
    c, q, bs = s["c"], s["q"], s["c"]["bs"]
    B, H, Hkv, D, G, Q, L = c["B"], c["H"], c["Hkv"], c["D"], c["H"] // c["Hkv"], c["nodes"], int(s["table"].shape[1]) * c["bs"]
    T = q.shape[0]
    table = s["table"].clamp(min=0).long()

    def gathered(codes, scales):
        x = codes.view(FP8)[table].float() * scales[table][..., None, None]  # [B, nb, Hkv, bs, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    lens, start = s["lens"].long(), s["start"].long()
    ql = start[1:] - start[:-1]
    i, j = torch.arange(Q, device=DEV), torch.arange(L, device=DEV)
    at = (start[:-1, None] + i).clamp(max=T - 1)  # [B, Q]
    qp = q[at].float() * s["scale"]
    qp = qp.reshape(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    x = (qp @ gathered(s["kc"], s["ks"]).transpose(2, 3)).view(B, Hkv, G, Q, L)
    ctx = lens - ql
    node = j[None, :] - ctx[:, None]  # [B, L]
    seen = (node < 0)[:, None, :].expand(B, Q, L)
    if c["window"]:
        seen = seen & (j > s["pos"][at][..., None] - c["window"])
    in_tree = ((node >= 0) & (j < lens[:, None]))[:, None, :]
    tree = _unpack(s["mask"], Q)[at]  # [B, Q, Q]
    tree = tree.gather(2, node.clamp(0, Q - 1)[:, None, :].expand(B, Q, L))
    seen = seen | (in_tree & tree)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=-3e38)).exp_()
    l = x.sum(-1, keepdim=True)
    v = gathered(s["vc"], s["vs"]).masked_fill((j >= lens[:, None])[:, None, :, None], 0.0)
    o = (x.view(B, Hkv, G * Q, L) @ v).view(B, Hkv, G, Q, D) / l.clamp(min=1e-38)
    lse = (m + l.log()).squeeze(-1)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    o = o.permute(0, 3, 1, 2, 4)[b, t - start[b]].reshape(T, H, D)
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2)[b, t - start[b]].reshape(T, H)}


def _masks(s):
    """The trees' reach by repeated products of their adjacency, padded to the largest tree."""
    c, n = s["c"], s["c"]["nodes"]
    start, lens = s["start"].long(), s["lens"].long()
    T, B = s["parents"].numel(), c["B"]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    i = t - start[b]
    reach = torch.zeros((B, n, n), device=DEV)
    reach[:, range(n), range(n)] = 1.0
    up = s["parents"].long()
    reach[b, i, torch.where(up >= 0, up, i)] = 1.0
    for _ in range(max(1, math.ceil(math.log2(n))) if n > 1 else 0):
        reach = (reach @ reach > 0).float()
    see = reach[b, i] > 0  # [T, n]
    depth = see.sum(1) - 1
    if c["window"]:
        there = torch.zeros((B, n), dtype=torch.int64, device=DEV)
        there[b, i] = depth
        see &= depth[:, None] - there[b] < c["window"]
    words = -(-n // 64)
    w = torch.zeros((T, words * 64), dtype=torch.int64, device=DEV)
    w[:, :n] = see.long()
    mask = (w.view(T, words, 64) << torch.arange(64, device=DEV)).sum(2)
    return {"mask": mask, "pos": (lens - (start[1:] - start[:-1]))[b] + depth}


def _norm(s):
    c, n = s["c"], s["c"]["rot"] // 2
    row = s["cs"][s["pos"]]
    cos, sin = row[:, None, :n], row[:, None, n:]

    def turned(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * (w.float() + c["plus"])
        part = y[..., c["off"]: c["off"] + 2 * n]
        a, b = (part[..., :n], part[..., n:]) if c["half"] else (part[..., 0::2], part[..., 1::2])
        p, r = a * cos - b * sin, b * cos + a * sin
        y[..., c["off"]: c["off"] + 2 * n] = torch.cat([p, r], -1) if c["half"] else torch.stack([p, r], -1).flatten(-2)
        return y.to(x.dtype)

    return {"q": turned(s["q"], s["wq"]), "k": turned(s["k"], s["wk"])}


def _kept(s, lens_out):
    """The caches and lengths as they come out: codes as the values they stand for."""
    out = {"lens": lens_out}
    for n, x in enumerate(s["caches"]):
        if s["c"]["latent"]:
            out["pool%d" % n] = x.view(FP8) if s["c"]["latent"] == 1 else x
        else:
            out.update({"k%d" % n: x[0].view(FP8), "v%d" % n: x[1].view(FP8), "ks%d" % n: x[2], "vs%d" % n: x[3]})
    return out


def _keep(s):
    """Rows gathered from their old places, then a block at a time: its scale, its older rows, its new ones."""
    c, bs = s["c"], s["c"]["bs"]
    B, W = s["kept"].shape
    lens, ql, count = s["lens"].long(), s["ql"].long(), s["count"].long()
    ctx = lens - ql
    i = torch.arange(W, device=DEV)
    live = i < count[:, None]
    src = torch.where(live, ctx[:, None] + s["kept"], 0)
    dst = torch.where(live, ctx[:, None] + i, 0)
    rows = torch.arange(B, device=DEV)[:, None]
    b, k = live.nonzero(as_tuple=True)
    last = s["table"].shape[1] - 1
    sb, so = s["table"][rows, (src // bs).clamp(max=last)].long()[b, k], (src % bs)[b, k]
    db, do = s["table"][rows, (dst // bs).clamp(max=last)].long()[b, k], (dst % bs)[b, k]
    if c["latent"]:
        for x in s["caches"]:
            x[db * bs + do] = x[sb * bs + so]
        return _kept(s, (ctx + count).to(torch.int32))
    # each request's first block that changes may hold older rows, which follow its scale
    fb = s["table"][rows[:, 0], (ctx // bs).clamp(max=last)].long()
    fb = torch.where(count > 0, fb, -1)
    has = fb >= 0
    fb = fb.clamp(min=0)
    older = (torch.arange(bs, device=DEV)[None, :] < (ctx % bs)[:, None]) & has[:, None]
    for kc, vc, ks, vs in s["caches"]:
        for codes, scale in ((kc, ks), (vc, vs)):
            was = scale.clone()
            scale.index_reduce_(0, db, was[sb], "amax")
            moved = codes[sb, :, so].view(FP8).float()  # [rows, Hkv, D]
            moved = moved * was[sb][..., None] / scale[db][..., None]
            old = codes[fb].view(FP8).float()
            now = old * was[fb][..., None, None] / scale[fb][..., None, None]
            grown = (scale[fb] > was[fb])[..., None, None] & older[:, None, :, None]
            bb, oo = (older & has[:, None]).nonzero(as_tuple=True)
            codes[fb[bb], :, oo] = torch.where(grown, now.clamp(-448, 448), old)[bb, :, oo].to(FP8).view(torch.uint8)
            codes[db, :, do] = moved.clamp(-448, 448).to(FP8).view(torch.uint8)
    return _kept(s, (ctx + count).to(torch.int32))


def _fork(s):
    c, bs, cap, ring, table = s["c"], s["c"]["bs"], s["cap"], s["ring"], s["table"].long()
    rows, width = table.shape
    source, held = s["source"].long(), s["held"].long()
    head, count = s["state"][0].long(), s["state"][1].long()
    j = torch.arange(width, device=DEV)[None, :]
    r = torch.arange(rows, device=DEV)
    from_ = source.clamp(min=0)
    n = torch.where(source >= 0, torch.minimum(s["keep"].long(), held[from_] * bs), 0)
    blocks = (n + bs - 1) // bs
    new = table[from_]  # [rows, width]
    has = j < blocks[:, None]
    tail = (n % bs != 0)[:, None] & (j == blocks[:, None] - 1)
    # who keeps a block: a row that has it whole (0), else the first row whose last one it is (1 + row); else what was held first
    order = 1 + rows + r[:, None] * width + j
    big = torch.full((cap + 1,), 1 << 40, dtype=torch.int64, device=DEV)
    at = lambda keep, which: torch.where(keep, which, cap).reshape(-1)  # noqa: E731
    big.scatter_reduce_(0, at(has & ~tail, new), torch.zeros((rows * width,), dtype=torch.int64, device=DEV), "amin")
    big.scatter_reduce_(0, at(tail, new), (1 + r)[:, None].expand(rows, width).reshape(-1), "amin")
    old = j < held[:, None]
    big.scatter_reduce_(0, at(old, table), order.reshape(-1), "amin")
    last = new[r, (blocks - 1).clamp(min=0)]
    copies = tail.any(1) & (big[last] != 1 + r)
    gives = (old & (big[table.clamp(min=0)] == order)).reshape(-1)
    took, gave = copies.sum(), gives.sum()
    short = (took - count).clamp(min=0)
    ok = short == 0
    k = copies.cumsum(0) - 1
    to = ring[((head + k) % cap).clamp(min=0)]
    src, dst = torch.where(copies & ok, last, -1), torch.where(copies & ok, to, -1)
    place = torch.where(gives & ok, (head + count + gives.cumsum(0) - 1) % cap, cap)
    ring.copy_(torch.cat([ring, ring[:1]]).scatter_(0, place, table.reshape(-1).to(torch.int32))[:cap])
    new = torch.where(tail & copies[:, None], dst[:, None], new)
    table_out = torch.where(has & ok, new, s["table_out"].long())
    i32 = torch.int32
    took, gave = torch.where(ok, took, 0), torch.where(ok, gave, 0)
    return {"table": table_out.to(i32), "held": torch.where(ok, blocks, s["held_out"]).to(i32), "ring": ring, "state": torch.stack([(head + took) % cap, count - took + gave]).to(i32), "src": src.to(i32),
            "dst": dst.to(i32), "counts": torch.stack([n.sum(), took, gave, short]).to(i32)}


def _copied(s):
    return {"pool%d" % i: x.view(FP8) if x.dtype == torch.uint8 else x for i, x in enumerate(s["pools"])}


def _copy(s):
    keep = (s["src"] >= 0).nonzero()[:, 0]
    src, dst = s["src"][keep].long(), s["dst"][keep].long()
    for x in s["pools"]:
        x[dst] = x[src]
    return _copied(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "attend":
        lens, n = _lens(c)
        ctx = lens - n
        T = int(n.sum())
        seen = np.minimum(ctx, c["window"]) if c["window"] else ctx
        words = -(-c["nodes"] // 64)
        return {"bytes": float((seen + n).sum()) * c["Hkv"] * (2 * c["D"] + 8 / c["bs"]) + T * (c["H"] * (4 * c["D"] + 4) + 8 * words), "flops": 4.0 * c["D"] * c["H"] * float((n * (seen + 1)).sum())}
    if c["op"] == "masks":
        T = int(_lens(c)[1].sum())
        return {"bytes": T * (4.0 + 8 + 8 * -(-c["nodes"] // 64)) + 8.0 * c["B"], "flops": 2.0 * T}
    if c["op"] == "norm":
        n = c["T"] * (c["H"] + c["Hk"])
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2.0 * n * c["D"] * size + c["T"] * (8 + 4 * c["rot"]), "flops": n * (4.0 * c["D"] + 3.0 * c["rot"])}
    if c["op"] == "keep":
        # about four rows of each request are moved
        n = c["B"] * min(4, c["nodes"]) * c["layers"] * c["D"]
        return {"bytes": 2.0 * n * (c["latent"] if c["latent"] else 2 * c["Hkv"]), "flops": 0.0 if c["latent"] else 2.0 * n * 2 * c["Hkv"]}
    if c["op"] == "fork":
        n = c["B"] * c["beams"] * (c["ctx"] / c["bs"] / 3 + 8)  # (lengths are spread over their logarithm)
        return {"bytes": 8.0 * n, "flops": 2.0 * n}
    return {"bytes": 2.0 * 0.9 * c["n"] * c["layers"] * 2 * c["Hkv"] * (c["bs"] * c["D"] + 4), "flops": 0.0}


# ---------------------------------------------------------------- the definitions in 64 bits
def _round_e4m3(x):
    """The nearest E4M3 value of each (ties to even), at most 448."""
    x = x.clamp(-448, 448)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(x.abs() < torch.exp2(e), e - 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    c = case
    if c["op"] in ("masks", "fork"):
        return None
    s = prepare(case, seed)
    if c["op"] == "copy":
        # where each block's bytes come from
        origin = np.arange(c["blocks"])
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            if a >= 0:
                origin[b] = a
        origin = torch.from_numpy(origin).to(DEV)
        return {n: x.double()[origin] for n, x in _copied(s).items()}
    if c["op"] == "attend":
        lens, ql = _lens(c)
        G, bs = c["H"] // c["Hkv"], c["bs"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        words = s["mask"].cpu().numpy().view(np.uint64)
        pos = s["pos"].cpu().numpy()
        at = 0
        for b, (n, q) in enumerate(zip(lens.tolist(), ql.tolist())):
            pages = s["table"][b, : -(-n // bs)].long()
            hide = np.zeros((q, n), bool)
            for i in range(q):
                bits = np.array([(int(words[at + i, m // 64]) >> (m % 64)) & 1 for m in range(q)], bool)
                hide[i, n - q:] = ~bits
                if c["window"]:
                    hide[i, : min(n - q, max(0, int(pos[at + i]) - c["window"] + 1))] = True
            hide = torch.from_numpy(hide).to(DEV)
            for h in range(c["Hkv"]):
                k, v = ((s[x + "c"][pages, h].view(FP8).double() * s[x + "s"][pages, h].double()[:, None, None]).reshape(-1, c["D"])[:n] for x in "kv")
                x = s["q"][at: at + q, h * G: h * G + G].double().transpose(0, 1) @ k.T * s["scale"]  # [G, q, n]
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, 2)
                lse[at: at + q, h * G: h * G + G] = z.T
                out[at: at + q, h * G: h * G + G] = (torch.exp(x - z[..., None]) @ v).transpose(0, 1)
            at += q
        return {"out": out, "lse": lse}
    if c["op"] == "norm":
        n = c["rot"] // 2
        row = s["cs"].double()[s["pos"]]
        z = torch.complex(row[:, :n], row[:, n:])[:, None, :]
        res = {}
        for x in "qk":
            y = s[x].double()
            y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["D"] + 1e-6) * (s["w" + x].double() + c["plus"])
            part = y[..., c["off"]: c["off"] + c["rot"]].clone()
            pair = part.reshape(*part.shape[:2], 2, n).transpose(2, 3) if c["half"] else part.reshape(*part.shape[:2], n, 2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            y[..., c["off"]: c["off"] + c["rot"]] = (w.transpose(2, 3) if c["half"] else w).reshape(part.shape)
            res[x] = y
        return res
    bs = c["bs"]
    lens, ql, count = (s[x].tolist() for x in ("lens", "ql", "count"))
    table, kept = s["table"].tolist(), s["kept"].tolist()
    res = {"lens": torch.tensor([n - q + k for n, q, k in zip(lens, ql, count)], dtype=torch.int32, device=DEV)}
    if c["latent"]:
        # where each slot's row comes from
        origin = np.arange(s["caches"][0].shape[0])
        for b in range(c["B"]):
            for i in range(count[b]):
                to, of = (lens[b] - ql[b] + x for x in (i, kept[b][i]))
                origin[table[b][to // bs] * bs + to % bs] = table[b][of // bs] * bs + of % bs
        origin = torch.from_numpy(origin).to(DEV)
        return {n: x if n == "lens" else x.double()[origin] for n, x in _kept(s, res["lens"]).items()}
    for m, (kc, vc, ks, vs) in enumerate(s["caches"]):
        for name, codes, scale in (("k", kc, ks), ("v", vc, vs)):
            val, sc = codes.view(FP8).double(), scale.double()
            for b in range(c["B"]):
                ctx = lens[b] - ql[b]
                moves = [(ctx + kept[b][i], ctx + i) for i in range(count[b])]
                for blk in sorted({d // bs for _, d in moves}):  # each block's rows come from it or from later ones
                    mine = [(x, d) for x, d in moves if d // bs == blk]
                    to = table[b][blk]
                    come = torch.tensor([table[b][x // bs] for x, _ in mine], device=DEV)
                    now = torch.maximum(sc[to], sc[come].amax(0))
                    rows = val[come, :, torch.tensor([x % bs for x, _ in mine], device=DEV)] * sc[come][..., None]
                    first = mine[0][1] % bs
                    grown = (now > sc[to])[:, None, None]
                    val[to, :, :first] = torch.where(grown, _round_e4m3(val[to, :, :first] * (sc[to] / now)[:, None, None]), val[to, :, :first])
                    val[to][:, [d % bs for _, d in mine]] = _round_e4m3(rows / now[None, :, None]).transpose(0, 1)
                    sc[to] = now
            res[name + "%d" % m], res[name + "s%d" % m] = val, sc
    return {n: res[n] for n in _kept(s, res["lens"])}
