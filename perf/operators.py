"""The serving-step operators that are measured: block tables and slot maps, rotary tables and rotations, the block-scaled
8-bit key/value cache's write, and attention over it. `run` holds their plain form in elementary torch operations and,
where `own` is set, the calls of the framework's own operators; `exact` holds their definitions in 64 bits."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short chat, one token: launch latency counts
        dict(name="attend one short", op="attend", B=1, H=16, Hkv=2, D=128, bs=64, ctx=509, q=1, window=0, mix=1),
        # a decode step of a ragged batch with long contexts: bandwidth counts
        dict(name="attend decode 64", op="attend", B=64, H=32, Hkv=8, D=128, bs=64, ctx=32768, q=1, window=0, mix=2),
        # a whole prompt at once
        dict(name="attend prompt 8192", op="attend", B=1, H=32, Hkv=8, D=128, bs=64, ctx=8192, q=8192, window=0, mix=3),
        # ragged chunks of several prompts behind long contexts, small heads and pages
        dict(name="attend chunks", op="attend", B=6, H=16, Hkv=2, D=64, bs=16, ctx=32001, q=701, window=0, mix=4),
        # one new token for each of 64 requests, in blocks that are partly full
        dict(name="append 64", op="append", B=64, Hkv=8, D=128, bs=64, ctx=8192, q=1, mix=5),
        # a prompt of 8192 tokens
        dict(name="append 8192", op="append", B=1, Hkv=8, D=128, bs=64, ctx=8192, q=8192, mix=6),
        # the maps of a decode step
        dict(name="tables decode 64", op="tables", B=64, bs=64, ctx=131072, q=1, mix=7),
        # the maps of a step that takes in many prompts while others end
        dict(name="tables prompts", op="tables", B=1000, bs=16, ctx=2048, q=2048, mix=8),
        # rotation of a decode step's queries and keys, the 64 rotary columns behind 128 plain ones
        dict(name="rope decode 64", op="rope", T=64, H=128, Hk=1, D=192, rot=64, off=128, half=True, inverse=False, far=131072, dtype="bf16"),
        # a prompt's queries and keys, the whole head rotated, pairs interleaved
        dict(name="rope prompt 8192", op="rope", T=8192, H=32, Hk=8, D=128, rot=128, off=0, half=False, inverse=False, far=131072, dtype="bf16"),
        # the table of a short context without scaling
        dict(name="rope table 4096", op="table", P=4096, rot=64, kind="none", factor=1.0, orig=4096),
        # the table of a long context: 32768 positions stretched to 1048576
        dict(name="rope table 1048576", op="table", P=1048576, rot=64, kind="yarn", factor=32.0, orig=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend"] * 5 + ["append", "append", "tables", "tables", "rope", "rope", "table"])
    mix = rng.randrange(1000, 1 << 20)
    bs = rng.choice([16, 32, 64, 128])
    if op == "attend":
        while True:
            Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
            H = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
            if rng.random() < 0.5:
                q, B, ctx = rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 64), _log(rng, 1, 32768)
            else:
                B, q = rng.randint(1, 6), _log(rng, 8, 6000)
                ctx = _log(rng, q, 32768)
            if H <= 64 and B * H * q * ctx <= 1 << 31 and B * Hkv * ctx * D <= 1 << 31:
                break
        w = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        return dict(op=op, B=B, H=H, Hkv=Hkv, D=D, bs=bs, ctx=max(ctx, q), q=q, window=w, mix=mix)
    if op == "append":
        q = rng.choice([1, _log(rng, 1, 8192)])
        B = _log(rng, 1, 512) if q == 1 else rng.randint(1, max(1, 8192 // q))
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), bs=bs, ctx=max(q, _log(rng, 64, 16384) if B < 64 else 2048), q=q, mix=mix)
    if op == "tables":
        B = _log(rng, 1, 2000)
        q = rng.choice([1, _log(rng, 1, max(2, 1000000 // B))])
        return dict(op=op, B=B, bs=bs, ctx=max(q, _log(rng, 64, 131072 if B < 300 else 8192)), q=q, mix=mix)
    if op == "rope":
        D = rng.choice([64, 96, 128, 192, 256, 576])
        rot = rng.choice([r for r in (32, 64, 96, 128) if r <= D])
        H = _log(rng, 1, 128)
        T = _log(rng, 1, min(8192, (8192 * 40 * 128) // ((H + 8) * D)))
        return dict(op=op, T=T, H=H, Hk=rng.choice([1, 2, 8]), D=D, rot=rot, off=rng.choice([0, D - rot]), half=rng.random() < 0.5, inverse=rng.random() < 0.3,
                    far=_log(rng, 64, 1000000), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    kind = rng.choice(["none", "linear", "ntk", "yarn"])
    return dict(op="table", P=_log(rng, 500, 1000000), rot=rng.choice([32, 64, 64]), kind=kind, factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0, 40.0]), orig=rng.choice([4096, 8192, 32768]))


def _lens(c):
    """Context lengths and new tokens of each request (ragged, the first the longest), from the case alone."""
    r = np.random.RandomState(c["mix"])
    B, ctx, q = c["B"], c["ctx"], c["q"]
    lens = np.exp(r.uniform(math.log(max(1, ctx // 32)), math.log(ctx + 1), B)).astype(np.int64).clip(1, ctx)
    lens[0] = ctx
    ql = np.ones(B, np.int64) if q == 1 else r.randint(1, q + 1, B)
    ql[0] = q
    return np.maximum(lens, ql), ql


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _pages(c, lens, gen):
    """A random block table over a pool that just holds the requests, and its number of blocks."""
    nb = -(-lens // c["bs"])
    total = int(nb.sum())
    width = int(nb.max())
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    start = torch.from_numpy(np.cumsum(nb) - nb).to(DEV)
    j = torch.arange(width, device=DEV)
    at = start[:, None] + j[None, :]
    keep = j[None, :] < torch.from_numpy(nb).to(DEV)[:, None]
    return torch.where(keep, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).contiguous(), total


def _cache(total, c, gen):
    """Codes and scales of one side of the cache: heads of different size, each block with its own largest value."""
    size = torch.rand((total, c["Hkv"], 1, 1), generator=gen, device=DEV) * 1.5 + 0.25
    x = torch.randn((total, c["Hkv"], c["bs"], c["D"]), generator=gen, device=DEV) * size
    s = x.abs().amax((2, 3)) / 448.0
    return (x / s[:, :, None, None]).to(FP8).view(torch.uint8), s


def _start(ql):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)).to(DEV)


def _slots(table, lens, ql, bs):
    """The slots of each request's last ql tokens, in order."""
    b = np.repeat(np.arange(len(ql)), ql)
    pos = np.concatenate([np.arange(n - q, n) for n, q in zip(lens, ql)])
    b, pos = torch.from_numpy(b).to(DEV), torch.from_numpy(pos).to(DEV)
    return table[b, pos // bs].long() * bs + pos % bs


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c=c)
    if c["op"] == "attend":
        lens, ql = _lens(c)
        table, total = _pages(c, lens, g)
        s["kc"], s["ks"] = _cache(total, c, g)
        s["vc"], s["vs"] = _cache(total, c, g)
        s["q"] = torch.randn((int(ql.sum()), c["H"], c["D"]), generator=g, device=DEV).to(torch.bfloat16)
        s.update(table=table, lens=torch.from_numpy(lens.astype(np.int32)).to(DEV), start=_start(ql), scale=1.0 / math.sqrt(c["D"]))
    elif c["op"] == "append":
        lens, ql = _lens(c)
        table, total = _pages(c, lens, g)
        s["kc"], s["ks"] = _cache(total, c, g)
        s["vc"], s["vs"] = _cache(total, c, g)
        T = int(ql.sum())
        for n in ("k", "v"):
            s[n] = (torch.randn((T, c["Hkv"], c["D"]), generator=g, device=DEV) * (torch.rand((T, c["Hkv"], 1), generator=g, device=DEV) + 0.5)).to(torch.bfloat16)
        s.update(slots=_slots(table, lens, ql, c["bs"]), start=_start(ql))
    elif c["op"] == "tables":
        lens, ql = _lens(c)
        r = np.random.RandomState(int(seed) % (1 << 31))
        width = int(-(-lens.max() // c["bs"]))
        held = -(-(lens - ql) // c["bs"])
        cap = int((-(-lens // c["bs"])).sum()) + c["B"] + 100  # blocks of the pool
        ends = r.rand(c["B"]) < 0.05  # requests that have ended: they give their blocks back
        ends[0] = False
        lens, ql = np.where(ends, 0, lens), np.where(ends, 0, ql)
        held = np.where(ends, np.maximum(held, 1), held).clip(0, width)
        perm = r.permutation(cap).astype(np.int32)
        table = np.full((c["B"], width), -1, np.int32)
        at = np.cumsum(held) - held
        mask = np.arange(width)[None, :] < held[:, None]
        table[mask] = perm[(at[:, None] + np.arange(width)[None, :])[mask]]
        head, count = int(r.randint(cap)), cap - int(held.sum())
        ring = np.full(cap, -1, np.int32)
        ring[(head + np.arange(count)) % cap] = perm[int(held.sum()):]
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)  # noqa: E731
        # a step's buffers are as long as its longest batch, as a captured step has them
        T = _capacity(c)
        s.update(lens=up(lens), ql=up(ql), held=up(held), table=up(table), ring=up(ring), state=up([head, count]), T=T, held_out=torch.empty(c["B"], dtype=torch.int32, device=DEV),
                 state_out=torch.empty(2, dtype=torch.int32, device=DEV), start=torch.empty(c["B"] + 1, dtype=torch.int32, device=DEV), pos=torch.empty(T, dtype=torch.int64, device=DEV),
                 slots=torch.empty(T, dtype=torch.int64, device=DEV), req=torch.empty(T, dtype=torch.int32, device=DEV), counts=torch.empty(4, dtype=torch.int32, device=DEV))
    elif c["op"] == "rope":
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[c["dtype"]]
        s["q"] = torch.randn((c["T"], c["H"], c["D"]), generator=g, device=DEV).to(dt)
        s["k"] = torch.randn((c["T"], c["Hk"], c["D"]), generator=g, device=DEV).to(dt)
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=g, device=DEV)
        f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        a = torch.arange(c["far"], device=DEV, dtype=torch.float64)[:, None] * f[None, :]
        s["cs"] = torch.cat([a.cos(), a.sin()], 1).float()
        s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        r = np.random.RandomState(int(seed) % (1 << 31))
        # the base differs from model to model, and from seed to seed here
        s["base"] = float(np.exp(r.uniform(math.log(1e4), math.log(1e6))))
        s["out"] = torch.empty((c["P"], c["rot"]), device=DEV)
    return s


def _capacity(c):
    """Tokens that the buffers of a maps step hold: its new tokens, up to the next 64."""
    return -(-int(_lens(c)[1].sum()) // 64) * 64


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "append": _append, "tables": _tables, "rope": _rope, "table": _table}[s["c"]["op"]](s)


def _own(s):
    from sparse_mla_attention_04_gb300 import binding as b
    c = s["c"]
    if c["op"] == "attend":
        out, lse = b.smla_kv8_attn_fwd(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["start"], s["scale"], max_query_len=c["q"], window=c["window"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        b.smla_kv8_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        return {"k": s["kc"].view(FP8), "v": s["vc"].view(FP8), "ks": s["ks"], "vs": s["vs"]}
    if c["op"] == "tables":
        b.smla_build_block_tables(s["lens"], s["ql"], s["held"], s["table"], s["ring"], s["state"], block_size=c["bs"], blocks_held_out=s["held_out"], ring_state_out=s["state_out"],
                                  query_start=s["start"], positions=s["pos"], slot_mapping=s["slots"], token_request=s["req"], counts=s["counts"])
        return {n: s[n] for n in ("table", "ring", "held_out", "state_out", "start", "pos", "slots", "req", "counts")}
    if c["op"] == "rope":
        b.smla_rope(s["q"], s["k"], s["pos"], s["cs"], rot_offset=c["off"], is_neox=c["half"], inverse=c["inverse"], q_out=s["qo"], k_out=s["ko"])
        return {"q": s["qo"], "k": s["ko"]}
    return b.smla_rope_cos_sin_cache(c["P"], c["rot"], base=s["base"], scaling=c["kind"], factor=c["factor"], original_max_position=c["orig"], out=s["out"])


def _attend(s):
    """Every request padded to the longest: gather, dequantise, scores, softmax, values."""
    c, q, bs = s["c"], s["q"], s["c"]["bs"]
    B, H, Hkv, D, G, Q, L = c["B"], c["H"], c["Hkv"], c["D"], c["H"] // c["Hkv"], c["q"], c["ctx"]
    T = q.shape[0]
    nb = -(-L // bs)
    table = s["table"][:, :nb].clamp(min=0).long()

    def gathered(codes, scales):
        x = codes.view(FP8)[table].float() * scales[table][..., None, None]  # [B, nb, Hkv, bs, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * bs, D)[:, :, :L]

    lens, start = s["lens"].long(), s["start"].long()
    ql = start[1:] - start[:-1]
    i, j = torch.arange(Q, device=DEV), torch.arange(L, device=DEV)
    qp = q[(start[:-1, None] + i).clamp(max=T - 1)].float() * s["scale"]  # [B, Q, H, D]
    qp = qp.reshape(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    x = (qp @ gathered(s["kc"], s["ks"]).transpose(2, 3)).view(B, Hkv, G, Q, L)
    pos = (lens - ql)[:, None] + i
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
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


def _append(s):
    slots, bs = s["slots"], s["c"]["bs"]
    blk, off = slots // bs, slots % bs
    first = slots[s["start"][:-1].long()]  # each request's first new token: its block may hold older ones
    fb, fo = first // bs, first % bs
    for n in ("k", "v"):
        x, codes, scales = s[n].float(), s[n + "c"], s[n + "s"]
        new = torch.zeros_like(scales).index_reduce_(0, blk, x.abs().amax(-1), "amax")
        new = torch.where(new > 0, (new / 448.0).clamp(min=2.0 ** -60), torch.ones_like(new))
        old = scales[fb]
        grown = torch.where((fo > 0)[:, None], torch.maximum(old, new[fb]), new[fb])
        new[fb] = grown
        keep = torch.arange(bs, device=DEV)[None, :] < fo[:, None]  # the older tokens
        was = codes[fb].view(FP8).float()  # [B, Hkv, bs, D]
        now = (was * old[..., None, None] / grown[..., None, None]).clamp(-448, 448)
        codes[fb] = torch.where(keep[:, None, :, None], now, was).to(FP8).view(torch.uint8)
        codes[blk, :, off] = (x / new[blk][..., None]).clamp(-448, 448).to(FP8).view(torch.uint8)
        scales[blk] = new[blk]
    return {"k": s["kc"].view(FP8), "v": s["vc"].view(FP8), "ks": s["ks"], "vs": s["vs"]}


def _tables(s):
    bs, table, ring, cap, T = s["c"]["bs"], s["table"], s["ring"], s["ring"].numel(), s["T"]
    lens, ql, held = s["lens"].long(), s["ql"].long(), s["held"].long()
    head, count = s["state"][0].long(), s["state"][1].long()
    need = (lens + bs - 1) // bs
    new, rel = (need - held).clamp(min=0), (held - need).clamp(min=0)
    short = (new.sum() - count).clamp(min=0) + (need - table.shape[1]).clamp(min=0).sum()
    ok = short == 0
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    gets = ok & (j >= held[:, None]) & (j < need[:, None])
    gives = ok & (j >= need[:, None]) & (j < held[:, None])
    k = (new.cumsum(0) - new)[:, None] + j - held[:, None]
    r = (rel.cumsum(0) - rel)[:, None] + j - need[:, None]
    at = torch.where(gives, (head + count + r) % cap, cap)  # what gives nothing goes to a place past the ring
    ring.copy_(torch.cat([ring, ring[:1]]).scatter_(0, at.reshape(-1), table.reshape(-1))[:cap])
    table.copy_(torch.where(gets, ring[((head + k) % cap).clamp(0, cap - 1)], table))
    a, d = torch.where(ok, new.sum(), 0), torch.where(ok, rel.sum(), 0)
    held_out = torch.where(ok, need, held)
    end = ql.cumsum(0)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(end, t, right=True)
    live = t < end[-1]
    b = torch.where(live, b, 0)
    pos = torch.where(live, lens[b] - ql[b] + t - (end - ql)[b], 0)
    page = table[b, (pos // bs).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (pos // bs < held_out[b]), page * bs + pos % bs, -1)
    i32 = torch.int32
    return {"table": table, "ring": ring, "held_out": held_out.to(i32), "state_out": torch.stack([(head + a) % cap, count - a + d]).to(i32), "start": torch.cat([end[:1] * 0, end]).to(i32),
            "pos": pos, "slots": slots, "req": torch.where(live, b, -1).to(i32), "counts": torch.stack([end[-1], a, d, short]).to(i32)}


def _rope(s):
    c, n = s["c"], s["c"]["rot"] // 2
    row = s["cs"][s["pos"]]
    cos, sin = row[:, None, :n], row[:, None, n:]
    sin = -sin if c["inverse"] else sin

    def turned(x):
        y = x.clone()
        part = x[..., c["off"]: c["off"] + 2 * n].float()
        a, b = (part[..., :n], part[..., n:]) if c["half"] else (part[..., 0::2], part[..., 1::2])
        p, r = a * cos - b * sin, b * cos + a * sin
        y[..., c["off"]: c["off"] + 2 * n] = (torch.cat([p, r], -1) if c["half"] else torch.stack([p, r], -1).flatten(-2)).to(x.dtype)
        return y

    return {"q": turned(s["q"]), "k": turned(s["k"])}


def _table(s):
    c, base, d = s["c"], s["base"], s["c"]["rot"]
    i = torch.arange(0, d, 2, device=DEV, dtype=torch.float64)
    if c["kind"] == "ntk":
        base = base * c["factor"] ** (d / (d - 2))
    f = base ** (-i / d)
    m = 1.0
    if c["kind"] == "linear":
        f = f / c["factor"]
    if c["kind"] == "yarn":
        # pairs that turn more than 32 times over the old context stay, those that turn less than once are stretched
        low, high = (d * math.log(c["orig"] / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
        m = 0.1 * math.log(c["factor"]) + 1.0
    a = torch.arange(c["P"], device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos() * m, a.sin() * m], 1).float()


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "attend":
        lens, ql = _lens(c)
        T = int(ql.sum())
        first = np.maximum(0, lens - ql + 1 - c["window"]) if c["window"] else np.zeros_like(lens)
        kv = int((lens - first).sum())
        pairs = 0
        for n, q in zip(lens, ql):
            seen = np.arange(n - q + 1, n + 1)
            pairs += int(np.minimum(seen, c["window"]).sum() if c["window"] else seen.sum())
        return {"bytes": kv * c["Hkv"] * (2 * c["D"] + 8 / c["bs"]) + T * c["H"] * (4 * c["D"] + 4), "flops": 4.0 * c["D"] * c["H"] * pairs}
    if c["op"] == "append":
        n = int(_lens(c)[1].sum()) * c["Hkv"] * c["D"] * 2
        return {"bytes": 3.0 * n, "flops": 3.0 * n}
    if c["op"] == "tables":
        lens, ql = _lens(c)
        return {"bytes": 20.0 * _capacity(c) + 20.0 * c["B"] + 8.0 * float((ql / c["bs"]).sum()), "flops": 4.0 * int(ql.sum())}
    if c["op"] == "rope":
        n = c["T"] * (c["H"] + c["Hk"])
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2.0 * n * c["D"] * size + c["T"] * (8 + 4 * c["rot"]), "flops": 3.0 * n * c["rot"]}
    return {"bytes": 4.0 * c["P"] * c["rot"], "flops": 2.0 * c["P"] * c["rot"]}


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
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    if c["op"] == "attend":
        lens, ql = _lens(c)
        G, bs = c["H"] // c["Hkv"], c["bs"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        at = 0
        for b, (n, q) in enumerate(zip(lens.tolist(), ql.tolist())):
            pages = s["table"][b, : -(-n // bs)].long()
            for h in range(c["Hkv"]):
                k, v = ((s[x + "c"][pages, h].view(FP8).double() * s[x + "s"][pages, h].double()[:, None, None]).reshape(-1, c["D"])[:n] for x in "kv")
                for lo in range(0, q, 2048):  # rows at a time
                    hi = min(q, lo + 2048)
                    p = torch.arange(n - q + lo, n - q + hi, device=DEV)
                    j = torch.arange(n, device=DEV)
                    hide = j[None, :] > p[:, None]
                    if c["window"]:
                        hide |= j[None, :] <= p[:, None] - c["window"]
                    for g in range(G):
                        x = (s["q"][at + lo: at + hi, h * G + g].double() @ k.T) * s["scale"]
                        x = x.masked_fill(hide, -math.inf)
                        z = torch.logsumexp(x, 1)
                        lse[at + lo: at + hi, h * G + g] = z
                        out[at + lo: at + hi, h * G + g] = torch.exp(x - z[:, None]) @ v
            at += q
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        lens, ql = _lens(c)
        bs, res = c["bs"], {}
        slots = s["slots"].tolist()
        runs, at = [], 0  # (block, first offset, first token, tokens)
        for q in ql.tolist():
            t = at
            while t < at + q:
                n = min(bs - slots[t] % bs, at + q - t)
                runs.append((slots[t] // bs, slots[t] % bs, t, n))
                t += n
            at += q
        for x in "kv":
            val, sc = s[x + "c"].view(FP8).double(), s[x + "s"].double()
            src = s[x].double()
            for blk, off, t, n in runs:
                rows = src[t: t + n].transpose(0, 1)  # [Hkv, n, D]
                amax = rows.abs().amax((1, 2))
                now = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -60), torch.ones_like(amax))
                if off > 0:
                    now = torch.maximum(now, sc[blk])
                    val[blk, :, :off] = _round_e4m3(val[blk, :, :off] * (sc[blk] / now)[:, None, None])
                val[blk, :, off: off + n] = _round_e4m3(rows / now[:, None, None])
                sc[blk] = now
            res[x], res[x + "s"] = val, sc
        return res
    if c["op"] == "rope":
        n = c["rot"] // 2
        row = s["cs"].double()[s["pos"]]
        z = torch.complex(row[:, :n], row[:, n:])[:, None, :]
        if c["inverse"]:
            z = z.conj()
        res = {}
        for x in "qk":
            y = s[x].double()
            part = y[..., c["off"]: c["off"] + c["rot"]].clone()
            pair = part.reshape(*part.shape[:2], 2, n).transpose(2, 3) if c["half"] else part.reshape(*part.shape[:2], n, 2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            y[..., c["off"]: c["off"] + c["rot"]] = (w.transpose(2, 3) if c["half"] else w).reshape(part.shape)
            res[x] = y
        return res
    d, base, k = c["rot"], s["base"], c["factor"]
    if c["kind"] == "ntk":
        base *= k ** (d / (d - 2.0))
    freq = np.array([base ** (-2.0 * i / d) for i in range(d // 2)])
    mult = 1.0
    if c["kind"] == "linear":
        freq = freq / k
    elif c["kind"] == "yarn":
        border = [0.5 * d * math.log(c["orig"] / (2 * math.pi * turns)) / math.log(base) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(border[0])), min(d - 1, math.ceil(border[1]))
        stretch = np.clip((np.arange(d // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        freq = freq * (1.0 - stretch + stretch / k)
        mult = 1.0 + 0.1 * math.log(k)
    ang = torch.outer(torch.arange(c["P"], dtype=torch.float64), torch.from_numpy(freq))
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1) * mult
