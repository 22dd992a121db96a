"""The block-scaled 8-bit cache: its write against the binary32 rules (bits),
and attention over it against a plain binary64 implementation.

Tolerances of the attention, derived: out is rounded once to bf16 (2^-8 of the
value at most); the weights are rounded to binary16 (2^-11 relative, 2^-25
absolute of a reference that the largest weight reaches to 2^-8 or above, so
2^-16 n max|V| covers n of them) and come from logits in binary32. A logit's
error is below 2^-18 of its reach scale * sum |q| |K| (eight partial sums in
binary32 with truncation, three products, a base-2 exponential of 2^-22), which
moves weights and lse by that much: together (2^-11 + 2^-17 (1 + reach)) * sum
p |V| for out and 2^-18 (1 + reach) for lse."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the write
def _fresh(nb, hk, bs, D, seed):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (nb, hk, bs, D), generator=g, dtype=torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0                              # no NaN codes
    scales = [torch.rand((nb, hk), generator=g) * 0.02 + 0.001 for _ in range(2)]
    return codes, scales


def _append_both(k, v, slots, codes, scales, **kw):
    want_c, want_s = [c.clone() for c in codes], [s.clone() for s in scales]
    for x, c, s in zip((k, v), want_c, want_s):
        ref.append(x.cpu(), slots, c, s)
    got_c, got_s = [c.to(DEV) for c in codes], [s.to(DEV) for s in scales]
    binding.smla_kv8_append(k, v, slots.to(DEV), *got_c, *got_s, **kw)
    torch.cuda.synchronize()
    for g, w in zip(got_s, want_s):
        assert torch.equal(g.cpu(), w)
    for g, w in zip(got_c, want_c):
        same = g.cpu() == w
        both_nan = ((g.cpu() & 0x7F) == 0x7F) & ((w & 0x7F) == 0x7F)
        assert bool((same | both_nan).all())
    return got_c, got_s


@pytest.mark.parametrize("hk,D,bs,runs", [
    (1, 64, 16, [(0, 1)]), (2, 128, 64, [(0, 1), (70, 1), (191, 1)]), (8, 128, 64, [(5, 200)]),
    (3, 64, 32, [(31, 1), (40, 17), (96, 64)]), (4, 128, 128, [(0, 128), (255, 2)]), (2, 64, 128, [(1, 383)]),
    (1, 128, 16, [(i * 16 + i % 16, 1) for i in range(40)]), (8, 64, 16, [(3, 1000)]),
    (5, 128, 32, [(i * 64 + 7, 9) for i in range(60)]),
    (8, 64, 16, [(i * 16 + 3, 1) for i in range(1500)]),       # a large decode step
    (8, 128, 64, [(i * 64 + i % 60, 1 + i % 4) for i in range(500)] + [(40000, 900)])])   # single tokens, then a prompt
@pytest.mark.parametrize("loud", [False, True])
def test_append_bits(hk, D, bs, runs, loud):
    """Runs (first slot, tokens) in whole and part blocks; loud: new values that make the blocks' scales grow."""
    g = torch.Generator().manual_seed(hk * D + bs)
    slots = torch.cat([torch.arange(a, a + n) for a, n in runs])
    T, nb = len(slots), int(slots.max()) // bs + 2
    k, v = ((torch.randn((T, hk, D), generator=g) * (40.0 if loud else 0.5)).to(torch.bfloat16).to(DEV) for _ in range(2))
    _append_both(k, v, slots, *_fresh(nb, hk, bs, D, 1))


def test_append_skips_strides_and_special_values():
    hk, D, bs, nb = 2, 128, 64, 6
    g = torch.Generator().manual_seed(3)
    slots = torch.tensor([10, 11, -1, 130, 131, 132, -1, -1, 200, 320, 321])
    wide = torch.randn((len(slots), hk + 1, 2 * D + 16), generator=g).to(torch.bfloat16).to(DEV)
    k, v = wide[:, 1:, 8:8 + D], wide[:, :hk, D + 16:]
    k[0, 0, 3], k[1, 1, 5], k[4, 0, 0], v[3, 1, 9] = math.inf, -math.inf, math.nan, math.nan
    v[8] = 0.0                                                 # a block of zeros: scale 1
    k[9:] = 1e-30                                              # below the smallest scale
    _append_both(k, v, slots, *_fresh(nb, hk, bs, D, 2))
    assert binding.smla_device_error(reset=True) == 0


def test_append_slots_past_the_pool():
    binding.smla_device_error(reset=True)
    hk, D, bs, nb = 1, 64, 16, 3
    slots = torch.tensor([47, 48, 1 << 40, 5])
    k = torch.randn((4, hk, D)).to(torch.bfloat16).to(DEV)
    _append_both(k, k.clone(), slots, *_fresh(nb, hk, bs, D, 4))
    assert binding.smla_device_error(reset=True) == 8


def test_append_same_slot_twice_keeps_one_of_the_two():
    hk, D, bs = 1, 64, 16
    (kc, vc), (ks, vs) = _fresh(2, hk, bs, D, 5)
    k = torch.randn((2, hk, D)).to(torch.bfloat16).to(DEV)
    kc, vc, ks, vs = (x.to(DEV) for x in (kc, vc, ks, vs))
    binding.smla_kv8_append(k, k, torch.tensor([4, 4], device=DEV), kc, vc, ks, vs)
    row = kc[0, 0, 4].view(FP8).float() * ks[0, 0]
    err = (row[None] - k[:, 0].float()).abs().amax(-1) / k.float().abs().amax()
    assert float(err.min()) <= 2.0 ** -4


# ------------------------------------------------------------------ the attention
def _problem(H, hk, D, bs, lens, ql, seed, extra=3, pad=0):
    """A cache of random blocks in random order; stale garbage (NaN codes among it) wherever no token is."""
    g = torch.Generator().manual_seed(seed)
    nblk = [-(-max(n, 0) // bs) for n in lens]
    total = sum(nblk) + extra
    perm = torch.randperm(total, generator=g)
    width = max(max(nblk), 1) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    kc, vc = (torch.randint(0, 256, (total, hk, bs, D), generator=g, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.rand((total, hk), generator=g) * 0.01 + 0.002 for _ in range(2))
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n].int()
        at += n
        for j in range(n):
            blk = int(table[b, j])
            m = min(bs, lens[b] - j * bs)
            for c, s in ((kc, ks), (vc, vs)):
                x = torch.randn((hk, m, D), generator=g) * (0.2 + 2 * torch.rand((hk, 1, 1), generator=g))
                sc = x.abs().amax((1, 2)) / 448
                s[blk] = sc
                c[blk, :, :m] = (x / sc[:, None, None]).to(FP8).view(torch.uint8)
    T = sum(ql)
    q = torch.randn((T + pad, H, D), generator=g).to(torch.bfloat16)
    start = torch.tensor([0] + list(np.cumsum(ql)), dtype=torch.int32)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32), start=start,
                scale=1.0 / math.sqrt(D), max_q=max(max(ql), 1))


def _run(p, window=0, sinks=None, **kw):
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    q = kw.pop("q", d["q"])
    table = kw.pop("table", d["table"])
    return binding.smla_kv8_attn_fwd(q, d["kc"], d["vc"], d["ks"], d["vs"], table, d["lens"], d["start"], p["scale"],
                                     max_query_len=kw.pop("max_query_len", p["max_q"]), window=window,
                                     sinks=None if sinks is None else sinks.to(DEV), **kw)


def _check(p, got, window=0, sinks=None):
    out, lse = got
    torch.cuda.synchronize()
    T = int(p["start"][-1])
    want, z, w, reach = ref.attention(p["q"][:T], p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], p["start"],
                                      p["scale"], window, sinks)
    n = p["lens"].clamp(min=0).max().double()
    top = (p["vs"].double() * 448).max()
    o, l = out[:T].cpu().double(), lse[:T].cpu().double()
    have = torch.isfinite(want)
    assert torch.equal(have, torch.isfinite(o)), "finite values in other places"
    tol = want.abs() * 2.0 ** -8 + w * (2.0 ** -11 + 2.0 ** -17 * (1 + reach[..., None])) + n * top * 2.0 ** -16 * 2.0 ** -8
    bad = ((o - want).abs() > tol) & have
    assert not bool(bad.any()), (int(bad.sum()), float(((o - want).abs() / tol)[have].max()))
    fin = torch.isfinite(z)
    assert torch.equal(torch.isinf(z), torch.isinf(l)) and torch.equal(torch.isnan(z), torch.isnan(l))
    assert bool(((l - z).abs() <= 2.0 ** -18 * (1 + reach))[fin].all()), float((l - z).abs()[fin].max())


SHAPES = [
    # H, H_kv, D, block, lens, new tokens
    (1, 1, 64, 16, [1], [1]),
    (8, 1, 128, 64, [509], [1]),
    (4, 2, 128, 64, [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300], [1] * 11),
    (6, 2, 64, 16, [5, 333, 16, 1, 48], [1, 1, 1, 1, 1]),
    (32, 8, 128, 32, [1000, 3, 77], [1, 1, 1]),
    (16, 1, 128, 128, [700, 129], [1, 1]),
    (10, 2, 64, 64, [130, 65], [1, 1]),
    (8, 2, 128, 16, [40, 17, 90], [4, 2, 3]),                  # several new tokens: 16 rows and less
    (5, 1, 64, 32, [100, 33], [7, 33]),
    (8, 8, 128, 64, [70], [70]),                               # a whole prompt, one query head each
    (12, 4, 64, 16, [200, 5, 1], [37, 5, 1]),
    (16, 2, 128, 64, [300, 64, 129], [150, 64, 2]),
    (4, 1, 128, 64, [3, 0, 200, 10], [5, 2, 0, 10]),           # more new tokens than positions, none, an idle request
    (64, 2, 64, 128, [257], [9]),
    (3, 1, 128, 32, [513], [200]),
    (2, 2, 64, 64, [390, 128, 129], [390, 128, 1]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_attention(shape, window):
    p = _problem(*shape, seed=len(shape[4]) + shape[0])
    _check(p, _run(p, window), window)


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[7], SHAPES[11], SHAPES[12]])
def test_sinks(shape):
    p = _problem(*shape, seed=9)
    sinks = torch.linspace(-3.0, 4.0, shape[0])
    _check(p, _run(p, sinks=sinks), sinks=sinks)
    sinks[0] = -math.inf
    _check(p, _run(p, 20, sinks), 20, sinks)


@pytest.mark.parametrize("ql", [[1, 1], [9, 40], [150, 200]])
def test_rows_behind_the_last_sequence_are_left(ql):
    p = _problem(8, 2, 128, 64, [70, 210], ql, seed=4, pad=5)
    T = sum(ql)
    out = torch.full((T + 5, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 5, 8), 5.0, device=DEV)
    got = _run(p, out=out, lse=lse)
    _check(p, got)
    assert bool((out[T:] == 3.0).all()) and bool((lse[T:] == 5.0).all())


@pytest.mark.parametrize("ql", [[1, 1, 1], [30, 1, 64]])
def test_bad_pages_are_not_read(ql):
    """Entries outside the pool: their positions are seen by no one; a row may be left with nothing."""
    p = _problem(8, 2, 64, 16, [100, 40, 64], ql, seed=6)
    p["table"][0, 2], p["table"][0, 5] = -1, p["kc"].shape[0]
    p["table"][1, :3] = -5
    p["table"][2, 0] = 1 << 30
    _check(p, _run(p))


@pytest.mark.parametrize("ql", [[1, 1], [20, 7], [130, 1]])
def test_strided_queries_and_tables(ql):
    p = _problem(8, 2, 128, 64, [131, 20], ql, seed=7)
    T = sum(ql)
    wide = torch.zeros((8, T, 256), dtype=torch.bfloat16, device=DEV)
    wide[:, :, 64:192] = p["q"].to(DEV).transpose(0, 1)
    q = wide.transpose(0, 1)[:, :, 64:192]
    big = torch.full((2, p["table"].shape[1] + 9), 1 << 30, dtype=torch.int32, device=DEV)
    big[:, :p["table"].shape[1]] = p["table"].to(DEV)
    _check(p, _run(p, q=q, table=big[:, :p["table"].shape[1]]))


@pytest.mark.parametrize("ql,window", [([6], 0), ([40], 0), ([140], 0), ([40], 5), ([140], 33)])
def test_nan_values_reach_only_the_rows_that_see_them(ql, window):
    """NaN codes in V (and K) at positions that some of a chunk's rows see and others do not."""
    p = _problem(4, 1, 128, 64, [200], ql, seed=8)
    for pos, d in ((199, 3), (200 - ql[0] + 2, 77), (200 - ql[0] // 2, 5), (120, 9)):
        p["vc"][int(p["table"][0, pos // 64]), 0, pos % 64, d] = 0x7F
    _check(p, _run(p, window), window)
    pos = 200 - ql[0] // 2
    p["kc"][int(p["table"][0, pos // 64]), 0, pos % 64, 11] = 0xFF
    want = ref.attention(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], p["start"], p["scale"], window)
    out, lse = _run(p, window)
    assert torch.equal(torch.isnan(lse.cpu()), torch.isnan(want[1]))
    assert torch.equal(torch.isnan(out.cpu().float()), torch.isnan(want[0]))


@pytest.mark.parametrize("ql", [[1, 1], [100, 1]])
def test_scales_far_apart(ql):
    """Blocks whose value scales differ by 2^60 keep a right denominator."""
    p = _problem(4, 2, 128, 16, [160, 64], ql, seed=10)
    p["vs"][p["table"][0, 3].long()] *= 2.0 ** -50
    p["vs"][p["table"][0, 5].long()] *= 2.0 ** 10
    p["ks"][p["table"][1, 1].long()] *= 2.0 ** -30
    p["vs"][p["table"][1, 2].long()] = 2.0 ** -60
    _check(p, _run(p))


@pytest.mark.parametrize("ql", [[1], [50]])
def test_large_and_tiny_queries(ql):
    p = _problem(8, 2, 64, 32, [90], ql, seed=11)
    p["q"][:, 0] *= 1e30
    p["q"][:, 1] *= 1e-30
    p["q"][:, 2] = 0.0
    p["q"][:, 3, 0] = 300.0
    p["scale"] = 1e-3
    p["ks"] *= 1e-2
    want, z, _, _ = ref.attention(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], p["start"], p["scale"])
    p2 = dict(p)
    out, lse = _run(p)
    rest = [1, 2, 3, 4, 5, 6, 7]
    assert bool(torch.isfinite(out.cpu().float()).all())
    d = (out.cpu().double() - want).abs()[:, rest]
    assert float(d.max()) <= float(want.abs().max()) * 2.0 ** -7
    # logits of 10^28: the softmax is one-hot
    assert float((out.cpu().double() - want).abs()[:, 0].max()) <= float(want.abs().max()) * 2.0 ** -7
    assert p2 is not p


def test_infinite_and_nan_queries_stay_in_their_rows():
    p = _problem(8, 2, 64, 32, [90], [3], seed=12)
    p["q"][1, 3, 5] = math.nan
    p["q"][2, 0, 7] = math.inf
    out, lse = _run(p)
    o = out.cpu().float()
    nan = torch.isnan(o).all(-1)
    assert bool(nan[1, 3]) and bool(nan[2, 0]) and int(torch.isnan(o).any(-1).sum()) == 2
    assert bool(torch.isnan(lse.cpu()[1, 3])) and bool(torch.isnan(lse.cpu()[2, 0]))


@pytest.mark.parametrize("B,max_q", [(300, 1), (70, 20), (40, 300), (3, 200), (3, 30)])
def test_many_requests_and_long_contexts(B, max_q):
    """More units than blocks and units that span many blocks, against a dense binary64 product on the GPU."""
    r = np.random.RandomState(B)
    H, hk, D, bs = 8, 2, 128, 64
    lens = np.maximum(r.randint(1, 400, B), 1)
    lens[:3] = [20000, 9001, 4097]
    ql = np.minimum(r.randint(0, max_q + 1, B) if max_q > 1 else np.ones(B, int), lens)
    ql[:3] = max_q
    nblk = -(-lens // bs)
    g = torch.Generator(device=DEV).manual_seed(B)
    total = int(nblk.sum())
    kc, vc = (torch.randint(0, 0x78, (total, hk, bs, D), generator=g, device=DEV, dtype=torch.uint8) |
              (torch.randint(0, 2, (total, hk, bs, D), generator=g, device=DEV, dtype=torch.uint8) << 7) for _ in range(2))
    ks, vs = (torch.rand((total, hk), generator=g, device=DEV) * 0.004 + 0.002 for _ in range(2))
    perm = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.full((B, int(nblk.max())), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
    T = int(ql.sum())
    q = (torch.randn((T, H, D), generator=g, device=DEV) * 0.2).to(torch.bfloat16)
    start = torch.tensor(np.concatenate([[0], np.cumsum(ql)]), dtype=torch.int32, device=DEV)
    out, lse = binding.smla_kv8_attn_fwd(q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                         start, 0.1, max_query_len=max_q)
    at = 0
    for b in range(B):
        n, m = int(lens[b]), int(ql[b])
        pages = table[b, :nblk[b]].long()
        for h in range(hk):
            k, v = (ref.values(c[pages][:, h:h + 1], s[pages][:, h:h + 1]).reshape(-1, D)[:n] for c, s in ((kc, ks), (vc, vs)))
            x = q[at:at + m, h * 4:h * 4 + 4].double()
            s = torch.einsum("thd,nd->thn", x, k) * 0.1
            hide = torch.arange(n, device=DEV)[None] > torch.arange(n - m, n, device=DEV)[:, None]
            s = s.masked_fill(hide[:, None], -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            want = w @ v
            o = out[at:at + m, h * 4:h * 4 + 4].double()
            reach = torch.einsum("thd,nd->thn", x.abs(), k.abs()).amax(-1, keepdim=True) * 0.1
            tol = want.abs() * 2.0 ** -8 + (w @ v.abs()) * (2.0 ** -11 + 2.0 ** -17 * (1 + reach)) + 2.0 ** -24 * n * 448 * 0.006
            assert bool(((o - want).abs() <= tol).all()), (b, h, float(((o - want).abs() / tol).max()))
            assert bool(((lse[at:at + m, h * 4:h * 4 + 4].double() - z).abs() <= 2.0 ** -18 * (1 + reach[..., 0])).all())
        at += m


@pytest.mark.parametrize("ql", [1, 130])
def test_blocks_past_four_gigabytes(ql):
    """A pool whose codes lie past 2^32 bytes: the last blocks are read."""
    hk, bs, D, H = 8, 64, 128, 16
    nb = (1 << 32) // (hk * bs * D) + 1100
    kc, vc = (torch.empty((nb, hk, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty((nb, hk), device=DEV) for _ in range(2))
    pages = torch.tensor([nb - 1, 2, nb - 700], device=DEV)
    small = _problem(H, hk, D, bs, [150], [ql], seed=13, extra=0)
    src = small["table"][0, :3].long()
    for big, x in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
        big[pages] = small[x][src].to(DEV)
    out, lse = binding.smla_kv8_attn_fwd(small["q"].to(DEV), kc, vc, ks, vs, pages.int()[None].contiguous(),
                                         small["lens"].to(DEV), small["start"].to(DEV), small["scale"], max_query_len=ql)
    _check(small, (out, lse))
    # the write at the pool's end
    k = torch.randn((2, hk, D), device=DEV).to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 2, nb * bs - 1], device=DEV)
    binding.smla_kv8_append(k, k, slots, kc, vc, ks, vs)
    got = kc[nb - 1, :, bs - 2:].view(FP8).float() * ks[nb - 1][:, None, None]
    err = (got.transpose(0, 1) - k.float()).abs()
    # half a step of E4M3 (2^-4), or of its subnormals (2^-10 of the scale)
    assert bool((err <= k.float().abs() * 2.0 ** -4 + ks[nb - 1][None, :, None] * 2.0 ** -10).all())


@pytest.mark.parametrize("bound", [0, 1, 4, 1000])
def test_any_bound_of_the_new_tokens_gives_the_result(bound):
    """max_query_len chooses kernels only: a wrong one costs time, not results."""
    p = _problem(8, 2, 128, 64, [300, 20, 129], [140, 1, 3], seed=14)
    _check(p, _run(p, max_query_len=bound))


@pytest.mark.parametrize("ql", [[1, 1, 1, 1], [33, 1, 140, 8]])
def test_runs_are_the_same_bits_on_other_streams_and_in_graphs(ql):
    p = _problem(8, 2, 128, 64, [300, 700, 1000, 128], ql, seed=15)
    first = _run(p)
    side = torch.cuda.Stream()
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    args = (d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"], p["scale"])
    torch.cuda.synchronize()
    outs = [binding.smla_kv8_attn_fwd(*args, max_query_len=max(ql), stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    # two graphs captured on one stream, replayed at the same time on two
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = binding.smla_kv8_attn_fwd(*args, max_query_len=max(ql))
        graphs.append((gr, res))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (gr, _r), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for _g, (o, l) in graphs:
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])


def test_a_captured_call_follows_the_lengths():
    p = _problem(8, 2, 128, 64, [300, 700], [1, 1], seed=16)
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    gr = torch.cuda.CUDAGraph()
    binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"], p["scale"],
                              max_query_len=1)
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        out = binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"],
                                        p["scale"], max_query_len=1)
    for lens in ([1, 2], [64, 65], [299, 0], [300, 700]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        gr.replay()
        q = dict(p, lens=torch.tensor(lens, dtype=torch.int32))
        _check(q, out)


def test_refuses_overlapping_shapes():
    p = _problem(8, 2, 128, 64, [70], [1], seed=17)
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    with pytest.raises(ValueError):
        binding.smla_kv8_attn_fwd(d["q"][:, :7].contiguous(), d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"],
                                  d["start"], 0.1, max_query_len=1)
    with pytest.raises(ValueError):
        binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"][:1],
                                  0.1, max_query_len=1)
    with pytest.raises(binding.SmlaError):
        binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"], 0.1,
                                  max_query_len=1, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"].cpu(), d["vs"], d["table"], d["lens"], d["start"],
                                  0.1, max_query_len=1)
    with pytest.raises(ValueError):
        binding.smla_kv8_append(d["q"], d["q"], torch.zeros(1, dtype=torch.int64, device=DEV), d["kc"], d["vc"], d["ks"],
                                d["vs"])


@pytest.mark.parametrize("ql", [[1, 1, 1], [40, 1, 20]])
@pytest.mark.parametrize("bad", [math.nan, 0.0, math.inf])
def test_pages_below_the_window_may_be_gone(ql, bad):
    """Blocks that no token sees any more (a window moved on) hold anything, their scales too."""
    p = _problem(8, 2, 128, 16, [300, 170, 95], ql, seed=18)
    window = 37
    for b, n in enumerate((300, 170, 95)):
        first = max(0, n - ql[b] - window + 1)                 # the lowest position that a token sees
        for j in range(first // 16):
            blk = int(p["table"][b, j])
            p["ks"][blk], p["vs"][blk] = bad, bad
            p["kc"][blk], p["vc"][blk] = 0x7F, 0x7F
    out, lse = _run(p, window)
    for b, n in enumerate((300, 170, 95)):                     # the reference multiplies what it masks
        for j in range(max(0, n - ql[b] - window + 1) // 16):
            blk = int(p["table"][b, j])
            p["ks"][blk], p["vs"][blk] = 1.0, 1.0
            p["kc"][blk], p["vc"][blk] = 0, 0
    _check(p, (out, lse), window)


@pytest.mark.parametrize("ql", [[1, 1], [30, 90]])
def test_an_empty_pool_and_a_table_without_width(ql):
    """Nothing is there to see: out 0, lse -inf (the sink with sinks)."""
    T, H, D = sum(ql), 4, 64
    q = torch.randn((T, H, D), device=DEV).to(torch.bfloat16)
    start = torch.tensor([0, ql[0], T], dtype=torch.int32, device=DEV)
    lens = torch.tensor([100, 120], dtype=torch.int32, device=DEV)
    sinks = torch.linspace(-1.0, 2.0, H, device=DEV)
    for nb, width in ((0, 4), (5, 0), (0, 0)):
        kc, vc, ks, vs = binding.new_kv8_cache(nb, 2, 32, D, device=DEV)
        table = torch.zeros((2, width), dtype=torch.int32, device=DEV)
        for s in (None, sinks):
            out, lse = binding.smla_kv8_attn_fwd(q, kc, vc, ks, vs, table, lens, start, 0.1, max_query_len=max(ql), sinks=s)
            assert bool((out == 0).all())
            want = torch.full((T, H), -math.inf, device=DEV) if s is None else s.expand(T, H)
            assert torch.allclose(lse, want, rtol=2.0 ** -18, atol=2.0 ** -18)
    assert binding.smla_device_error(reset=True) == 0


@pytest.mark.parametrize("ql", [[1, 1], [60, 70]])
def test_lengths_beyond_the_table_and_the_widest_windows(ql):
    """seq_lens are cut to the table; a window of everything is none."""
    p = _problem(8, 2, 64, 16, [96, 64], ql, seed=19)
    width = 6
    cut = dict(p, table=p["table"][:, :width].contiguous())
    cut["table"][1, 4:] = -1
    long = dict(cut, lens=torch.tensor([2 ** 31 - 1, 64], dtype=torch.int32))
    got = _run(long, 2 ** 31 - 1)
    _check(dict(cut, lens=torch.tensor([96, 64], dtype=torch.int32)), got)


@pytest.mark.parametrize("ql", [1, 150])
def test_starts_that_overlap_stay_within_the_buffers(ql):
    """Requests that name the same tokens again (an error of the caller): some result in
    their rows, the other rows and everything outside as they were."""
    p = _problem(8, 2, 128, 64, [200] * 6, [ql] * 6, seed=20, pad=2)
    T = 6 * ql
    p["start"] = torch.tensor([0, T, 0, T, 0, T, 0], dtype=torch.int32)
    out = torch.full((T + 2, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    c = binding._KV8_ATTN_PARAMS
    need = binding.lib().smla_kv8_attn_workspace_size_of(c.pack(c.size, *([0] * 10), p["table"].shape[1], 0, 0, 6, T + 2, 8, 2, 128,
                                                                64, ql, 0, 0.0, 0, 0, 0, 0, 0, 0))
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    _run(p, out=out, workspace=room[:need])
    torch.cuda.synchronize()
    assert bool((out[T:] == 3.0).all()) and bool((room[need:] == 0x5A).all())


@pytest.mark.parametrize("ql", [[1, 1, 1], [70, 130, 1]])
def test_strides_of_single_rows_and_of_own_workspaces(ql):
    """H = 1 with any head stride; a workspace of the caller, used again and again."""
    p = _problem(1, 1, 64, 32, [90, 150, 31], ql, seed=21)
    T = sum(ql)
    flat = torch.zeros((T, 64 + 8), dtype=torch.bfloat16, device=DEV)
    flat[:, :64] = p["q"].to(DEV)[:, 0]
    q = flat.as_strided((T, 1, 64), (72, 3, 1))
    room = torch.full((binding.smla_kv8_attn_workspace_size(3, T, 1, 1, 64, max(ql)),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        _check(p, _run(p, q=q, workspace=room))


def test_append_of_nothing_and_of_one_head():
    hk, D, bs, nb = 1, 128, 16, 3
    codes, scales = _fresh(nb, hk, bs, D, 9)
    _append_both(torch.empty((0, hk, D), dtype=torch.bfloat16, device=DEV), torch.empty((0, hk, D), dtype=torch.bfloat16, device=DEV),
                 torch.empty(0, dtype=torch.int64), codes, scales)
    rows = torch.randn((5, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    k = rows.as_strided((5, 1, D), (D, 7, 1))
    _append_both(k, k, torch.arange(3, 8), codes, scales)


@pytest.mark.parametrize("ql", [[1, 400, 3, 0, 1, 64], [200, 1, 1, 1, 33, 129]])
def test_prompts_and_single_tokens_in_one_call(ql):
    """A batch that mixes prompts with decoding requests: row tiles without rows beside full ones."""
    p = _problem(8, 2, 128, 16, [900, 400, 2000, 50, 1, 64] if ql[0] == 1 else [200, 3000, 17, 1, 33, 700], ql, seed=22)
    _check(p, _run(p))
    _check(p, _run(p, 100), 100)
    assert binding.smla_device_error(reset=True) == 0


@pytest.mark.parametrize("H,hk,D,B,q", [(16, 2, 128, 1, 1), (32, 8, 128, 64, 1), (8, 8, 64, 3, 2), (8, 1, 64, 5, 300)])
def test_the_workspace_of_a_call_is_within_the_bound(H, hk, D, B, q):
    """And a call runs in exactly what it asks for, whatever the table's width."""
    bound = binding.smla_kv8_attn_workspace_size(B, B * q, H, hk, D, q)
    for width in (0, 1, 7, 600):
        kc, vc, ks, vs = binding.new_kv8_cache(4, hk, 16, D, device=DEV)
        kc.fill_(0x30)
        vc.fill_(0x38)                                         # 1.0 everywhere
        table = torch.arange(width, device=DEV).remainder(4).int().repeat(B, 1)
        lens = torch.full((B,), max(width * 16 - 3, 0), dtype=torch.int32, device=DEV)
        start = torch.arange(0, B * q + 1, q, dtype=torch.int32, device=DEV)
        x = torch.randn((B * q, H, D), device=DEV).to(torch.bfloat16)
        p = binding._KV8_ATTN_PARAMS
        need = binding.lib().smla_kv8_attn_workspace_size_of(p.pack(p.size, *([0] * 10), width, 0, 0, B, B * q, H, hk, D, 16, q,
                                                                    0, 0.0, 0, 0, 0, 0, 0, 0))
        assert 0 < need <= bound
        room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        out, _ = binding.smla_kv8_attn_fwd(x, kc, vc, ks, vs, table, lens, start, 0.1, max_query_len=q, workspace=room[:need])
        seen = (torch.arange(B * q, device=DEV) % q + lens[0] - q >= 0)
        assert torch.allclose(out.float(), seen[:, None, None].float().expand_as(out), rtol=2.0 ** -7, atol=0)
        assert bool((room[need:] == 0x5A).all())
