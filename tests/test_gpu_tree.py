"""Masks of drafted trees, and attention of such trees over the block-scaled cache against a plain binary64
implementation (tolerances: see test_gpu_kv8.py, the arithmetic is the same)."""
import math

import numpy as np
import pytest
import torch

import branch_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding
from test_gpu_kv8 import _problem

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the masks
def _masks(parents, lens, start, **kw):
    up = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)  # noqa: E731
    m = binding.smla_build_tree_masks(up(parents), up(lens), up(start), **kw)
    torch.cuda.synchronize()
    return m


@pytest.mark.parametrize("sizes", [[1], [8], [64, 1, 65, 0, 3], [128], [1000, 5], [1024], [3] * 700])
@pytest.mark.parametrize("window", [0, 1, 5])
def test_masks(sizes, window):
    r = np.random.RandomState(len(sizes) + window)
    parents = np.concatenate([ref.random_tree(n, r, chain=i % 3 == 2 or n == 1000) for i, n in enumerate(sizes)] + [[9, 9, 9]])
    lens = [n + int(r.randint(0, 100)) for n in sizes]
    start = np.concatenate([[0], np.cumsum(sizes)])
    most = max(sizes)
    words = (most + 63) // 64
    got = _masks(parents, lens, start, max_query_len=most, window=window)
    mask, pos = ref.tree_masks(parents, lens, start, words, window)     # (three rows behind the last request: zeros)
    assert torch.equal(got.tree_mask.cpu(), ref.words_of(mask))
    assert torch.equal(got.positions.cpu(), torch.from_numpy(pos))
    assert binding.smla_device_error() == 0


def test_masks_of_bad_trees():
    """Parents that do not come before their children are none; nodes past the words see nothing; each is reported."""
    binding.smla_device_error(reset=True)
    start = [0, 4, 4, 6]
    for parents in ([-1, 1, 0, 0, -1, 0], [-1, 0, 7, 1, -1, 0], [-2, 0, 1, 1, -1, 5]):
        got = _masks(parents, [10, 0, 2], start, max_query_len=6)
        mask, pos = ref.tree_masks(parents, [10, 0, 2], start, 1, 0)
        assert torch.equal(got.tree_mask.cpu(), ref.words_of(mask)) and torch.equal(got.positions.cpu(), torch.from_numpy(pos))
        assert binding.smla_device_error(reset=True) == 16
    parents = ref.random_tree(100, np.random.RandomState(0), chain=True)
    got = _masks(parents, [50], [0, 100], max_query_len=64)       # and a context that is shorter than the tree
    mask, pos = ref.tree_masks(parents, [50], [0, 100], 1, 0)
    assert torch.equal(got.tree_mask.cpu(), ref.words_of(mask)) and torch.equal(got.positions.cpu(), torch.from_numpy(pos))
    assert binding.smla_device_error(reset=True) == 16
    with pytest.raises(binding.SmlaError):
        _masks(parents, [100], [0, 100], max_query_len=1025)
    got = _masks([5, 5], [], [0], max_query_len=3)                # no request: rows behind the last
    assert not bool(got.tree_mask.any()) and not bool(got.positions.any())
    empty = _masks([], [3], [0, 0], max_query_len=0)
    assert empty.tree_mask.shape == (0, 1)


# ------------------------------------------------------------------ the attention
def _trees(p, ql, seed, words=None, kind="tree"):
    """(truth values [T, 64 words], positions) for the requests' new tokens."""
    r = np.random.RandomState(seed)
    T = p["q"].shape[0]
    start = np.concatenate([[0], np.cumsum(ql)])
    words = words or max(1, -(-max(ql) // 64))
    parents = np.concatenate([ref.random_tree(n, r, chain=kind == "chain") for n in ql] + [np.zeros(0, np.int32)])
    lens = np.minimum(p["lens"].numpy(), p["table"].shape[1] * p["kc"].shape[2])
    mask, pos = ref.tree_masks(parents, lens, start, words, 0)
    if kind == "any":                                             # any mask at all: forward, backward, empty
        mask = r.rand(*mask.shape) < 0.4
        mask[r.rand(len(mask)) < 0.2] = False
    mask = np.concatenate([mask, np.ones((T - len(mask), mask.shape[1]), bool)])
    return mask, np.concatenate([pos, np.zeros(T - len(pos), np.int64)])


def _run(p, mask, pos=None, window=0, sinks=None, **kw):
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    bits = ref.words_of(mask).to(DEV)
    return binding.smla_kv8_tree_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"], bits,
                                          p["scale"], max_query_len=kw.pop("max_query_len", p["max_q"]), window=window,
                                          positions=None if pos is None else torch.from_numpy(pos).to(DEV),
                                          sinks=None if sinks is None else sinks.to(DEV), **kw)


def _check(p, mask, got, pos=None, window=0, sinks=None):
    out, lse = got
    torch.cuda.synchronize()
    assert binding.smla_device_error(reset=True) == 0
    want, z, w, reach = ref.tree_attention(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], p["start"], mask,
                                           p["scale"], window, pos, sinks)
    T = int(p["start"][-1])
    out, lse, want, z, w, reach = (x[:T].cpu().double() for x in (out, lse, want, z, w, reach))
    n, top = int(p["lens"].max()), float(p["vs"].max()) * 448
    tol = want.abs() * 2.0 ** -8 + w * (2.0 ** -11 + 2.0 ** -17 * (1 + reach[..., None])) + n * top * 2.0 ** -24
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / tol.clamp(min=1e-30)).max())
    none = torch.isinf(z)
    assert torch.equal(none, torch.isinf(lse))
    assert bool(((lse - z).abs()[~none] <= 2.0 ** -18 * (1 + reach[~none])).all())


@pytest.mark.parametrize("H,hk,D,bs,lens,ql", [
    (4, 4, 128, 64, [1], [1]),                                     # one token, no context
    (8, 2, 128, 64, [70, 5, 64], [1, 5, 2]),                       # streaming kernel, 8 rows
    (8, 1, 64, 16, [33, 150, 2], [2, 1, 2]),                       # 16 rows
    (4, 2, 128, 16, [100, 17, 300], [8, 3, 5]),
    (16, 2, 128, 64, [200, 41, 77], [40, 9, 13]),                  # one row tile to a CTA, several items
    (8, 8, 64, 32, [129, 128, 127], [100, 128, 1]),
    (12, 4, 64, 128, [500, 90, 260], [70, 90, 33]),                # two row tiles
    (16, 1, 128, 64, [310], [130]),                                # masks of three words
    (5, 1, 64, 16, [37, 0, 600], [37, 0, 20]),                     # no context; no tokens
    (2, 2, 64, 16, [3, 40], [8, 3]), (4, 1, 128, 64, [5, 40], [20, 3])])   # more new tokens than there are positions
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_attention(H, hk, D, bs, lens, ql, kind):
    p = _problem(H, hk, D, bs, lens, ql, seed=H * D + len(lens), pad=3)
    mask, pos = _trees(p, ql, 1, kind=kind)
    _check(p, mask, _run(p, mask))
    # a bound of the trees' sizes that is too high, and masks that are wider than they need be: the other kernel, the same values
    wide = np.concatenate([mask, np.ones((len(mask), 64), bool)], 1)
    _check(p, mask, _run(p, wide, max_query_len=200))


@pytest.mark.parametrize("H,hk,D,bs,lens,ql", [(8, 2, 128, 64, [300, 70], [2, 2]), (16, 2, 64, 16, [200, 300, 41], [30, 17, 41])])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 100000])
def test_window(H, hk, D, bs, lens, ql, window):
    """A token sees the context's positions above its own minus the window; nothing of the pages below is used."""
    p = _problem(H, hk, D, bs, lens, ql, seed=window)
    mask, pos = _trees(p, ql, 2)
    pos[0], pos[1] = -5, 10 ** 12                                  # positions that no new token has: the nearest
    if window < 30:                                                # blocks that nobody sees went to somebody else
        for b, n in enumerate(lens):
            for j in range(max(0, n - ql[b] - window) // bs):
                blk = int(p["table"][b, j])
                p["ks"][blk], p["vs"][blk] = math.nan, math.inf
    _check(p, mask, _run(p, mask, pos, window), pos, window)


def test_a_chain_is_causal():
    """Trees without branches: the same bits as the causal form wherever both take the same steps."""
    p = _problem(16, 4, 128, 64, [300, 130, 64], [20, 3, 40], seed=4)
    mask, _ = _trees(p, [20, 3, 40], 1, kind="chain")
    out, lse = _run(p, mask)
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    want, z = binding.smla_kv8_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"], p["scale"], max_query_len=40)
    err = (out.float() - want.float()).abs()
    assert float(err.max()) <= 2.0 ** -6 * float(want.float().abs().max())
    assert float((lse - z).abs().max()) <= 2.0 ** -16
    _check(p, mask, (out, lse))


@pytest.mark.parametrize("ql", [[2, 1], [40, 7]])
def test_sinks_empty_rows_and_rows_behind(ql):
    p = _problem(4, 1, 64, 16, [ql[0], 50], ql, seed=6, pad=2)
    mask, pos = _trees(p, ql, 3, kind="any")
    mask[0] = False                                                # a row without context that sees nothing
    sinks = torch.tensor([0.5, -2.0, 3.0, -math.inf])
    T = sum(ql)
    out = torch.full((T + 2, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 2, 4), 5.0, device=DEV)
    _check(p, mask, _run(p, mask, sinks=sinks, out=out, lse=lse), sinks=sinks)
    assert float(out[0].abs().max()) == 0 and torch.equal(lse[0].cpu(), sinks)
    assert bool((out[T:] == 5.0).all()) and bool((lse[T:] == 5.0).all())
    got = _run(p, mask, out=out, lse=lse)
    _check(p, mask, got)
    assert bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("ql", [[3], [60]])
def test_nan_codes_reach_only_those_who_see_them(ql):
    p = _problem(4, 1, 128, 16, [100 + ql[0]], ql, seed=8)
    mask, _ = _trees(p, ql, 4, kind="any")
    mask[0, 2], mask[1, 2] = True, False
    at = 100 + 2
    blk = int(p["table"][0, at // 16])
    clean, _ = _run(p, mask)
    p["vc"][blk, 0, at % 16, 7] = 0x7F
    out, _ = _run(p, mask)
    sees = torch.from_numpy(mask[:ql[0], 2].copy()).to(DEV)
    assert bool(out[sees][..., 7].isnan().all())
    out[sees, :, 7] = clean[sees, :, 7]
    assert torch.equal(out, clean)
    mask[:, 2] = False                                             # one that nobody sees reaches nobody
    out, lse = _run(p, mask)
    assert not bool(out.isnan().any()) and not bool(lse.isnan().any())


def test_split_over_many_blocks_streams_and_replay():
    """Long contexts cut over the GPU, on a stream of the caller's; a captured call follows masks and lengths."""
    ql = [16, 7, 1]
    p = _problem(8, 2, 128, 64, [5000, 2100, 900], ql, seed=9)
    mask, pos = _trees(p, ql, 5)
    want = _run(p, mask)
    _check(p, mask, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _run(p, mask, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d = {n: x.to(DEV) for n, x in p.items() if isinstance(x, torch.Tensor)}
    bits = ref.words_of(mask).to(DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = binding.smla_kv8_tree_attn_fwd(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lens"], d["start"],
                                             bits, p["scale"], max_query_len=16)
    mask2, _ = _trees(p, ql, 6, kind="any")
    bits.copy_(ref.words_of(mask2))
    p["lens"] = torch.tensor([3000, 2100, 64], dtype=torch.int32)
    d["lens"].copy_(p["lens"])
    graph.replay()
    _check(p, mask2, got)


@pytest.mark.parametrize("bound", [20, 100])
def test_many_requests(bound):
    """So many units that they are planned and taken whole, by one and by two row tiles to a CTA."""
    r = np.random.RandomState(bound)
    ql = [int(x) for x in r.randint(0, 4, 130)]
    lens = [n + int(x) for n, x in zip(ql, r.randint(0, 60, 130))]
    p = _problem(16, 8, 64, 16, lens, ql, seed=bound)
    mask, pos = _trees(p, ql, 7)
    _check(p, mask, _run(p, mask, max_query_len=bound))


@pytest.mark.parametrize("H,hk,D", [(8, 2, 128), (4, 1, 64)])
def test_requests_without_tokens_among_cut_units(H, hk, D):
    """Units that several CTAs share, with requests between them that have no tokens, or no context."""
    ql = [0, 20, 0, 0, 7, 33, 0, 1, 40, 0]
    lens = [50, 3000, 0, 700, 1500, 33, 9, 2000, 900, 5]
    p = _problem(H, hk, D, 64, lens, ql, seed=D)
    mask, pos = _trees(p, ql, 8)
    _check(p, mask, _run(p, mask))


def test_two_calls_at_once():
    """Calls on two streams, each with outputs and a workspace of its own: the bits of one call at a time."""
    problems = [_problem(8, 2, 128, 64, [3000, 500], ql, seed=len(ql) + ql[0]) for ql in ([20, 9], [2, 1])]
    masks = [_trees(p, [int(x) for x in p["start"].diff()], 3)[0] for p in problems]
    want = [_run(p, m) for p, m in zip(problems, masks)]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    got = [[_run(p, m, stream=s) for p, m, s in zip(problems, masks, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_refusals():
    p = _problem(4, 1, 64, 16, [20], [4], seed=1)
    mask, pos = _trees(p, [4], 1)
    with pytest.raises(ValueError):
        _run(p, mask, window=5)
    with pytest.raises(ValueError):
        _run(p, mask[:3])
    with pytest.raises(ValueError):
        _run(p, mask, pos[:2], window=5)
