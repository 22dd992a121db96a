"""How tree attention divides its work: several requests to a thread where the CTAs find their parts by themselves, planned
units that are cut, and contexts of tens of thousands of positions. Against plain binary64 (tolerances: test_gpu_tree.py)."""
import numpy as np
import pytest
import torch

from test_gpu_kv8 import _problem
from test_gpu_tree import _check, _run, _trees

pytestmark = pytest.mark.gpu


def _ragged(B, r, nodes, ctx, empty):
    """(lens, ql): requests without tokens strewn among the others, and a row of them at both ends and in the middle."""
    ql = r.randint(1, nodes + 1, B)
    ql[r.rand(B) < empty] = 0
    for at in (0, B // 2, B - 1):
        ql[max(0, at - 5):at + 5] = 0
    ql[B // 3] = nodes
    lens = ql + r.randint(0, ctx + 1, B)
    lens[::7] = ql[::7]                                           # no context
    return [int(x) for x in lens], [int(x) for x in ql]


@pytest.mark.parametrize("B", [257, 300, 700])
@pytest.mark.parametrize("G,D,nodes", [(4, 64, 5), (8, 128, 3), (1, 64, 20)])
@pytest.mark.parametrize("empty", [0.1, 0.95])
def test_more_requests_than_threads(B, G, D, nodes, empty):
    """One kv head, 17 to 128 rows to a request: parts are found without a plan, each thread adding up several requests."""
    r = np.random.RandomState(B + G)
    lens, ql = _ragged(B, r, nodes, 40, empty)
    lens[B // 3] += 700                                           # one that several CTAs share
    p = _problem(G, 1, D, 16, lens, ql, seed=B, pad=2)
    mask, _ = _trees(p, ql, B)
    _check(p, mask, _run(p, mask))


@pytest.mark.parametrize("H,hk,D,bound", [(16, 8, 64, 20), (8, 8, 128, 30), (16, 8, 64, 100)])
def test_planned_units_that_are_cut(H, hk, D, bound):
    """Many short requests, so that there is a plan, and one so long that equal parts cut it (one and two row tiles to a CTA)."""
    r = np.random.RandomState(bound)
    lens, ql = _ragged(130, r, 3, 60, 0.2)
    lens[77], ql[77] = 8000, 3
    p = _problem(H, hk, D, 64, lens, ql, seed=bound)
    mask, _ = _trees(p, ql, 7)
    _check(p, mask, _run(p, mask, max_query_len=bound))


@pytest.mark.parametrize("H,hk,D,ql", [(4, 1, 64, [3, 1]), (4, 2, 128, [2, 8]), (4, 1, 128, [17, 5]), (2, 2, 64, [30, 9]), (8, 1, 64, [20, 2])])
@pytest.mark.parametrize("window", [0, 21000])
def test_long_contexts(H, hk, D, ql, window):
    """33000 and 20000 positions, up to 8, 16, 128 and more rows to a request; a window that leaves out most of a third."""
    p = _problem(H, hk, D, 128, [33000 + ql[0], 20000 + ql[1]], ql, seed=H * D + ql[0])
    mask, pos = _trees(p, ql, 3)
    got = _run(p, mask, pos if window else None, window)
    _check(p, mask, got, pos if window else None, window)
    again = _run(p, mask, pos if window else None, window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("H,D,ql,kind", [(1, 64, [1000, 3], "tree"), (1, 128, [1024], "any"), (2, 64, [513, 64], "chain")])
def test_the_largest_trees(H, D, ql, kind):
    """Masks of up to sixteen words, trees that span many tiles of positions."""
    p = _problem(H, 1, D, 16, [n + 90 for n in ql], ql, seed=ql[0])
    mask, _ = _trees(p, ql, 5, kind=kind)
    _check(p, mask, _run(p, mask))
