"""Attention over the block-scaled cache with sinks at the ends of binary32: e^sink joins the denominator, so
an infinite one leaves out 0 and lse the sink itself."""
import math

import pytest
import torch

from parity import DEV
from sparse_mla_attention_04_gb300 import binding
from test_gpu_kv8 import _problem, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,ql", [([300, 70], [1, 1]), ([300, 70], [40, 2]), ([300, 200], [150, 9]), ([40000], [1]),
                                     ([20000], [30]), ([0, 5], [3, 9])])
def test_infinite_and_largest_sinks(lens, ql):
    p = _problem(8, 2, 128, 64, lens, ql, seed=23)
    sinks = torch.tensor([math.inf, 3.0e38, 1e30, -3.0e38, -math.inf, 0.5, math.inf, 200.0])
    out, lse = (x.cpu().double() for x in _run(p, sinks=sinks))
    plain, z = (x.cpu().double() for x in _run(p, sinks=torch.full((8,), -math.inf)))
    big = [0, 1, 2, 6]
    assert bool((out[:, big] == 0).all())
    # in log2 units and back: three roundings of 2^-24
    want = sinks[big].double().expand_as(lse[:, big])
    assert bool(((lse[:, big] == want) | ((lse[:, big] - want).abs() <= want.abs() * 2.0 ** -22)).all())
    none = [3, 4]
    z[:, 3] = torch.where(torch.isinf(z[:, 3]), sinks[3].double(), z[:, 3])  # a row that sees nothing: the sink
    assert torch.equal(out[:, none], plain[:, none]) and torch.equal(lse[:, none], z[:, none])
    assert bool(torch.isfinite(out).all()) and not bool(torch.isnan(lse).any())


def test_rows_that_are_nan_stay_so():
    p = _problem(4, 2, 64, 32, [90], [3], seed=24)
    p["q"][1, 1, 5] = math.nan
    sinks = torch.full((4,), math.inf, device=DEV)
    out, lse = _run(p, sinks=sinks)
    nan = torch.isnan(out.float()).all(-1)
    assert bool(nan[1, 1]) and int(torch.isnan(out.float()).any(-1).sum()) == 1
    assert bool(torch.isnan(lse[1, 1])) and int(torch.isinf(lse).sum()) == 11
    assert binding.smla_device_error(reset=True) == 0
