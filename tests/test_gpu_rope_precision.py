"""smla_rope_cos_sin_cache value by value, small sines too.

Tolerance, derived. The angle's distance to the nearest quarter turn is exact to
2^-65 of a turn a position (the frequency's last place) and becomes binary32
with a rounding of the integer, of 2 pi 2^-64 and of their product (3 times 2^-24
relative). The sine's series adds a rounding of the result, a tenth of those of
its terms and 2^-28 for what it leaves out; the cosine's the same, and 0.9 of the
angle's: below 6 times 2^-24 of the value with the factor's product. The
frequency in binary64 (powers, a quotient; their exponents' rounding counts up
to 14 times) is off by less than 2^-48 of itself, here as there: an angle of
p f by p f 2^-47."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,base,scaling,factor,orig", [
    (64, 1e4, "none", 1.0, 0), (64, 1e6, "none", 1.0, 0), (128, 5e5, "linear", 40.0, 0), (128, 1e6, "ntk", 8.0, 0),
    (64, 1e6, "yarn", 40.0, 4096), (2, 1e4, "none", 1.0, 0), (6, 1e8, "none", 1.0, 0), (256, 1e9, "linear", 3.0, 0)])
@pytest.mark.parametrize("first,n", [(0, 3000), (1, 1), (100000, 700), (1048000, 100)])
def test_each_value(rot, base, scaling, factor, orig, first, n):
    got = binding.smla_rope_cos_sin_cache(n, rot, base=base, scaling=scaling, factor=factor, original_max_position=orig,
                                          first_position=first).cpu().numpy().astype(np.float64)
    f, m = ref.frequencies(rot, base, scaling, factor, orig, 32.0, 1.0)
    p = np.arange(first, first + n, dtype=np.float64)[:, None]
    ang = p * f
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1) * m
    off = m * (np.tile(ang, 2) * 2.0 ** -47 + p * 2.0 ** -62)
    assert (np.abs(got - want) <= np.abs(want) * 6 * 2.0 ** -24 + off).all()


def test_angles_just_below_a_turn_keep_their_sign_and_size():
    """The positions of a long table that come nearest to whole, half and quarter turns, from either side."""
    rot, n = 64, 400000
    t = binding.smla_rope_cos_sin_cache(n, rot).cpu().numpy().astype(np.float64)
    f, _ = ref.frequencies(rot, 1e4, "none", 1.0, 0, 32.0, 1.0)
    ang = np.arange(n, dtype=np.float64) * f[0]
    quarter = np.rint(ang / (np.pi / 2))
    near = ang - quarter * (np.pi / 2)                         # 53 bits of pi: off by quarter 2^-53, in all below 2^-34
    at = np.argsort(np.abs(near))[1:40]                        # (without position 0)
    small = np.where(quarter[at] % 2 == 0, t[at, rot // 2], t[at, 0])
    sign = np.where(np.isin(quarter[at] % 4, (0, 3)), 1.0, -1.0)
    assert (np.abs(small - sign * near[at]) <= np.abs(near[at]) * 6 * 2.0 ** -24 + 2.0 ** -33).all()
    assert np.abs(near[at]).max() < 2.0 ** -10


def test_misaligned_tables_have_the_same_bits():
    """Rows whose pairs go four to a store, and one."""
    flat = torch.empty(50 * 64 + 1, device="cuda")
    odd = binding.smla_rope_cos_sin_cache(50, 64, out=flat[1:].view(50, 64))
    assert torch.equal(odd, binding.smla_rope_cos_sin_cache(50, 64))
