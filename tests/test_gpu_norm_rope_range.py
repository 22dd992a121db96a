"""smla_qk_norm_rope of rows whose squares pass binary32: the widest ones, and ones with elements far below the largest.

Tolerance: as in test_gpu_norm_rope.py, with the row's width: the sum of squares adds D / 32 + 16 terms one after another and
five levels, half of its rounding counts, with nine more: (D / 64 + 20) 2^-24 of a value. The root of such a row may be below
the normals, down to 2^-128, where a step is 2^-149 and a rounding 2^-22 = 4 * 2^-24 of it. 2 * 2^-24 of a pair's size for the
rotation, half a step of the type, and 2^-146 below the normals."""
import pytest
import torch

import branch_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding
from test_gpu_norm_rope import TYPES, _table

pytestmark = pytest.mark.gpu


def _close(got, x, pos, cs, off, neox):
    want, size = ref.norm_rope(x.cpu(), None, 0.0, 1e-6, pos.cpu(), cs.cpu(), off, neox)
    least = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 0.0}[x.dtype] + 2.0 ** -146
    tol = size * (x.shape[-1] / 64 + 26) * 2.0 ** -24 + want.abs() * torch.finfo(x.dtype).eps / 2 + least
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [512, 4096, 4100, 8192, 65536])
def test_the_widest_rows_of_the_largest_values(dtype, D):
    g = torch.Generator().manual_seed(D)
    x = torch.rand((3, 2, D), generator=g) * 1e38 + 2.3e38
    x[1] = 3.3e38
    x[2, :, ::3] = -1e-3                                           # and some beside them that count for nothing
    x = x.to(TYPES[dtype]).to(DEV)
    pos, cs = torch.tensor([3, 0, 7], device=DEV), _table(8, 64, g).to(DEV)
    got = binding.smla_qk_norm_rope(x, None, None, None, pos, cs, rot_offset=8)[0]
    _close(got, x, pos, cs, 8, True)


@pytest.mark.parametrize("D", [128, 70, 4100])
@pytest.mark.parametrize("neox", [True, False])
def test_small_elements_of_large_rows_keep_their_bits(D, neox):
    """Beside 2^64.5, whose square is the sum, every size down to 2^-66: results down to 2^-127, all 24 bits of each."""
    g = torch.Generator().manual_seed(D)
    x = (1 + torch.rand((4, 3, D), generator=g)) * torch.exp2(torch.randint(-66, 30, (4, 3, D), generator=g).float())
    x[..., D // 2] = 2.0 ** 64.5
    x = x.to(DEV)
    pos, cs = torch.tensor([3, 0, 7, 1], device=DEV), _table(8, 32, g).to(DEV)
    got = binding.smla_qk_norm_rope(x, None, None, None, pos, cs, is_neox=neox)[0]
    _close(got, x, pos, cs, 0, neox)
