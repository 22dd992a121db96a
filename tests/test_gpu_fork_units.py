"""smla_fork_block_tables at the border between its two forms: rows of several units in one block, and narrow rows, a unit each."""
import numpy as np
import pytest

from test_gpu_fork import _both, _state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B_old,B,width,bs", [
    (1, 4, 600, 16), (3, 5, 700, 64), (1, 1, 4096, 16), (1, 1, 4097, 16), (16, 16, 256, 32), (16, 16, 257, 32), (31, 1, 2, 16),
    (64, 64, 2, 64), (256, 256, 2, 16), (1000, 1000, 2, 64), (4000, 4000, 1, 16), (1, 31, 8, 128), (1, 32, 8, 128)])
@pytest.mark.parametrize("seed", [0, 1])
def test_units(B_old, B, width, bs, seed):
    r = np.random.RandomState(seed + B + width)
    held, table, ring, state, nb = _state(B_old, width, bs, r, spare=B + 5)
    source = r.randint(-1, B_old, B) if not seed else np.arange(B) % B_old
    keep = np.array([0 if s < 0 else r.choice([int(held[s]) * bs, r.randint(0, int(held[s]) * bs + 2)]) for s in source], np.int64)
    _both(source, keep, held, table, ring, state, bs, nb)
