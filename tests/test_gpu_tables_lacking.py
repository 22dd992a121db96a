"""smla_build_block_tables says how many blocks lack, however many (whole numbers: equal), by one launch and by two."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [300, 6000])
@pytest.mark.parametrize("long", [1, 3, 40, 1100])
@pytest.mark.parametrize("width,free", [(4, 10), (0, 0), (7, 500)])
def test_lengths_far_beyond_the_table(T, long, width, free):
    """`long` requests of 2^31 - 1 positions among short ones: nothing changes, the sum is cut to 2^31 - 1 only."""
    bs, top = 16, 2 ** 31 - 1
    lens = np.array([5, 30] + [top] * long + [0], np.int64)
    ql = np.array([1, 30] + [2] * long + [0], np.int64)
    held = np.array([1, 0] + [0] * long + [2], np.int64).clip(0, width)
    table = np.full((len(lens), width), 3, np.int32)
    ring = np.arange(max(free, 1) + 8, dtype=np.int32)
    state = np.array([2, free])
    want = ref.block_tables(lens, ql, held, table, ring, state, bs, T)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)  # noqa: E731
    d_table, d_ring = up(table), up(ring)
    got = binding.smla_build_block_tables(up(lens), up(ql), up(held), d_table, d_ring, up(state), block_size=bs, num_tokens=T)
    counts = got.counts.cpu().numpy().astype(np.int64)
    assert want["counts"][3] > 2 ** 27 - 8
    assert counts.tolist() == np.minimum(want["counts"], top).tolist()
    for name in ("query_start", "blocks_held", "ring_state", "positions", "token_request", "slot_mapping"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_ring.cpu().numpy(), ring)
