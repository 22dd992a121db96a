"""smla_build_block_tables against an entry-by-entry reference (whole numbers: equal)."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


def _state(lens, ql, held, bs, width, spare, seed, head=None):
    r = np.random.RandomState(seed)
    lens, ql, held = (np.asarray(x, np.int64) for x in (lens, ql, held))
    used = int(held.sum())
    cap = used + spare
    perm = r.permutation(max(cap, 1)).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    k = 0
    for b in range(len(lens)):
        table[b, :held[b]] = perm[k:k + held[b]]
        k += held[b]
    ring = np.full(max(cap, 1), -9, np.int32)
    head = int(r.randint(max(cap, 1))) if head is None else head
    ring[(head + np.arange(spare)) % max(cap, 1)] = perm[used:used + spare]
    return lens, ql, held, table, ring, np.array([head, spare])


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _check(lens, ql, held, table, ring, state, bs, T, in_place=True, wide_rows=False):
    want = ref.block_tables(lens, ql, held, table, ring, state, bs, T)
    d_table = _up(table)
    if wide_rows:
        big = torch.full((table.shape[0], table.shape[1] + 5), 77, dtype=torch.int32, device=DEV)
        big[:, :table.shape[1]] = d_table
        d_table = big[:, :table.shape[1]]
    d_ring, d_held, d_state = _up(ring), _up(held), _up(state)
    kw = {} if in_place else dict(blocks_held_out=torch.empty_like(d_held), ring_state_out=torch.empty_like(d_state))
    got = binding.smla_build_block_tables(_up(lens), _up(ql), d_held, d_table, d_ring, d_state, block_size=bs,
                                          num_tokens=T, **kw)
    torch.cuda.synchronize()
    for name in ("counts", "query_start", "blocks_held", "ring_state", "positions", "token_request", "slot_mapping"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(d_table.cpu().numpy(), want["table"])
    assert np.array_equal(d_ring.cpu().numpy(), want["ring"])
    if in_place:
        assert got.blocks_held.data_ptr() == d_held.data_ptr() and got.ring_state.data_ptr() == d_state.data_ptr()
    else:
        assert np.array_equal(d_held.cpu().numpy(), held) and np.array_equal(d_state.cpu().numpy(), state)
    if wide_rows:
        assert int((big[:, table.shape[1]:] != 77).sum()) == 0
    return want


@pytest.mark.parametrize("B,bs,most,T_over,seed", [
    (1, 16, 1, 0, 0), (1, 64, 5000, 3, 1), (3, 16, 40, 5, 2), (64, 64, 1, 0, 3), (33, 32, 70, 1, 4),
    (1000, 16, 9, 64, 5), (1025, 128, 1, 7, 6), (2500, 16, 2, 100, 7), (40, 16, 900, 33, 8), (7, 128, 4096, 0, 9)])
@pytest.mark.parametrize("in_place", [True, False])
def test_random_steps(B, bs, most, T_over, seed, in_place):
    """Requests that grow, shrink, end and are empty; one launch and two (T above and below 4096)."""
    r = np.random.RandomState(seed)
    ql = r.randint(0, most + 1, B)
    old = r.randint(0, 6 * bs, B)
    lens = old + ql
    held = -(-old // bs) + (r.rand(B) < 0.2)          # some hold a block more than they need
    ended = r.rand(B) < 0.15
    lens = np.where(ended, 0, lens)
    ql = np.where(ended, r.randint(0, 3, B), ql)      # an ended request has no new tokens, whatever it says
    need = -(-lens // bs)
    width = int(max(need.max(), held.max())) + 1
    args = _state(lens, ql, held, bs, width, int(np.maximum(need - held, 0).sum()) + 5, seed)
    tokens = int(np.minimum(ql, lens).sum())
    want = _check(*args, bs, tokens + T_over, in_place, wide_rows=seed % 2 == 1)
    assert want["counts"][3] == 0


def test_fewer_map_entries_than_tokens():
    args = _state([100, 50], [100, 20], [0, 2], 16, 8, 40, 1)
    _check(*args, 16, 70)
    args = _state([100, 50], [100, 20], [0, 2], 16, 8, 40, 1)
    _check(*args, 16, 0)


@pytest.mark.parametrize("T", [300, 6000])
def test_lacking_blocks_change_nothing(T):
    # 19 blocks are asked for, 10 are free; then a row too narrow
    args = _state([300, 5], [300, 1], [0, 1], 16, 30, 10, 2)
    want = _check(*args, 16, T)
    assert want["counts"].tolist() == [301, 0, 0, 9]
    args = _state([300, 64], [300, 0], [0, 4], 16, 15, 100, 3)
    want = _check(*args, 16, T)
    assert want["counts"][3] == 4


def test_no_requests_and_negative_lengths():
    args = _state(np.zeros(0), np.zeros(0), np.zeros(0), 16, 4, 10, 4)
    _check(*args, 16, 9)
    args = _state([-5, 20, 17], [3, -2, 30], [2, 2, 0], 16, 4, 10, 5)
    _check(*args, 16, 40)


def test_full_ring_wraps():
    # every block free, the ring's head at its last entry
    args = _state([160, 33], [160, 33], [0, 0], 16, 12, 13, 6, head=12)
    want = _check(*args, 16, 193)
    assert want["ring_state"].tolist() == [12, 0]


def test_steps_in_a_captured_graph():
    """A captured step replays on the device's own lengths: 40 tokens for each request, then all end."""
    B, bs, width, cap = 5, 16, 8, 64
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(cap, dtype=torch.int32, device=DEV)
    state = torch.tensor([3, cap], dtype=torch.int32, device=DEV)

    def step():
        lens.add_(1)
        return binding.smla_build_block_tables(lens, one, held, table, ring, state, block_size=bs, num_tokens=8)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    seen = set()
    for n in range(2, 41):
        graph.replay()
        torch.cuda.synchronize()
        slots = got.slot_mapping.cpu().tolist()
        assert got.positions.cpu().tolist() == [n - 1] * B + [0] * 3
        assert slots[B:] == [-1] * 3 and len(set(slots[:B])) == B and not seen & set(slots[:B])
        seen |= set(slots[:B])
    assert held.cpu().tolist() == [3] * B and state.cpu().tolist() == [3 + 3 * B, cap - 3 * B]
    lens.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert held.cpu().tolist() == [0] * B and state.cpu().tolist() == [3 + 3 * B, cap]
    h = 3 + 3 * B
    assert sorted(ring.cpu().tolist()[(h + i) % cap] for i in range(cap)) == list(range(cap))
