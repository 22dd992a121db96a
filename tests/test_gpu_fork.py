"""smla_fork_block_tables against a plain implementation, an entry at a time, and smla_copy_blocks."""
import numpy as np
import pytest
import torch

import branch_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _state(B_old, width, bs, r, share=0.5, spare=20):
    """Old rows that share some of their first blocks, and the ring of the rest."""
    held = r.randint(0, width + 1, B_old)
    held[0] = width
    table = np.full((B_old, width), -1, np.int64)
    used = 0
    for b in range(B_old):
        common = 0
        if b and r.rand() < share:
            a = r.randint(0, b)
            common = r.randint(0, min(held[a], held[b]) + 1)
            table[b, :common] = table[a, :common]
        n = held[b] - common
        table[b, common:held[b]] = used + np.arange(n)
        used += n
    nb = used + spare
    perm = r.permutation(nb)
    table = np.where(table >= 0, perm[table.clip(min=0)], -1).astype(np.int32)
    cap = nb + int(r.randint(0, 5))
    ring = np.full(cap, -9, np.int32)
    head = int(r.randint(cap))
    ring[(head + np.arange(spare)) % cap] = perm[used:]
    return held.astype(np.int32), table, ring, np.array([head, spare], np.int32), nb


def _both(source, keep, held, table, ring, state, bs, nb, **kw):
    B, width = len(source), table.shape[1]
    before = np.full((B, width), -5, np.int32)
    want = ref.fork(source, keep, held, table, ring, state, bs, nb, before)
    ring_d, table_d, held_d = _up(ring), _up(table), _up(held)
    out = kw.pop("out", None)
    out = _up(before) if out is None else out
    held_out = torch.full((B,), -3, dtype=torch.int32, device=DEV)
    got = binding.smla_fork_block_tables(_up(source), _up(keep), held_d, table_d, ring_d, _up(state), block_size=bs, num_blocks=nb,
                                         block_table_out=out, blocks_held_out=held_out, **kw)
    torch.cuda.synchronize()
    for n in ("copy_from", "copy_to", "counts", "block_table", "ring_state"):
        assert np.array_equal(getattr(got, n).cpu().numpy(), want[n]), n
    assert np.array_equal(ring_d.cpu().numpy(), want["ring"])
    assert np.array_equal(held_out.cpu().numpy(), np.full(B, -3) if want["blocks_held"] is None else want["blocks_held"])
    assert np.array_equal(table_d.cpu().numpy(), table) and np.array_equal(held_d.cpu().numpy(), held)
    return got, want


@pytest.mark.parametrize("B_old,B,width,bs", [
    (1, 1, 1, 16), (1, 4, 8, 64), (4, 4, 5, 16), (3, 0, 4, 32), (0, 3, 4, 32), (7, 20, 33, 128), (256, 256, 60, 64),
    (64, 200, 300, 16), (1500, 1100, 9, 16), (1000, 1200, 3, 16), (2, 1400, 1000, 64), (5, 5, 2600, 32), (33, 40, 0, 16)])
@pytest.mark.parametrize("seed", [0, 1])
def test_forks(B_old, B, width, bs, seed):
    r = np.random.RandomState(seed + B + width)
    if B_old and width:
        held, table, ring, state, nb = _state(B_old, width, bs, r, spare=B + 5)
    else:
        held, table, nb = np.zeros(B_old, np.int32), np.zeros((B_old, width), np.int32), 9
        ring, state = np.arange(9, dtype=np.int32), np.array([4, 9], np.int32)
    source = r.randint(-1, B_old + (r.rand() < 0.3), B)
    keep = np.array([0 if s < 0 or s >= B_old else r.choice([int(held[s]) * bs, r.randint(0, int(held[s]) * bs + 2), -4, 1 << 30]) for s in source], np.int64)
    if B and B_old and seed:                                        # every row goes on as it was
        source, keep = np.arange(B) % B_old, np.minimum(held[np.arange(B) % B_old].astype(np.int64) * bs, 1 << 30)
    got, want = _both(source, keep, held, table, ring, state, bs, nb)
    # nobody shares a block that is to be written to, and every block is held or free
    if B and B_old and width and int(want["counts"][3]) == 0:
        live = got.block_table.cpu().numpy()
        n = got.blocks_held.cpu().numpy()
        tails = [live[b, n[b] - 1] for b in range(B) if n[b] and 0 < min(keep[b], int(held[source[b]]) * bs) % bs]
        rows = np.concatenate([live[b, :n[b]] for b in range(B)] + [[]])
        for t in tails:
            assert (rows == t).sum() == 1
        head, count = got.ring_state.tolist()
        free = want["ring"][(head + np.arange(count)) % len(ring)]
        assert len(set(free) & set(rows)) == 0 and len(set(free)) == len(free)


def test_who_keeps_a_shared_last_block():
    """A row that has it full before rows that end in it, then the first of those; others copy."""
    bs, nb = 16, 10
    table, held = np.array([[3, 5, 7], [3, 5, 2]], np.int32), np.array([3, 3], np.int32)
    ring, state = np.array([0, 1, 4, 6, 8, 9, -1, -1, -1, -1], np.int32), np.array([0, 6], np.int32)
    for source, keep, frm in (([0, 0], [40, 40], [-1, 7]), ([0, 0], [48, 40], [-1, 7]), ([0, 0], [40, 48], [7, -1]),
                              ([0, 1], [20, 32], [5, -1]), ([0, 1], [20, 20], [-1, 5]), ([1, 0], [1, 1], [-1, 3]), ([0, 1], [32, 32], [-1, -1]),
                              ([0, 0, 0], [0, 48, 47], [-1, -1, 7])):
        got, _ = _both(np.array(source), np.array(keep), held, table, ring, state, bs, nb)
        assert got.copy_from.tolist() == frm, (source, keep)


def test_blocks_lacking_and_bad_entries():
    bs, nb = 16, 12
    table, held = np.array([[3, 5, 7, 99], [-4, 11, 2, 1]], np.int32), np.array([4, 9], np.int32)     # more held than the row has
    ring, state = np.full(12, -1, np.int32), np.array([11, 2], np.int32)
    ring[11], ring[0] = 8, 9
    _both(np.array([0, 0, 0, 0]), np.array([40, 40, 40, 40]), held, table, ring, state, bs, nb)      # three copies, two blocks
    got, _ = _both(np.array([0, 0, 0]), np.array([40, 40, 40]), held, table, ring, state, bs, nb)    # just enough
    assert got.counts.tolist() == [120, 2, 3, 0]
    got, _ = _both(np.array([0, 0, 1, 1]), np.array([64, 60, 16, 9]), held, table, ring, state, bs, nb)   # last blocks outside the pool
    assert got.counts.tolist()[1] == 0
    _both(np.array([1, -1, 2, -7]), np.array([64, 5, 5, 5]), held, table, ring, np.array([-1, 99], np.int32), bs, nb)


@pytest.mark.parametrize("W", [12, 1500])
def test_strided_tables_streams_and_replay(W):
    bs, r = 32, np.random.RandomState(3)
    held, table, ring, state, nb = _state(6, W, bs, r)
    buffers = torch.full((2, 6, W + 8), -5, dtype=torch.int32, device=DEV)       # two tables that take turns
    buffers[0, :, :W] = _up(table)
    source, keep = np.array([0, 0, 2, 3, 3, 5]), held[[0, 0, 2, 3, 3, 5]].astype(np.int64) * bs - 7
    want = ref.fork(source, keep, held, table, ring, state, bs, nb, np.full((6, W), -5, np.int32))
    src, kp, hd, rg, st = _up(source), _up(keep), _up(held), _up(ring), _up(state)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb,
                                             block_table_out=buffers[1, :, :W])
    src.copy_(_up([5, 5, 5, -1, 0, 1]))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.fork([5, 5, 5, -1, 0, 1], keep, held, table, ring, state, bs, nb, np.full((6, W), -5, np.int32))
    assert np.array_equal(buffers[1, :, :W].cpu().numpy(), want["block_table"])
    assert bool((buffers[1, :, W:] == -5).all())
    assert np.array_equal(got.ring_state.cpu().numpy(), want["ring_state"]) and got.ring_state.data_ptr() == st.data_ptr()
    with pytest.raises(binding.SmlaError):
        binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb,
                                       block_table_out=buffers[0, :, 4:W + 4])
    with pytest.raises(ValueError):
        binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb,
                                       block_table_out=buffers[1])
    with pytest.raises(binding.SmlaError):
        binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb,
                                       block_table_out=buffers[1, :, :W], workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(binding.SmlaError):
        binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=24, num_blocks=nb)
    with pytest.raises(ValueError):
        binding.smla_fork_block_tables(src, kp[:3], hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb)
    side = torch.cuda.Stream()
    rg, st = _up(ring), _up(state)
    torch.cuda.synchronize()
    got = binding.smla_fork_block_tables(src, kp, hd, buffers[0, :, :W], rg, st, block_size=bs, num_blocks=nb, stream=side)
    side.synchronize()
    fresh = np.where(want["block_table"] == -5, -1, want["block_table"])
    assert np.array_equal(got.block_table.cpu().numpy(), fresh)


@pytest.mark.parametrize("table_out", [False, True])
@pytest.mark.parametrize("held_out", [False, True])
def test_fresh_outputs_where_blocks_lack(table_out, held_out):
    """Two rows from one whose last block is partly full, and an empty ring: nothing is written, and what is fresh says so."""
    table, held = _up([[4, 2, -1]]), _up([2])
    ring, state = _up([0] * 6), _up([3, 0])
    given = {}
    if table_out:
        given["block_table_out"] = _up(np.full((2, 3), -7))
    if held_out:
        given["blocks_held_out"] = _up([-7, -7])
    torch.empty(4096, dtype=torch.uint8, device=DEV).fill_(0x5A)      # (the allocator hands it out again)
    got = binding.smla_fork_block_tables(_up([0, 0]), _up([20, 20]), held, table, ring, state, block_size=16, num_blocks=6, **given)
    assert got.counts.tolist()[1:] == [0, 0, 1]
    assert got.block_table.tolist() == [[-7 if table_out else -1] * 3] * 2
    assert got.blocks_held.tolist() == [-7 if held_out else -1] * 2
    assert got.copy_from.tolist() == got.copy_to.tolist() == [-1, -1] and state.tolist() == [3, 0]
    ring.fill_(5)
    state[1] = 1
    got = binding.smla_fork_block_tables(_up([0, 0]), _up([20, 20]), held, table, ring, state, block_size=16, num_blocks=6, **given)
    rest = -7 if table_out else -1
    assert got.block_table.tolist() == [[4, 2, rest], [4, 5, rest]] and got.blocks_held.tolist() == [2, 2]
    assert got.copy_from.tolist() == [-1, 2] and got.copy_to.tolist() == [-1, 5]


# ------------------------------------------------------------------ copies
def test_copies():
    r = np.random.RandomState(1)
    shapes = [((50, 4, 16, 64), torch.uint8), ((50, 4), torch.float32), ((50, 1000), torch.bfloat16), ((50, 3), torch.uint8),
              ((50, 70001), torch.uint8), ((50, 33000), torch.float32), ((50, 0), torch.float32), ((50,), torch.int64)]
    pools = [torch.from_numpy(r.randint(0, 100, s)).to(t) for s, t in shapes]
    odd = torch.zeros(50 * 64 + 1, dtype=torch.uint8)[1:].view(50, 64)
    odd.copy_(torch.from_numpy(r.randint(0, 100, (50, 64))))
    frm = np.array([3, 3, -1, 7, 60, 12, 9, 10], np.int32)
    to = np.array([20, 21, 22, -1, 23, 50, 9, 40], np.int32)         # the same, none, past the pool, onto itself
    got = [p.to(DEV) for p in pools]
    room = torch.zeros(50 * 64 + 1, dtype=torch.uint8, device=DEV)
    got.append(room[1:].view(50, 64))
    got[-1].copy_(odd)
    binding.smla_copy_blocks(got, _up(frm), _up(to))
    torch.cuda.synchronize()
    for have, want in zip(got, pools + [odd]):
        want = want.clone()
        for a, b in ((3, 20), (3, 21), (10, 40)):
            want[b] = want[a]
        assert torch.equal(have.cpu(), want)


def test_copies_in_many_pools_past_32_bits_and_in_a_graph():
    pools = [torch.full((8, 4), float(i), device=DEV) + torch.arange(8, device=DEV)[:, None] for i in range(300)]   # three launches
    big = torch.zeros((8, (1 << 30) + 16), dtype=torch.uint8, device=DEV)
    big[5] = 7
    handle = binding.BlockPools(pools + [big])
    frm, to = _up([1, 5]), _up([0, 6])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.smla_copy_blocks(handle, frm, to)
    frm.copy_(_up([2, 5]))
    graph.replay()
    torch.cuda.synchronize()
    for i, p in enumerate(pools):
        assert p[:, 0].tolist() == [i + x for x in (2, 1, 2, 3, 4, 5, 5, 7)]
    assert bool((big[6] == 7).all()) and not bool(big[4].any()) and not bool(big[7].any())
    binding.smla_copy_blocks(handle, frm[:0], to[:0])
    with pytest.raises(ValueError):
        binding.BlockPools([pools[0], torch.zeros((9, 4), device=DEV)])
    with pytest.raises(ValueError):
        binding.BlockPools([pools[0][:, :2]])
    with pytest.raises(ValueError):
        binding.smla_copy_blocks(handle, frm, to[:1])
