"""The operators of steps that draft and branch together, as an engine's steps use them.

Drafting: block tables -> tree masks -> norms with rotation -> cache write -> tree attention -> kept tokens -> block tables
that take the rest back; the next step goes on from what was kept. Branching: one prompt's row becomes several, their last
blocks are copied, each grows by its own tokens, rows are reordered, ended and cut back.

Attention is checked against binary64 attention over the values that the cache stands for (tolerances: see
test_gpu_kv8.py). What the cache stands for is checked against the rotated keys and the values that were written: a code is
off by half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below the normals) for its own write and for each time that
its block's scale grows, which takes a new largest value: with at most fifteen of those in a block's history (of n random values
the k-th is a new largest one with 1 / k, so ln n or four in a block of 64) sixteen half steps of the last, widest scale."""
import math

import numpy as np
import pytest
import torch

import branch_reference as bref
import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding as b
from test_gpu_serving_step import Engine

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _held_right(e, caches, limit):
    """Every request's rows are in the caches, at its length."""
    table = e.table.cpu()
    for kc, vc, ks, vs in ([x.cpu() for x in c] for c in caches):
        for r in range(e.B):
            for j in range(-(-len(e.rows[r]) // e.bs)):
                blk = int(table[r, j])
                part = e.rows[r][j * e.bs:(j + 1) * e.bs]
                for i, (codes, scales) in enumerate(((kc, ks), (vc, vs))):
                    x = torch.stack([y[i] for y in part]).transpose(0, 1)
                    got = codes[blk, :, :len(part)].view(ref.FP8).float() * scales[blk][:, None, None]
                    s = scales[blk][:, None, None]
                    assert bool(((got - x).abs() <= limit * (x.abs() * 2.0 ** -4 + s * 2.0 ** -10)).all())


def _attention_right(q, out, lse, cache, table, lens, start, mask, scale):
    T = int(start[-1])
    kc, vc, ks, vs = (x.cpu() for x in cache)
    want, z, w, reach = bref.tree_attention(q[:T].cpu(), kc, vc, ks, vs, table.cpu(), lens.cpu(), start.cpu(), mask, scale)
    tol = want.abs() * 2.0 ** -8 + w * (2.0 ** -11 + 2.0 ** -17 * (1 + reach[..., None])) + \
        int(lens.max()) * float(vs.max()) * 448 * 2.0 ** -24
    assert bool(((out[:T].cpu().double() - want).abs() <= tol).all())
    assert bool(((lse[:T].cpu().double() - z).abs() <= 2.0 ** -18 * (1 + reach)).all())


@pytest.mark.parametrize("H,hk,D,bs,nodes", [(8, 2, 128, 64, 3), (8, 2, 64, 16, 24), (16, 2, 128, 16, 40)])
def test_drafted_trees_are_verified_and_kept(H, hk, D, bs, nodes):
    B = 4
    e = Engine(B, H, hk, D, bs, blocks=30 if bs == 64 else 100, width=6 if bs == 64 else 24, seed=H + nodes)
    r = np.random.RandomState(nodes)
    e.step([70, 1, 130, 33])                                             # prompts
    caches = [e.cache] + [tuple(x.clone() for x in e.cache)]             # a second layer, which gets the same rows
    pools = b.TokenPools(caches)
    wq, wk = (torch.rand(D, device=DEV) + 0.5 for _ in range(2))
    scale = 1 / math.sqrt(D)
    for step in range(4):
        ql = [int(r.randint(1, nodes + 1)) for _ in range(B)]
        ql[step] = nodes
        have = [len(x) for x in e.rows]
        e.lens.copy_(torch.tensor([n + m for n, m in zip(have, ql)]))
        e.ql.copy_(torch.tensor(ql))
        T = sum(ql) + 5                                                  # padded
        parents = np.concatenate([bref.random_tree(n, r, chain=i == 1) for i, n in enumerate(ql)] + [np.full(5, 3, np.int32)])
        maps = b.smla_build_block_tables(e.lens, e.ql, e.held, e.table, e.ring, e.state, block_size=bs, num_tokens=T)
        masks = b.smla_build_tree_masks(_up(parents), e.lens, maps.query_start, max_query_len=nodes)
        q, k, v = (torch.randn((T, h, D), generator=e.gen, device=DEV).to(torch.bfloat16) for h in (H, hk, hk))
        qr, kr = b.smla_qk_norm_rope(q, k, wq, wk, masks.positions, e.cs, rot_offset=D // 2, is_neox=False)
        for c in caches:
            b.smla_kv8_append(kr, v, maps.slot_mapping, *c)
        out, lse = b.smla_kv8_tree_attn_fwd(qr, *e.cache, e.table, e.lens, maps.query_start, masks.tree_mask, scale, max_query_len=nodes)
        torch.cuda.synchronize()
        assert b.smla_device_error() == 0 and int(maps.counts[3]) == 0
        mask, pos = bref.tree_masks(parents, e.lens.cpu().numpy(), maps.query_start.cpu().numpy(), -(-nodes // 64), 0)
        assert torch.equal(masks.tree_mask.cpu(), bref.words_of(mask)) and torch.equal(masks.positions.cpu(), torch.from_numpy(pos))
        _attention_right(qr, out, lse, e.cache, e.table, e.lens, maps.query_start, mask, scale)
        # a path down each tree is kept
        kept, count, at = np.zeros((B, nodes), np.int32), np.zeros(B, np.int32), 0
        kf, vf = kr.cpu().float(), v.cpu().float()
        for i, n in enumerate(ql):
            leaf = int(r.randint(-1, n))
            path = [x for x in range(n) if leaf >= 0 and mask[at + leaf, x]]
            kept[i, :len(path)], count[i] = path, len(path)
            e.rows[i] += [(kf[at + x], vf[at + x]) for x in path]
            at += n
        lens = b.smla_keep_tokens(pools, e.table, e.lens, e.ql, _up(kept), _up(count))
        assert lens.tolist() == [len(x) for x in e.rows]
        # blocks of what was not kept go back
        e.lens.copy_(lens)
        none = b.smla_build_block_tables(e.lens, torch.zeros_like(e.ql), e.held, e.table, e.ring, e.state, block_size=bs, num_tokens=0)
        assert int(none.counts[1]) == 0 and e.held.tolist() == [-(-len(x) // bs) for x in e.rows]
        _held_right(e, caches, 16)
    e.check(*e.step([1, 2, 1, 30]))                                      # and plain steps go on from there


def test_samples_of_a_prompt_and_beams():
    B, H, hk, D, bs, blocks, width = 4, 8, 2, 64, 16, 60, 10
    e = Engine(B, H, hk, D, bs, blocks=blocks, width=width, seed=5)
    e.step([41, 0, 0, 20])
    caches = b.BlockPools(list(e.cache))
    spare = torch.full_like(e.table, -1)

    def fork(source, keep):
        lens = _up(keep)
        f = b.smla_fork_block_tables(_up(source), lens, e.held, e.table, e.ring, e.state, block_size=bs, num_blocks=blocks,
                                     block_table_out=spare)
        b.smla_copy_blocks(caches, f.copy_from, f.copy_to)
        assert int(f.counts[3]) == 0
        e.table.copy_(f.block_table)
        e.held.copy_(f.blocks_held)
        e.rows = [e.rows[s][:n] if s >= 0 else [] for s, n in zip(source, keep)]
        # every block is held or free, once; a row's last block is its own if it is not full
        held, table = e.held.tolist(), e.table.tolist()
        live = [x for row, n in zip(table, held) for x in row[:n]]
        head, count = e.state.tolist()
        free = [int(e.ring[(head + i) % len(e.ring)]) for i in range(count)]
        assert sorted(set(live) | set(free)) == list(range(blocks)) and len(set(live)) + len(free) == blocks
        for row, n, x in zip(table, held, e.rows):
            assert n == -(-len(x) // bs)
            if len(x) % bs:
                assert live.count(row[n - 1]) == 1
        return f

    def go(new):
        """A step of new tokens of each row: what the tables and the cache hold is each row's own history."""
        lens = [len(x) + n for x, n in zip(e.rows, new)]
        e.lens.copy_(torch.tensor(lens))
        e.ql.copy_(torch.tensor(new))
        T = sum(new)
        maps = b.smla_build_block_tables(e.lens, e.ql, e.held, e.table, e.ring, e.state, block_size=bs, num_tokens=T)
        assert int(maps.counts[2]) == 0 and int(maps.counts[3]) == 0     # rows that share blocks only grow here
        q, k, v = (torch.randn((T, h, D), generator=e.gen, device=DEV).to(torch.bfloat16) for h in (H, hk, hk))
        b.smla_kv8_append(k, v, maps.slot_mapping, *e.cache)
        out, lse = b.smla_kv8_attn_fwd(q, *e.cache, e.table, e.lens, maps.query_start, 0.125, max_query_len=max(new))
        kf, vf, at = k.cpu().float(), v.cpu().float(), 0
        for i, n in enumerate(new):
            e.rows[i] = e.rows[i] + [(kf[at + x], vf[at + x]) for x in range(n)]
            at += n
        chain = np.zeros((T, 64 * -(-max(new) // 64)), bool)
        at = 0
        for n in new:
            for x in range(n):
                chain[at + x, :x + 1] = True
            at += n
        _attention_right(q, out, lse, e.cache, e.table, e.lens, maps.query_start, chain, 0.125)
        _held_right(e, [e.cache], 16)

    f = fork([0, 0, 0, 3], [41, 41, 41, 20])                             # three samples of one prompt
    assert f.counts.tolist()[1:] == [2, 0, 0]
    go([1, 2, 9, 3])
    go([20, 1, 1, 1])
    f = fork([2, 0, 2, -1], [len(e.rows[2]), len(e.rows[0]), len(e.rows[2]), 0])   # beams go on from one another; one request ends
    assert f.counts.tolist()[2] > 0
    go([1, 1, 1, 30])
    fork([0, 1, 1, 3], [32, 45, 48, len(e.rows[3])])                     # cut back, onto a block's end and into one
    go([17, 1, 1, 1])
    fork([-1, -1, -1, -1], [0, 0, 0, 0])
    assert e.state.tolist()[1] == blocks


def test_a_verification_step_in_one_graph():
    """Maps, masks, norms, write, attention and the move of what is kept, captured once and replayed as contexts grow."""
    B, H, hk, D, bs, nodes = 3, 8, 2, 64, 16, 8
    e = Engine(B, H, hk, D, bs, blocks=64, width=16, seed=3)
    e.step([30, 1, 47])
    T = B * nodes
    ql, kept, count = torch.full((B,), nodes, **I32), torch.zeros((B, nodes), **I32), torch.zeros(B, **I32)
    parents, after = torch.zeros(T, **I32), torch.zeros(B, **I32)
    q, k, v = (torch.randn((T, h, D), generator=e.gen, device=DEV).to(torch.bfloat16) for h in (H, hk, hk))
    w = torch.ones(D, device=DEV)
    pools = b.TokenPools([e.cache])
    ko = torch.empty_like(k)

    def verify():
        e.lens.add_(ql)
        maps = b.smla_build_block_tables(e.lens, ql, e.held, e.table, e.ring, e.state, block_size=bs, num_tokens=T)
        masks = b.smla_build_tree_masks(parents, e.lens, maps.query_start, max_query_len=nodes)
        qr, kr = b.smla_qk_norm_rope(q, k, w, w, masks.positions, e.cs, rot_offset=D // 2, is_neox=False, k_out=ko)
        b.smla_kv8_append(kr, v, maps.slot_mapping, *e.cache)
        out, lse = b.smla_kv8_tree_attn_fwd(qr, *e.cache, e.table, e.lens, maps.query_start, masks.tree_mask, 0.1, max_query_len=nodes)
        return maps, masks, qr, out, lse

    def keep():
        b.smla_keep_tokens(pools, e.table, e.lens, ql, kept, count, seq_lens_out=after)
        e.lens.copy_(after)

    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        maps, masks, qr, out, lse = verify()
    with torch.cuda.graph(graphs[1]):
        keep()
    r = np.random.RandomState(4)
    for step in range(12):
        par = np.concatenate([bref.random_tree(nodes, r) for _ in range(B)])
        parents.copy_(_up(par))
        for x in (q, k, v):
            x.normal_(generator=e.gen)
        graphs[0].replay()
        torch.cuda.synchronize()
        start, lens = maps.query_start.cpu().numpy(), e.lens.cpu()
        mask, _ = bref.tree_masks(par, lens.numpy(), start, 1, 0)
        if step in (0, 11):
            _attention_right(qr, out, lse, e.cache, e.table, e.lens, maps.query_start, mask, 0.1)
        kept.zero_()
        for i in range(B):
            path = [x for x in range(nodes) if mask[i * nodes + int(r.randint(nodes)), x]][:int(r.randint(0, 4))]
            kept[i, :len(path)], count[i] = torch.tensor(path, **I32), len(path)
            e.rows[i] += [(ko[i * nodes + x].cpu().float(), v[i * nodes + x].cpu().float()) for x in path]
        graphs[1].replay()
        assert e.lens.tolist() == [len(x) for x in e.rows]
    assert b.smla_device_error() == 0
    _held_right(e, [e.cache], 16)


def test_kept_rows_of_the_latent_cache_serve_the_sparse_forward():
    """Drafted rows of the latent pool are kept; the sparse forward over the request's slots sees the same rows as one
    that never drafted: the same bits."""
    H, bs, ctx, n, path = 16, 64, 100, 30, [0, 3, 4, 11, 29]
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = torch.randn((ctx + n, 512), generator=g, device=DEV).to(torch.bfloat16)
    table = _up([[5, 2, 7]])
    slot = lambda j: int(table[0, j // bs]) * bs + j % bs  # noqa: E731
    pool = torch.zeros((8 * bs, 512), dtype=torch.bfloat16, device=DEV)
    pool[[slot(j) for j in range(ctx + n)]] = rows
    lens = b.smla_keep_tokens([pool], table, _up([ctx + n]), _up([n]), _up([path]), _up([len(path)]), block_size=bs)
    assert lens.tolist() == [ctx + len(path)]
    plain = torch.zeros_like(pool)
    plain[[slot(j) for j in range(ctx + len(path))]] = torch.cat([rows[:ctx], rows[[ctx + x for x in path]]])
    q = torch.randn((1, H, 512), generator=g, device=DEV).to(torch.bfloat16)
    idx = _up([[slot(j) for j in range(ctx + len(path))]])
    for x, y in zip(b.sparse_mla_fwd(q, pool, idx, 0.05), b.sparse_mla_fwd(q, plain, idx, 0.05)):
        assert torch.equal(x, y)
