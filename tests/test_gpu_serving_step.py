"""The serving-step operators together, as an engine's steps use them: prompts in
chunks, then tokens one by one, requests that end and others that take their
blocks; block tables -> rotary table -> rotation -> cache write -> attention.
And the maps and the table with the framework's latent path: fused producer ->
cache -> sparse forward.

The step is checked against binary64 attention over the values that the cache
stands for (so the tolerance is the attention's: see test_gpu_kv8.py), and the
cache against the rotated keys and values: each code is off by half a step of
E4M3 (2^-4 of the value, 2^-10 of the scale below the normals) for each time its
block's scale grew and once for its own write."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


class Engine:
    """One layer's state on the device and what the host knows of it."""

    def __init__(self, B, H, hk, D, bs, blocks, width, seed):
        self.B, self.H, self.hk, self.D, self.bs = B, H, hk, D, bs
        i32 = dict(dtype=torch.int32, device=DEV)
        self.lens, self.ql, self.held = (torch.zeros(B, **i32) for _ in range(3))
        self.table = torch.full((B, width), -1, **i32)
        self.ring = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).int().to(DEV)
        self.state = torch.tensor([blocks // 2, blocks], **i32)
        self.cache = binding.new_kv8_cache(blocks, hk, bs, D)
        self.cs = binding.smla_rope_cos_sin_cache(4096, D // 2, scaling="yarn", factor=4.0, original_max_position=1024)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.rows = [[] for _ in range(B)]  # each request's rotated keys and values so far

    def step(self, new, ended=()):
        B = self.B
        for b in ended:
            self.rows[b] = []
        lens = [len(r) + n for r, n in zip(self.rows, new)]
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.ql.copy_(torch.tensor(new, dtype=torch.int32))
        T = -(-sum(new) // 8) * 8  # padded
        maps = binding.smla_build_block_tables(self.lens, self.ql, self.held, self.table, self.ring, self.state,
                                               block_size=self.bs, num_tokens=T)
        q, k, v = (torch.randn((T, h, self.D), generator=self.gen, device=DEV).to(torch.bfloat16)
                   for h in (self.H, self.hk, self.hk))
        qr, kr = binding.smla_rope(q, k, maps.positions, self.cs, rot_offset=self.D // 2, is_neox=False)
        binding.smla_kv8_append(kr, v, maps.slot_mapping, *self.cache)
        out, lse = binding.smla_kv8_attn_fwd(qr, *self.cache, self.table, self.lens, maps.query_start,
                                             1 / math.sqrt(self.D), max_query_len=max(new))
        torch.cuda.synchronize()
        assert binding.smla_device_error() == 0
        at = 0
        kr, v = kr.cpu().float(), v.cpu().float()
        for b, n in enumerate(new):
            self.rows[b] += [(kr[at + i], v[at + i]) for i in range(n)]
            at += n
        return maps, qr, out, lse

    def check(self, maps, qr, out, lse):
        T = int(maps.query_start[-1])
        kc, vc, ks, vs = (x.cpu() for x in self.cache)
        table = self.table.cpu()
        want, z, w, reach = ref.attention(qr[:T].cpu(), kc, vc, ks, vs, table, self.lens.cpu(), maps.query_start.cpu(),
                                          1 / math.sqrt(self.D))
        n = int(self.lens.max())
        top = float(vs.max()) * 448
        tol = want.abs() * 2.0 ** -8 + w * (2.0 ** -11 + 2.0 ** -17 * (1 + reach[..., None])) + n * top * 2.0 ** -24
        assert bool(((out[:T].cpu().double() - want).abs() <= tol).all())
        assert bool(((lse[:T].cpu().double() - z).abs() <= 2.0 ** -18 * (1 + reach)).all())
        # the cache holds each request's keys and values
        seen = []
        for b in range(self.B):
            for j in range(-(-len(self.rows[b]) // self.bs)):
                blk = int(table[b, j])
                seen.append(blk)
                rows = self.rows[b][j * self.bs:(j + 1) * self.bs]
                for i, (codes, scales) in enumerate(((kc, ks), (vc, vs))):
                    x = torch.stack([r[i] for r in rows]).transpose(0, 1)           # [H_kv, n, D]
                    got = codes[blk, :, :len(rows)].view(ref.FP8).float() * scales[blk][:, None, None]
                    s = scales[blk][:, None, None]
                    # a block of bs rows has its scale raised at most bs - 1 times, by more than the
                    # last step's rounding each; 4 steps cover what is drawn here
                    assert bool(((got - x).abs() <= 4 * (x.abs() * 2.0 ** -4 + s * 2.0 ** -10)).all())
        assert len(set(seen)) == len(seen), "two requests share a block"


@pytest.mark.parametrize("H,hk,D,bs", [(8, 2, 128, 64), (12, 4, 64, 16)])
def test_steps_of_a_layer(H, hk, D, bs):
    e = Engine(5, H, hk, D, bs, blocks=40 if bs == 64 else 120, width=16 if bs == 64 else 48, seed=H)
    e.check(*e.step([70, 1, 150, 33, 5]))                  # prompts, of every length
    e.check(*e.step([60, 1, 1, 64, 1]))                    # a chunk more of some, one token of others
    for _ in range(3):
        got = e.step([1, 1, 1, 1, 1])
    e.check(*got)
    e.check(*e.step([40, 1, 2, 0, 1], ended=(0, 3)))       # one ends, one is replaced by a new prompt
    e.check(*e.step([1, 1, 1, 90, 1]))
    e.check(*e.step([1, 1, 1, 1, 1]))


def test_a_decode_step_in_one_graph():
    """Maps, rotation, write and attention of one token each, captured once and replayed as contexts grow."""
    B, H, hk, D, bs = 4, 8, 2, 128, 16
    e = Engine(B, H, hk, D, bs, blocks=64, width=12, seed=3)
    e.step([30, 1, 47, 16])
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn((B, h, D), generator=e.gen, device=DEV).to(torch.bfloat16) for h in (H, hk, hk))
    ko = torch.empty_like(k)

    def decode():
        e.lens.add_(1)
        maps = binding.smla_build_block_tables(e.lens, one, e.held, e.table, e.ring, e.state, block_size=bs, num_tokens=B)
        qr, kr = binding.smla_rope(q, k, maps.positions, e.cs, rot_offset=D // 2, is_neox=False, k_out=ko)
        binding.smla_kv8_append(kr, v, maps.slot_mapping, *e.cache)
        out, lse = binding.smla_kv8_attn_fwd(qr, *e.cache, e.table, e.lens, maps.query_start, 1 / math.sqrt(D),
                                             max_query_len=1)
        return maps, qr, out, lse

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        decode()
    torch.cuda.synchronize()
    for b in range(B):
        e.rows[b].append((ko[b].cpu().float(), v[b].cpu().float()))
    with torch.cuda.graph(graph):
        got = decode()
    for _ in range(20):
        for x in (q, k, v):
            x.normal_(generator=e.gen)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            e.rows[b].append((ko[b].cpu().float(), v[b].cpu().float()))
    e.ql.fill_(1)
    e.check(*got)


def test_maps_and_table_serve_the_latent_path():
    """Block tables' slots and positions and the rotary table drive the fused producer; the sparse forward reads the
    rows back by slot: the same bits as with maps and a pool made by hand."""
    B, H, P, bs = 3, 16, 600, 64
    lens, ql = [130, 64, 200], [130, 64, 200]
    i32 = dict(dtype=torch.int32, device=DEV)
    T = sum(ql)
    table = torch.full((B, 4), -1, **i32)
    maps = binding.smla_build_block_tables(torch.tensor(lens, **i32), torch.tensor(ql, **i32), torch.zeros(B, **i32),
                                           table, torch.arange(20, **i32).flip(0).contiguous(),
                                           torch.tensor([7, 20], **i32), block_size=bs, num_tokens=T)
    cs = binding.smla_rope_cos_sin_cache(P, 64, base=5e5)
    g = torch.Generator(device=DEV).manual_seed(1)
    ql_nope = torch.randn((T, H, 512), generator=g, device=DEV).to(torch.bfloat16)
    q_pe = torch.randn((T, H, 64), generator=g, device=DEV).to(torch.bfloat16)
    kv_c, k_pe = torch.randn((T, 512), generator=g, device=DEV).to(torch.bfloat16), torch.randn((T, 64), generator=g, device=DEV).to(torch.bfloat16)
    pools, outs = [], []
    by_hand_pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
    by_hand_slots = torch.arange(T, device=DEV)
    start = np.concatenate([[0], np.cumsum(lens)])
    t_cpu = table.cpu()
    for slots, pos in ((maps.slot_mapping, maps.positions), (by_hand_slots, by_hand_pos)):
        pool = torch.zeros((20 * bs, 576), dtype=torch.bfloat16, device=DEV)
        q = binding.smla_fused_qk_rope_cache(ql_nope, q_pe, kv_c, k_pe, pos, cs, slots, pool)
        idx = np.full((T, 96), -1, np.int32)
        for b in range(B):
            for i in range(lens[b]):
                js = np.random.RandomState(1000 * b + i).permutation(i + 1)[:96]
                if slots is maps.slot_mapping:
                    idx[start[b] + i, :len(js)] = [int(t_cpu[b, j // bs]) * bs + j % bs for j in js]
                else:
                    idx[start[b] + i, :len(js)] = start[b] + js
        out, lse = binding.sparse_mla_fwd(q, pool, torch.from_numpy(idx).to(DEV), 0.05)
        outs.append((q, out, lse))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
