"""Scales of the block-scaled cache that say little about what a block holds: rows
of zeros among others.

The write, derived: the first row that is not zero is the block's largest, so no
code is requantized but those of zeros, which stay zeros. Every way to cut the
tokens into calls then gives the same bits, and each value is off by half a step
of E4M3 at most (2^-4 of it, 2^-10 of the scale below the normals)."""
import math

import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu
SMALLEST = 2.0 ** -60


def _append(cuts, slots, k, v, cache):
    at = 0
    for n in cuts:
        binding.smla_kv8_append(k[at:at + n], v[at:at + n], slots[at:at + n], *cache)
        at += n
    assert at == len(slots)


def _cuts(n, how):
    return {"one call": [n], "one by one": [1] * n, "the first apart": [1, n - 1], "the last apart": [n - 1, 1]}[how]


@pytest.mark.parametrize("how", ["one by one", "the first apart", "the last apart"])
@pytest.mark.parametrize("zero", [[0], [0, 1, 2], [1], [9], [15], [3, 8, 15]])
@pytest.mark.parametrize("D,bs,size", [(128, 16, 0.5), (64, 16, 0.002), (128, 64, 1e-5), (64, 128, 0.02)])
def test_zero_rows_change_no_scale(D, bs, size, zero, how):
    """Sixteen rows of a block, some of them zeros, in one call and in several."""
    hk, n = 3, 16
    g = torch.Generator().manual_seed(D + bs + len(zero))
    k, v = (torch.randn((n, hk, D), generator=g) * size for _ in range(2))
    top = min(set(range(n)) - set(zero))
    for x in (k, v):
        x[top, :, 5] = 6 * size                                # the largest of the block
        x.clamp_(-6 * size, 6 * size)
        x[zero] = 0.0
    k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    slots = torch.arange(2 * bs, 2 * bs + n, device=DEV)
    caches = []
    for cut in (how, "one call"):
        cache = binding.new_kv8_cache(4, hk, bs, D)
        _append(_cuts(n, cut), slots, k, v, cache)
        caches.append(cache)
    for a, b in zip(*caches):
        assert torch.equal(a, b)
    kc, vc, ks, vs = caches[0]
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        got = ref.values(c, s)[2, :, :n].transpose(0, 1)
        half = x.double().abs() * 2.0 ** -4 + s[2].double()[None, :, None] * 2.0 ** -10
        assert bool(((got - x.double()).abs() <= half).all())


@pytest.mark.parametrize("requests", [3, 400])
def test_zero_and_not_finite_rows_leave_a_part_filled_block(requests):
    """One such row for each of several requests: the older tokens' codes and the scale stay."""
    hk, D, bs = 2, 64, 16
    g = torch.Generator().manual_seed(requests)
    codes = torch.randint(0, 0x7F, (requests, hk, bs, D), generator=g, dtype=torch.uint8)
    scales = torch.rand((requests, hk), generator=g) * 0.02 + 0.001
    cache = [x.to(DEV) for x in (codes, codes, scales, scales)]
    k = torch.zeros((requests, hk, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    v[1::3], v[2::3, :, ::2] = math.inf, math.nan
    off = torch.arange(requests) % (bs - 1) + 1
    binding.smla_kv8_append(k, v, (torch.arange(requests) * bs + off).to(DEV), *cache)
    kc, vc, ks, vs = (x.cpu() for x in cache)
    assert torch.equal(ks, scales) and torch.equal(vs, scales)
    rows = torch.arange(bs)[None, :] == off[:, None]
    keep = ~rows[:, None, :, None].expand_as(codes)
    assert torch.equal(kc[keep], codes[keep]) and torch.equal(vc[keep], codes[keep])
    assert int(kc[~keep].count_nonzero()) == 0
    new = vc[~keep].view(requests, hk, D)
    assert bool((new[0::3] == 0).all()) and bool((new[1::3] == 0x7E).all())
    assert bool((new[2::3, :, ::2] & 0x7F == 0x7F).all()) and bool((new[2::3, :, 1::2] == 0).all())


@pytest.mark.parametrize("tokens", [16, 3000])
def test_blocks_of_zeros_have_the_smallest_scale(tokens):
    """Of a prompt of zeros; the next row that is not sets its block's."""
    hk, D, bs = 2, 128, 64
    nb = tokens // bs + 2
    cache = binding.new_kv8_cache(nb, hk, bs, D)
    zeros = torch.zeros((tokens, hk, D), dtype=torch.bfloat16, device=DEV)
    binding.smla_kv8_append(zeros, zeros, torch.arange(tokens, device=DEV), *cache)
    used = (tokens + bs - 1) // bs
    for s in cache[2:]:
        assert bool((s[:used] == SMALLEST).all()) and bool((s[used:] == 1).all())
    row = torch.full((1, hk, D), 0.0625, dtype=torch.bfloat16, device=DEV)
    binding.smla_kv8_append(row, row, torch.tensor([tokens], device=DEV), *cache)
    b, o = tokens // bs, tokens % bs
    for c, s in ((cache[0], cache[2]), (cache[1], cache[3])):
        assert float((s[b] - 0.0625 / 448).abs().max()) <= 2.0 ** -24 * 0.0625 / 448
        assert bool((c[b, :, o] == 0x7E).all()) and int(c[b, :, :o].count_nonzero()) == 0
