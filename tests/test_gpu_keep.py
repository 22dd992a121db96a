"""smla_keep_tokens against a plain implementation, an entry at a time (bits)."""
import numpy as np
import pytest
import torch

import branch_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


def _requests(lens, ql, bs, width, r, extra=2):
    nblk = [-(-n // bs) for n in lens]
    perm = r.permutation(sum(nblk) + extra)
    table = np.full((len(lens), max([width] + nblk)), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


def _lists(ql, r, share=0.3, width=None):
    width = width or max(max(ql), 1)
    kept, count = np.full((len(ql), width), -7, np.int32), np.zeros(len(ql), np.int32)
    for b, n in enumerate(ql):
        x = np.nonzero(r.rand(n) < share)[0][:width]
        count[b] = len(x)
        kept[b, :len(x)] = x
    return kept, count


def _cache(nb, hk, bs, D, g, even=False):
    codes = torch.randint(0, 256, (nb, hk, bs, D), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 3
    scale = torch.full((nb, hk), 0.03) if even else torch.rand((nb, hk), generator=g) * 0.05 + 0.001
    return codes, scale


def _up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


CASES = [
    (1, 64, 16, [40], [12]), (2, 128, 64, [100, 64, 70, 3], [30, 64, 1, 3]), (8, 128, 64, [300] * 9, [32] * 9),
    (3, 64, 32, [33, 200, 0, 500], [33, 100, 0, 333]),               # whole prompts, several blocks
    (4, 128, 128, [1000, 130], [900, 5]), (1, 64, 16, [20, 700], [3, 300]),
    (2, 64, 16, [9, 5], [20, 5])]                                    # more new tokens than there are


@pytest.mark.parametrize("hk,D,bs,lens,ql", CASES)
@pytest.mark.parametrize("share", [0.15, 0.9])
@pytest.mark.parametrize("even", [False, True])
def test_scaled(hk, D, bs, lens, ql, share, even):
    r = np.random.RandomState(hk + D + len(lens))
    g = torch.Generator().manual_seed(3)
    table, nb = _requests(lens, ql, bs, 2, r)
    n = [min(a, b) for a, b in zip(ql, lens)]
    kept, count = _lists(n, r, share)
    caches = []
    for _ in range(2):
        (kc, ks), (vc, vs) = _cache(nb, hk, bs, D, g, even), _cache(nb, hk, bs, D, g, even)
        caches.append((kc, vc, ks, vs))
    got = [tuple(x.to(DEV) for x in c) for c in caches]
    i32 = [np.array(x, np.int32) for x in (lens, ql)]
    out = binding.smla_keep_tokens(got, _up(table), _up(i32[0]), _up(i32[1]), _up(kept), _up(count))
    torch.cuda.synchronize()
    assert binding.smla_device_error(reset=True) == 0
    assert out.tolist() == [a - m + int(k) for a, m, k in zip(lens, n, count)]
    for (kc, vc, ks, vs), c in zip(got, caches):
        for codes, scale, have_c, have_s in ((c[0], c[2], kc, ks), (c[1], c[3], vc, vs)):
            ref.keep_scaled(codes, scale, table, lens, ql, kept, count)
            assert torch.equal(have_s.cpu(), scale)
            assert torch.equal(have_c.cpu(), codes)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 576), (torch.uint8, 576), (torch.uint8, 520), (torch.float32, 2), (torch.uint8, 8)])
@pytest.mark.parametrize("bs,lens,ql", [(64, [100, 64, 70, 3], [30, 64, 1, 3]), (16, [500, 33], [300, 33])])
def test_rows(dtype, D, bs, lens, ql):
    r = np.random.RandomState(D)
    table, nb = _requests(lens, ql, bs, 3, r)
    kept, count = _lists(ql, r)
    pools = [torch.randint(0, 100, (nb * bs, D)).to(dtype) for _ in range(3)]
    got = [p.to(DEV) for p in pools]
    i32 = [np.array(x, np.int32) for x in (lens, ql)]
    handle = binding.TokenPools(got, bs)
    out = binding.smla_keep_tokens(handle, _up(table), _up(i32[0]), _up(i32[1]), _up(kept), _up(count))
    assert out.tolist() == [a - m + int(k) for a, m, k in zip(lens, ql, count)]
    for have, want in zip(got, pools):
        ref.keep_rows(want, bs, table, lens, ql, kept, count)
        assert torch.equal(have.cpu(), want)


@pytest.mark.parametrize("latent", [False, True])
def test_bad_lists_and_pages(latent):
    """What does not ascend ends a list and is reported; rows outside the pool or the table stay where they are."""
    binding.smla_device_error(reset=True)
    bs, lens, ql = 16, [60, 60, 60, 60, 60], [30, 30, 30, 30, 30]
    r = np.random.RandomState(1)
    table, nb = _requests(lens, ql, bs, 2, r)
    kept = np.array([[3, 9, 9, 20], [5, 4, 6, 7], [-1, 2, 3, 4], [1, 2, 29, 30], [0, 1, 5, 12]], np.int32)
    count = np.array([4, 4, 4, 4, 9], np.int32)
    table[4, 2] = nb + 5                                             # a block past the pool
    table[3, 3] = -1
    g = torch.Generator().manual_seed(3)
    up = [np.array(x, np.int32) for x in (lens, ql)]
    if latent:
        pool = torch.randint(0, 255, (nb * bs, 64), generator=g, dtype=torch.uint8)
        have = pool.to(DEV)
        out = binding.smla_keep_tokens([have], _up(table), _up(up[0]), _up(up[1]), _up(kept), _up(count), block_size=bs)
        ref.keep_rows(pool, bs, table, lens, ql, kept, count)
        assert torch.equal(have.cpu(), pool)
    else:
        (kc, ks), (vc, vs) = _cache(nb, 2, bs, 64, g), _cache(nb, 2, bs, 64, g)
        have = [x.to(DEV) for x in (kc, vc, ks, vs)]
        out = binding.smla_keep_tokens([have], _up(table), _up(up[0]), _up(up[1]), _up(kept), _up(count))
        ref.keep_scaled(kc, ks, table, lens, ql, kept, count)
        ref.keep_scaled(vc, vs, table, lens, ql, kept, count)
        for a, b in zip(have, (kc, vc, ks, vs)):
            assert torch.equal(a.cpu(), b)
    assert out.tolist() == [30 + len(ref.kept_list(kept[b], count[b], 30, 4)[0]) for b in range(5)]
    assert binding.smla_device_error(reset=True) == 16


def test_strided_tables_many_layers_and_replay():
    """More pools than a launch holds, strided tables and lists, a captured call that follows the lists."""
    bs, hk, D, lens, ql = 16, 1, 64, [40, 23], [20, 10]
    r = np.random.RandomState(5)
    g = torch.Generator().manual_seed(5)
    table, nb = _requests(lens, ql, bs, 4, r)
    kept, count = _lists(ql, r)
    layers = [_cache(nb, hk, bs, D, g) + _cache(nb, hk, bs, D, g) for _ in range(70)]
    got = [tuple(x.to(DEV) for x in (a, c, b, d)) for a, b, c, d in layers]
    wide = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = _up(table)
    list_wide = torch.full((2, kept.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    list_wide[:, :kept.shape[1]] = _up(kept)
    n, q, c = (_up(np.array(x, np.int32)) for x in (lens, ql, count))
    handle = binding.TokenPools(got)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = binding.smla_keep_tokens(handle, wide[:, :table.shape[1]], n, q, list_wide[:, :kept.shape[1]], c)
    kept2, count2 = _lists(ql, r, 0.5, kept.shape[1])
    list_wide[:, :kept.shape[1]] = _up(kept2)
    c.copy_(_up(count2))
    graph.replay()
    assert out.tolist() == [a - m + int(k) for a, m, k in zip(lens, ql, count2)]
    for (kc, ks, vc, vs), have in zip(layers, got):
        ref.keep_scaled(kc, ks, table, lens, ql, kept2, count2)
        ref.keep_scaled(vc, vs, table, lens, ql, kept2, count2)
        for a, b in zip(have, (kc, vc, ks, vs)):
            assert torch.equal(a.cpu(), b)
    with pytest.raises(binding.SmlaError):
        binding.smla_keep_tokens(handle, wide[:, :table.shape[1]], n, q, list_wide[:, :kept.shape[1]], c, seq_lens_out=n)
    with pytest.raises(ValueError):
        binding.smla_keep_tokens(handle, wide, n, q, list_wide, c, block_size=32)
    with pytest.raises(ValueError):
        binding.TokenPools([got[0], tuple(x[:1] for x in got[1])])
    with pytest.raises(ValueError):
        binding.TokenPools([got[0], got[1], got[0]])                 # its rows would move twice
    with pytest.raises(ValueError):
        binding.TokenPools([got[0][0].view(-1, 64), got[1][0].view(-1, 64)])                   # latent pools without block_size
    with pytest.raises(ValueError, match="block_size"):
        binding.TokenPools([got[0][0].view(-1, 64)], block_size=0)


def test_pools_past_32_bits():
    """Rows whose byte offsets pass 2^32."""
    bs, D = 128, 576
    nb = (1 << 32) // (bs * D) + 40
    pool = torch.zeros((nb * bs, D), dtype=torch.uint8, device=DEV)
    table = np.array([[nb - 1, nb - 30]], np.int32)
    rows = torch.randint(1, 255, (200, D), dtype=torch.uint8, device=DEV)
    slots = torch.cat([torch.arange((nb - 1) * bs, nb * bs), torch.arange((nb - 30) * bs, (nb - 30) * bs + 72)]).to(DEV)
    pool[slots] = rows
    kept = np.array([[5, 90, 150]], np.int32)
    one = lambda x: _up(np.array([x], np.int32))  # noqa: E731
    out = binding.smla_keep_tokens([pool], _up(table), one(200), one(190), _up(kept), one(3), block_size=bs)
    assert out.tolist() == [13]
    want = rows.clone()
    want[10:13] = rows[[15, 100, 160]]
    assert torch.equal(pool[slots], want)
