"""Arrays that are read while others are written must be apart: refused on the host wherever they meet, not only where they
begin together (CPU only: the fake addresses are never dereferenced)."""
import ctypes

import pytest

from sparse_mla_attention_04_gb300 import binding as b

P = 0x100000


@pytest.fixture(scope="module")
def L():
    from sparse_mla_attention_04_gb300 import build
    build.build()
    return b.lib()


def _call(fn, structure, base, **kw):
    a = dict(base, size=ctypes.sizeof(structure))
    a.update(kw)
    return fn(ctypes.byref(structure(*[a[n] for n, _ in structure._fields_])))


def test_fork_held_counts(L):
    """Five old rows' counts and four new rows': every place of the new ones that meets the old. Those apart go on to the
    last check, of the workspace's size."""
    base = dict(source_rows=P, seq_lens=P, B=4, blocks_held=8 * P, B_old=5, block_table=2 * P, table_stride=8, blocks_held_out=9 * P,
                block_table_out=3 * P, table_out_stride=8, table_width=8, block_size=64, num_blocks=100, free_ring=4 * P,
                ring_size=100, ring_state=P, ring_state_out=P, copy_from=5 * P, copy_to=6 * P, counts=7 * P, workspace=10 * P,
                workspace_bytes=1 << 20, stream=None)

    def call(**kw):
        return _call(L.smla_fork_block_tables, b.SmlaForkBlockTablesParams, base, **kw)

    for words in range(-8, 10):
        meets = -4 < words < 5
        got = call(blocks_held_out=8 * P + 4 * words, workspace_bytes=1 << 20 if meets else 8)
        assert got == (b.SMLA_ERR_BAD_SHAPE if meets else b.SMLA_ERR_WORKSPACE_TOO_SMALL), words


@pytest.mark.parametrize("name", ["seq_lens", "query_lens", "kept_lens", "kept", "block_table"])
def test_kept_tokens_lengths(L, name):
    """Three requests: every place of the new lengths that meets an array of theirs. Apart from it the call is fine but for
    the pool's address, 4 bytes past a multiple of 8."""
    pools = (ctypes.c_void_p * 1)(20 * P)
    base = dict(block_table=P, table_stride=6, table_width=4, seq_lens=2 * P, query_lens=3 * P, kept=4 * P, kept_stride=9,
                kept_width=8, kept_lens=5 * P, seq_lens_out=6 * P, B=3, heads=1, block_size=64, row_bytes=128, num_blocks=10,
                num_pools=1, pools=ctypes.addressof(pools), scales=None, stream=None)
    words = {"kept": 2 * 9 + 8, "block_table": 2 * 6 + 4}.get(name, 3)
    for at in range(-6, words + 4):
        meets = -3 < at < words
        pools[0] = 20 * P + (0 if meets else 4)
        got = _call(L.smla_keep_tokens, b.SmlaKeepTokensParams, base, seq_lens_out=base[name] + 4 * at)
        assert got == (b.SMLA_ERR_BAD_SHAPE if meets else b.SMLA_ERR_MISALIGNED), at


def test_memory_that_meets():
    for apart in ([], [(5, 3)], [(8, 4), (0, 8), (12, 1)], [(3, 0), (0, 8), (3, 0), (8, 0), (8, 2)], [(1 << 60, 5), (7, (1 << 60) - 7)]):
        assert not b._meet(apart), apart
    for meet in ([(0, 8), (0, 8)], [(8, 4), (0, 9)], [(0, 100), (200, 5), (40, 2)], [(5, 1), (0, 6)], [(0, 10), (2, 2), (11, 3), (13, 9)]):
        assert b._meet(meet), meet
