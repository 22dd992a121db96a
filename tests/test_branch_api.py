"""The operators of a step that drafts and branches refuse bad arguments on the host, before any launch
(CPU only: the fake addresses are never dereferenced)."""
import ctypes

import pytest
import torch

from sparse_mla_attention_04_gb300 import binding as b

P = 0x10000


@pytest.fixture(scope="module")
def L():
    from sparse_mla_attention_04_gb300 import build
    build.build()
    return b.lib()


def _call(fn, structure, base, **kw):
    a = dict(base, size=ctypes.sizeof(structure))
    a.update(kw)
    return fn(ctypes.byref(structure(*[a[n] for n, _ in structure._fields_])))


def test_norm_rope_argument_checks(L):
    base = dict(dtype=0, weight_dtype=0, q=P, q_stride_t=2048, q_stride_h=128, q_out=2 * P, q_out_stride_t=2048,
                q_out_stride_h=128, k=3 * P, k_stride_t=256, k_stride_h=128, k_out=4 * P, k_out_stride_t=256,
                k_out_stride_h=128, q_weight=P, q_weight_stride_h=0, k_weight=P, k_weight_stride_h=128, weight_offset=0.0,
                eps=1e-6, positions=P, cos_sin_cache=P, max_position=100, T=3, H=16, H_k=2, D=128, rot_dim=64,
                rot_offset=64, is_neox=1, stream=None)

    def call(**kw):
        return _call(L.smla_qk_norm_rope, b.SmlaQkNormRopeParams, base, **kw)

    assert L.smla_qk_norm_rope(None) == b.SMLA_ERR_NULL_POINTER
    assert call(T=0) == b.SMLA_OK
    assert call(H=0, H_k=0) == b.SMLA_OK
    inf, nan = float("inf"), float("nan")
    for bad in (dict(size=8), dict(T=-1), dict(H=-1), dict(H_k=-1), dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=258),
                dict(rot_offset=65), dict(rot_offset=-1), dict(D=1 << 17), dict(max_position=-1), dict(q_stride_t=-1),
                dict(k_weight_stride_h=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-31), dict(eps=inf), dict(eps=nan),
                dict(weight_offset=nan), dict(weight_offset=inf), dict(q=2 * P, q_stride_h=256), dict(q_out_stride_h=64),
                dict(k_out_stride_t=0)):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    assert call(dtype=3) == b.SMLA_ERR_BAD_DTYPE
    assert call(weight_dtype=1) == b.SMLA_ERR_BAD_DTYPE          # fp16 weights of bf16 tensors
    assert call(dtype=2, weight_dtype=0) == b.SMLA_ERR_BAD_DTYPE
    for name in ("q", "q_out", "k", "k_out", "positions", "cos_sin_cache"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    for name in ("q", "q_out", "k", "k_out", "q_weight", "k_weight"):
        assert call(**{name: P + 1}) == b.SMLA_ERR_MISALIGNED, name
    assert call(positions=P + 4) == b.SMLA_ERR_MISALIGNED
    assert call(weight_dtype=2, q_weight=P + 2) == b.SMLA_ERR_MISALIGNED


def test_tree_mask_argument_checks(L):
    def call(parents=P, lens=P, start=P, B=2, T=5, words=1, window=0, mask=P, pos=P):
        return L.smla_build_tree_masks(parents, lens, start, B, T, words, window, mask, pos, None)

    assert call(T=0) == b.SMLA_OK
    for bad in (dict(B=-1), dict(T=-1), dict(words=0), dict(window=-1)):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    assert call(words=17) == b.SMLA_ERR_UNSUPPORTED
    assert call(T=(1 << 31) - 1) == b.SMLA_ERR_UNSUPPORTED
    for name in ("parents", "lens", "start", "mask", "pos"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
        assert call(**{name: P + 2}) == b.SMLA_ERR_MISALIGNED, name
    assert call(mask=P + 4) == b.SMLA_ERR_MISALIGNED


def test_tree_attention_argument_checks(L):
    attn = dict(size=ctypes.sizeof(b.SmlaKv8AttnParams), q=P, q_stride_t=1024, q_stride_h=128, k_cache=P, v_cache=P, k_scale=P,
                v_scale=P, num_blocks=10, block_table=P, table_stride=4, table_width=4, seq_lens=P, query_start=P, B=2, T=6,
                H=8, H_kv=2, D=128, block_size=64, max_query_len=3, window=0, scale=0.1, sinks=None, out=P, lse=None,
                workspace=P, workspace_bytes=1 << 30, stream=None)

    def call(size=ctypes.sizeof(b.SmlaKv8TreeAttnParams), mask=P, words=1, positions=None, **kw):
        a = dict(attn, **kw)
        inner = b.SmlaKv8AttnParams(*[a[n] for n, _ in b.SmlaKv8AttnParams._fields_])
        return L.smla_kv8_tree_attn_fwd(ctypes.byref(b.SmlaKv8TreeAttnParams(size, inner, mask, words, positions)))

    assert L.smla_kv8_tree_attn_fwd(None) == b.SMLA_ERR_NULL_POINTER
    assert call(T=0) == b.SMLA_OK
    for bad in (dict(words=0), dict(words=(1 << 20) + 1)):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    n = ctypes.sizeof(b.SmlaKv8TreeAttnParams)
    assert L.smla_kv8_tree_attn_fwd(ctypes.byref(b.SmlaKv8TreeAttnParams(n - 8))) == b.SMLA_ERR_BAD_SHAPE
    assert call(H=9) == b.SMLA_ERR_BAD_SHAPE                      # and what smla_kv8_attn_fwd refuses
    assert call(D=96) == b.SMLA_ERR_UNSUPPORTED
    assert call(block_size=48) == b.SMLA_ERR_UNSUPPORTED
    assert call(mask=None) == b.SMLA_ERR_NULL_POINTER
    assert call(window=5) == b.SMLA_ERR_NULL_POINTER              # a window without positions
    assert call(mask=P + 4) == b.SMLA_ERR_MISALIGNED
    assert call(window=5, positions=P + 4) == b.SMLA_ERR_MISALIGNED


def _pointers(*x):
    return (ctypes.c_void_p * len(x))(*x)


def test_keep_argument_checks(L):
    pools, scales = _pointers(P, 2 * P), _pointers(3 * P, 4 * P)
    base = dict(block_table=P, table_stride=4, table_width=4, seq_lens=P, query_lens=2 * P, kept=P, kept_stride=8, kept_width=8,
                kept_lens=3 * P, seq_lens_out=4 * P, B=2, heads=2, block_size=64, row_bytes=128, num_blocks=10, num_pools=2,
                pools=ctypes.addressof(pools), scales=ctypes.addressof(scales), stream=None)

    def call(**kw):
        for n in ("pools", "scales"):
            if isinstance(kw.get(n), ctypes.Array):
                kw[n] = ctypes.addressof(kw[n])
        return _call(L.smla_keep_tokens, b.SmlaKeepTokensParams, base, **kw)

    assert L.smla_keep_tokens(None) == b.SMLA_ERR_NULL_POINTER
    assert call(B=0) == b.SMLA_OK
    for bad in (dict(size=8), dict(B=-1), dict(num_pools=0), dict(heads=0), dict(row_bytes=0), dict(num_blocks=-1),
                dict(table_width=-1), dict(table_stride=3), dict(kept_width=-1), dict(kept_stride=7),
                dict(seq_lens_out=P), dict(seq_lens_out=2 * P), dict(seq_lens_out=3 * P)):   # lengths in place
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    for bad in (dict(block_size=48), dict(row_bytes=96), dict(scales=None, row_bytes=12), dict(scales=None, row_bytes=1 << 17),
                dict(num_blocks=1 << 31), dict(table_width=1 << 25, table_stride=1 << 25), dict(B=1 << 20, heads=1 << 20)):
        assert call(**bad) == b.SMLA_ERR_UNSUPPORTED, bad
    for name in ("block_table", "seq_lens", "query_lens", "kept", "kept_lens", "pools"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    none, odd = _pointers(P, None), _pointers(P, P + 8)
    assert call(pools=none) == b.SMLA_ERR_NULL_POINTER
    assert call(scales=none) == b.SMLA_ERR_NULL_POINTER
    assert call(pools=odd) == b.SMLA_ERR_MISALIGNED              # (rows as they are: 8 bytes will do)
    odd4 = _pointers(P, P + 4)
    assert call(pools=odd4, scales=None) == b.SMLA_ERR_MISALIGNED
    for name in ("block_table", "seq_lens", "kept", "seq_lens_out"):
        assert call(**{name: P + 2}) == b.SMLA_ERR_MISALIGNED, name


def test_copy_argument_checks(L):
    pools, size = _pointers(P, 2 * P), (ctypes.c_int64 * 2)(64, 1024)

    def call(pools=pools, size=size, count=2, frm=P, to=P, n=3, blocks=10):
        return L.smla_copy_blocks(pools, size, count, frm, to, n, blocks, None)

    for none in (dict(count=0), dict(n=0), dict(blocks=0)):
        assert call(**none) == b.SMLA_OK, none
    for bad in (dict(count=-1), dict(n=-1), dict(blocks=-1), dict(size=(ctypes.c_int64 * 2)(64, -1))):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    assert call(blocks=1 << 31) == b.SMLA_ERR_UNSUPPORTED
    for bad in (dict(pools=None), dict(size=None), dict(frm=None), dict(to=None), dict(pools=_pointers(P, None))):
        assert call(**bad) == b.SMLA_ERR_NULL_POINTER, bad
    assert call(frm=P + 2) == b.SMLA_ERR_MISALIGNED


def test_fork_argument_checks(L):
    base = dict(source_rows=P, seq_lens=P, B=4, blocks_held=P, B_old=2, block_table=P, table_stride=8, blocks_held_out=2 * P,
                block_table_out=2 * P, table_out_stride=8, table_width=8, block_size=64, num_blocks=100, free_ring=P,
                ring_size=100, ring_state=P, ring_state_out=P, copy_from=P, copy_to=P, counts=P, workspace=P,
                workspace_bytes=1 << 20, stream=None)

    def call(**kw):
        return _call(L.smla_fork_block_tables, b.SmlaForkBlockTablesParams, base, **kw)

    assert L.smla_fork_block_tables(None) == b.SMLA_ERR_NULL_POINTER
    for bad in (dict(size=8), dict(B=-1), dict(B_old=-1), dict(table_width=-1), dict(num_blocks=-1), dict(ring_size=0),
                dict(table_stride=7), dict(table_out_stride=7), dict(blocks_held_out=P), dict(block_table_out=P),
                dict(block_table_out=P + 15 * 4), dict(block_table_out=P - 31 * 4)):       # the new rows over the old
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    for bad in (dict(block_size=8), dict(num_blocks=1 << 31), dict(table_width=1 << 25, table_stride=1 << 25, table_out_stride=1 << 25),
                dict(B=1 << 29)):
        assert call(**bad) == b.SMLA_ERR_UNSUPPORTED, bad
    for name in ("source_rows", "seq_lens", "blocks_held", "block_table", "blocks_held_out", "block_table_out", "free_ring",
                 "ring_state", "ring_state_out", "copy_from", "copy_to", "counts", "workspace"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
        assert call(**{name: 5 * P + 2}) == b.SMLA_ERR_MISALIGNED, name
    need = L.smla_fork_block_tables_workspace_size(2, 4, 8, 100)
    assert call(workspace_bytes=need - 1) == b.SMLA_ERR_WORKSPACE_TOO_SMALL
    assert L.smla_fork_block_tables_workspace_size(-1, 4, 8, 100) == ctypes.c_size_t(-1).value
    assert L.smla_fork_block_tables_workspace_size(1 << 20, 4, 1 << 20, 100) == ctypes.c_size_t(-1).value


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    cs = torch.zeros((8, 64))
    with pytest.raises(ValueError):                               # not on a GPU
        b.smla_qk_norm_rope(x, None, None, None, i64, cs)
    with pytest.raises(TypeError):
        b.smla_qk_norm_rope(x.double(), None, None, None, i64, cs)
    with pytest.raises(ValueError):
        b.smla_build_tree_masks(i32, i32, i32, max_query_len=4)
    with pytest.raises(ValueError):
        b.smla_kv8_tree_attn_fwd(x, x, x, x, x, i32, i32, i32, None, 1.0, max_query_len=1)
    with pytest.raises(ValueError):
        b.smla_keep_tokens([], i32, i32, i32, i32, i32)
    with pytest.raises(ValueError):
        b.smla_keep_tokens([torch.zeros((64, 576))], i32, i32, i32, i32, i32, block_size=64)
    with pytest.raises(ValueError):
        b.smla_fork_block_tables(i32, i32, i32, i32, i32, i32, block_size=16, num_blocks=4)
    with pytest.raises(ValueError):
        b.smla_copy_blocks([], i32, i32)
    with pytest.raises(ValueError):
        b.smla_copy_blocks([torch.zeros((4, 4))], i32, i32)


def test_one_tensor_is_not_a_sequence_of_pools():
    pool, i32 = torch.zeros((4, 4, 8)), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: b.BlockPools(pool), lambda: b.smla_copy_blocks(pool, i32, i32), lambda: b.TokenPools(pool[0], 2),
                 lambda: b.smla_keep_tokens(pool[0], i32, i32, i32, i32, i32, block_size=2)):
        with pytest.raises(TypeError, match="sequence"):
            call()
