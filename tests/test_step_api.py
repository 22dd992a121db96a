"""The serving-step operators refuse bad arguments on the host, before any
launch (CPU only: the fake addresses are never dereferenced)."""
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


def test_block_tables_argument_checks(L):
    def call(**kw):
        a = dict(lens=P, ql=P, held=P, held_out=P, B=4, bs=64, table=P, stride=10, width=10, ring=P, cap=100, state=P,
                 state_out=P, start=P, pos=P, slots=P, req=P, T=8, counts=P, ws=P, wsb=1 << 20)
        a.update(kw)
        return L.smla_build_block_tables(*[a[n] for n in (
            "lens", "ql", "held", "held_out", "B", "bs", "table", "stride", "width", "ring", "cap", "state",
            "state_out", "start", "pos", "slots", "req", "T", "counts", "ws", "wsb")], None)

    assert call(B=-1) == b.SMLA_ERR_BAD_SHAPE
    assert call(T=-1) == b.SMLA_ERR_BAD_SHAPE
    assert call(T=1 << 31) == b.SMLA_ERR_BAD_SHAPE
    assert call(stride=9) == b.SMLA_ERR_BAD_SHAPE           # rows would overlap
    assert call(cap=0) == b.SMLA_ERR_BAD_SHAPE
    assert call(bs=48) == b.SMLA_ERR_UNSUPPORTED
    for name in ("lens", "ql", "held", "held_out", "table", "ring", "state", "state_out", "start", "pos", "slots",
                 "counts", "ws"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    for name in ("lens", "table", "ring", "pos", "slots", "req", "ws"):
        assert call(**{name: P + 2}) == b.SMLA_ERR_MISALIGNED, name
    need = L.smla_build_block_tables_workspace_size(4)
    assert call(wsb=need - 1) == b.SMLA_ERR_WORKSPACE_TOO_SMALL
    assert L.smla_build_block_tables_workspace_size(-1) == ctypes.c_size_t(-1).value


def test_rope_table_argument_checks(L):
    def call(table=P, n=16, first=0, rot=64, base=1e4, kind=0, factor=1.0, orig=4096, fast=32.0, slow=1.0, m=0.0):
        return L.smla_rope_cos_sin_cache(table, n, first, rot, base, kind, factor, orig, fast, slow, m, None)

    assert call(n=0) == b.SMLA_OK
    assert call(table=None) == b.SMLA_ERR_NULL_POINTER
    assert call(table=P + 2) == b.SMLA_ERR_MISALIGNED
    for bad in (dict(n=-1), dict(first=-1), dict(first=1 << 31), dict(rot=0), dict(rot=63), dict(rot=258),
                dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(m=-1.0), dict(m=float("nan")),
                dict(kind=1, factor=0.5), dict(kind=1, factor=float("nan")), dict(kind=2, factor=2.0, rot=2),
                dict(kind=3, factor=2.0, orig=0), dict(kind=3, factor=2.0, slow=0.0),
                dict(kind=3, factor=2.0, fast=1.0), dict(kind=3, factor=2.0, fast=float("inf"))):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    assert call(kind=4) == b.SMLA_ERR_BAD_DTYPE


def test_rope_argument_checks(L):
    def call(**kw):
        a = dict(size=ctypes.sizeof(b.SmlaRopeParams), dtype=0, q=P, q_stride_t=2048, q_stride_h=128, q_out=2 * P,
                 q_out_stride_t=2048, q_out_stride_h=128, k=3 * P, k_stride_t=256, k_stride_h=128, k_out=4 * P,
                 k_out_stride_t=256, k_out_stride_h=128, positions=P, cos_sin_cache=P, max_position=100, T=3, H=16,
                 H_k=2, D=128, rot_dim=64, rot_offset=64, is_neox=1, inverse=0, stream=None)
        a.update(kw)
        return L.smla_rope(ctypes.byref(b.SmlaRopeParams(*[a[n] for n, _ in b.SmlaRopeParams._fields_])))

    assert L.smla_rope(None) == b.SMLA_ERR_NULL_POINTER
    assert call(T=0) == b.SMLA_OK
    for bad in (dict(size=8), dict(T=-1), dict(H=-1), dict(rot_dim=63), dict(rot_dim=258), dict(rot_offset=65),
                dict(rot_offset=-1), dict(D=1 << 17), dict(max_position=-1), dict(q_stride_t=-1),
                dict(q=2 * P, q_stride_h=256),          # in place with other strides
                dict(q_out_stride_h=64),                # output rows over one another
                dict(k_out_stride_t=0)):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    assert call(dtype=3) == b.SMLA_ERR_BAD_DTYPE
    for name in ("q", "q_out", "k", "k_out", "positions", "cos_sin_cache"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    for name in ("q", "q_out", "k", "k_out"):
        assert call(**{name: 5 * P + 1}) == b.SMLA_ERR_MISALIGNED, name
    assert call(positions=P + 4) == b.SMLA_ERR_MISALIGNED


def test_append_argument_checks(L):
    def call(**kw):
        a = dict(k=P, kt=1024, kh=128, v=P, vt=1024, vh=128, slots=P, T=4, H=8, D=128, bs=64, kc=P, vc=P, ks=P, vs=P,
                 nb=10)
        a.update(kw)
        return L.smla_kv8_append(*[a[n] for n in ("k", "kt", "kh", "v", "vt", "vh", "slots", "T", "H", "D", "bs",
                                                  "kc", "vc", "ks", "vs", "nb")], None)

    assert call(T=0) == b.SMLA_OK
    for bad in (dict(T=-1), dict(H=0), dict(nb=-1), dict(kt=-8)):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    for bad in (dict(D=96), dict(bs=8), dict(bs=256)):
        assert call(**bad) == b.SMLA_ERR_UNSUPPORTED, bad
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    for bad in (dict(kt=1020), dict(vh=4), dict(k=P + 8), dict(kc=P + 8), dict(slots=P + 4), dict(ks=P + 2)):
        assert call(**bad) == b.SMLA_ERR_MISALIGNED, bad


def test_attention_argument_checks(L):
    def call(**kw):
        a = dict(size=ctypes.sizeof(b.SmlaKv8AttnParams), q=P, q_stride_t=4096, q_stride_h=128, k_cache=P, v_cache=P,
                 k_scale=P, v_scale=P, num_blocks=100, block_table=P, table_stride=16, table_width=16, seq_lens=P,
                 query_start=P, B=2, T=2, H=32, H_kv=8, D=128, block_size=64, max_query_len=1, window=0, scale=0.1,
                 sinks=None, out=P, lse=P, workspace=P, workspace_bytes=1 << 40, stream=None)
        a.update(kw)
        return L.smla_kv8_attn_fwd(ctypes.byref(b.SmlaKv8AttnParams(*[a[n] for n, _ in b.SmlaKv8AttnParams._fields_])))

    assert L.smla_kv8_attn_fwd(None) == b.SMLA_ERR_NULL_POINTER
    assert call(T=0) == b.SMLA_OK
    assert call(B=0) == b.SMLA_OK
    for bad in (dict(size=8), dict(B=-1), dict(T=-1), dict(H=0), dict(H_kv=0), dict(H=30), dict(max_query_len=-1),
                dict(num_blocks=-1), dict(table_stride=15), dict(window=-1), dict(q_stride_t=-8),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == b.SMLA_ERR_BAD_SHAPE, bad
    for bad in (dict(D=96), dict(block_size=48), dict(table_width=1 << 26, table_stride=1 << 26), dict(T=(1 << 30) + 8)):
        assert call(**bad) == b.SMLA_ERR_UNSUPPORTED, bad
    for name in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "seq_lens", "query_start", "out",
                 "workspace"):
        assert call(**{name: None}) == b.SMLA_ERR_NULL_POINTER, name
    for bad in (dict(q=P + 8), dict(q_stride_h=132), dict(out=P + 8), dict(k_cache=P + 4), dict(lse=P + 2),
                dict(sinks=P + 1), dict(workspace=P + 16), dict(seq_lens=P + 2)):
        assert call(**bad) == b.SMLA_ERR_MISALIGNED, bad


def test_binding_refusals():
    """The binding's own checks, on tensors that are not on a GPU or do not fit together."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        b.smla_build_block_tables(i32(3), i32(3), i32(3), i32(3, 4), i32(9), i32(2), block_size=16, num_tokens=4)
    with pytest.raises(TypeError):
        b.smla_build_block_tables(i32(3).long(), i32(3), i32(3), i32(3, 4), i32(9), i32(2), block_size=16, num_tokens=4)
    with pytest.raises(ValueError):
        b.smla_rope_cos_sin_cache(16, 64, scaling="other")
    with pytest.raises(ValueError):
        b.smla_rope_cos_sin_cache(16, 64, attention_factor=0.0)
    with pytest.raises(TypeError):
        b.smla_rope(torch.zeros(2, 2, 64, dtype=torch.float64), None, torch.zeros(2, dtype=torch.int64),
                    torch.zeros(8, 64))
    with pytest.raises(TypeError):
        b.smla_kv8_append(torch.zeros(2, 2, 64), torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int64),
                          torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64), torch.ones(4, 2), torch.ones(4, 2))
    with pytest.raises(ValueError):
        b._kv8_cache(torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
                     torch.ones(4, 2), torch.ones(4, 2))   # not on a GPU


def test_packed_structures_match_the_headers():
    """The packed layouts have the C structures' size and field offsets."""
    for packed, st in ((b._ROPE_PARAMS, b.SmlaRopeParams), (b._KV8_ATTN_PARAMS, b.SmlaKv8AttnParams)):
        assert packed.size == ctypes.sizeof(st)
        n = len(st._fields_)
        values = [i + 1 for i in range(n)]
        got = st.from_buffer_copy(packed.pack(*values))
        assert [getattr(got, name) for name, _ in st._fields_] == values


def test_row_strides_that_no_row_uses_and_rows_over_one_another(L):
    """Strides of a single token or head are free; output rows of a rotation must lie apart."""
    def rope(st, sh, positions=P, T=4, H=8):
        a = dict(size=ctypes.sizeof(b.SmlaRopeParams), dtype=0, q=P, q_stride_t=4096, q_stride_h=128, q_out=2 * P,
                 q_out_stride_t=st, q_out_stride_h=sh, k=None, k_stride_t=0, k_stride_h=0, k_out=None, k_out_stride_t=0,
                 k_out_stride_h=0, positions=positions, cos_sin_cache=P, max_position=100, T=T, H=H, H_k=0, D=128,
                 rot_dim=64, rot_offset=0, is_neox=1, inverse=0, stream=None)
        return L.smla_rope(ctypes.byref(b.SmlaRopeParams(*[a[n] for n, _ in b.SmlaRopeParams._fields_])))

    for st, sh in ((128, 128), (64, 1024), (0, 128), (256, 192), (1000, 128)):
        assert rope(st, sh) == b.SMLA_ERR_BAD_SHAPE, (st, sh)
    # heads within a token, tokens within a head: refused for the positions' address only
    for st, sh in ((1024, 128), (4096, 130), (128, 512)):
        assert rope(st, sh, P + 4) == b.SMLA_ERR_MISALIGNED, (st, sh)

    def append(**kw):
        a = dict(k=P, kt=1024, kh=128, v=P, vt=1024, vh=128, slots=P + 4, T=4, H=8, D=128, bs=64, kc=P, vc=P, ks=P, vs=P,
                 nb=10)
        a.update(kw)
        return L.smla_kv8_append(*[a[n] for n in ("k", "kt", "kh", "v", "vt", "vh", "slots", "T", "H", "D", "bs",
                                                  "kc", "vc", "ks", "vs", "nb")], None)

    assert append(T=(1 << 31) - 1) == b.SMLA_ERR_UNSUPPORTED
    for kw in (dict(T=1, kt=1021, vt=3), dict(H=1, kh=5, vh=7)):
        assert append(**kw) == b.SMLA_ERR_MISALIGNED       # (the slots' address)


def test_workspace_of_a_call(L):
    """-1 for what the call would refuse; on a GPU no more than the bound without the table's width."""
    def need(**kw):
        a = dict(size=ctypes.sizeof(b.SmlaKv8AttnParams), q=None, q_stride_t=0, q_stride_h=0, k_cache=None, v_cache=None,
                 k_scale=None, v_scale=None, num_blocks=0, block_table=None, table_stride=0, table_width=16, seq_lens=None,
                 query_start=None, B=2, T=2, H=32, H_kv=8, D=128, block_size=64, max_query_len=1, window=0, scale=0.1,
                 sinks=None, out=None, lse=None, workspace=None, workspace_bytes=0, stream=None)
        a.update(kw)
        return L.smla_kv8_attn_workspace_size_of(ctypes.byref(b.SmlaKv8AttnParams(*[a[n] for n, _ in b.SmlaKv8AttnParams._fields_])))

    none = ctypes.c_size_t(-1).value
    assert L.smla_kv8_attn_workspace_size_of(None) == none
    for bad in (dict(size=8), dict(B=-1), dict(D=96), dict(block_size=48), dict(table_width=-1), dict(table_width=1 << 26)):
        assert need(**bad) == none, bad
