"""More arguments that the serving-step operators refuse on the host, before any launch (CPU only: the fake addresses
are never dereferenced)."""
import pytest

from sparse_mla_attention_04_gb300 import binding as b

P = 0x10000


@pytest.fixture(scope="module")
def L():
    from sparse_mla_attention_04_gb300 import build
    build.build()
    return b.lib()


@pytest.mark.parametrize("m", [1e39, 1.7e308, 3.5e38])
def test_attention_factors_beyond_binary32(L, m):
    """The table would hold infinities, and NaN where a cosine or sine is 0."""
    assert L.smla_rope_cos_sin_cache(P, 16, 0, 64, 1e4, b.SMLA_ROPE_NONE, 1.0, 0, 32.0, 1.0, m, None) == b.SMLA_ERR_BAD_SHAPE


def test_requests_and_table_widths_whose_indexes_pass_31_bits(L):
    """Loops over requests and over a row's blocks step beyond their ends before they stop."""
    most = 1 << 30

    def tables(B, width):
        return L.smla_build_block_tables(P, P, P, P, B, 16, P, width, width, P, 100, P, P, P, P, P, P, 8, P, P, 1 << 50, None)

    for B, width in ((most + 1, 1), ((1 << 31) - 1, 0), (1, most + 1), (1, (1 << 31) - 1), (1024, 1 << 21), (1 << 16, 1 << 15)):
        assert tables(B, width) == b.SMLA_ERR_UNSUPPORTED, (B, width)
    none = b.ctypes.c_size_t(-1).value
    assert L.smla_build_block_tables_workspace_size(most) != none
    assert L.smla_build_block_tables_workspace_size(most + 1) == none

    def attention(B):
        a = dict(size=b.ctypes.sizeof(b.SmlaKv8AttnParams), q=P, q_stride_t=4096, q_stride_h=128, k_cache=P, v_cache=P,
                 k_scale=P, v_scale=P, num_blocks=100, block_table=P, table_stride=16, table_width=16, seq_lens=P,
                 query_start=P, B=B, T=2, H=1, H_kv=1, D=128, block_size=64, max_query_len=1, window=0, scale=0.1,
                 sinks=None, out=P, lse=P, workspace=P, workspace_bytes=1 << 50, stream=None)
        return L.smla_kv8_attn_fwd(b.ctypes.byref(b.SmlaKv8AttnParams(*[a[n] for n, _ in b.SmlaKv8AttnParams._fields_])))

    for B in (most + 1, (1 << 31) - 1):
        assert attention(B) == b.SMLA_ERR_UNSUPPORTED, B
