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
