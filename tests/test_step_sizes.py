"""The binding's memory of workspace sizes: bounded, and without failed answers (CPU only, a library that is not there)."""
import ctypes

import pytest

from sparse_mla_attention_04_gb300 import binding as b


class Library:
    def __init__(self):
        self.asked, self.fails = 0, False

    def smla_kv8_attn_workspace_size_of(self, params):
        self.asked += 1
        return ctypes.c_size_t(-1).value if self.fails else 4096 + self.asked

    def smla_status_string(self, status):
        return b"status %d" % status

    def smla_build_block_tables_workspace_size(self, B):
        self.asked += 1
        return 256 + B


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(b, "_lib", lib)
    caches = (b._kv8_attn_workspace, b._tables_workspace)
    for c in caches:
        c.cache_clear()
    yield lib
    for c in caches:
        c.cache_clear()


def test_a_failed_query_is_asked_again(library):
    sizes = (0, 2, 2, 32, 8, 128, 1, 16, 64)
    library.fails = True
    for _ in range(2):
        with pytest.raises(b.SmlaError):
            b._kv8_attn_workspace(*sizes)
    library.fails = False
    assert b._kv8_attn_workspace(*sizes) == b._kv8_attn_workspace(*sizes) == 4096 + 3
    assert library.asked == 3


def test_sizes_without_end_are_not_all_kept(library):
    for T in range(1, 5000):
        b._kv8_attn_workspace(0, 2, T, 32, 8, 128, 1, 16, 64)
        b._tables_workspace(T)
    for c in (b._kv8_attn_workspace, b._tables_workspace):
        assert c.cache_info().currsize <= 1024
    # no other table of the module grows with the sizes of calls
    assert not hasattr(b, "_sizes")


def test_devices_have_sizes_of_their_own(library):
    one, two = (b._kv8_attn_workspace(d, 2, 2, 32, 8, 128, 1, 16, 64) for d in (0, 1))
    assert one != two
