"""Which caches smla_keep_tokens takes in one call: their tensors lie apart (GPU: the handle wants tensors there)."""
import pytest
import torch

from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


def test_shared_memory_is_refused():
    a, c = binding.new_kv8_cache(6, 2, 16, 64), binding.new_kv8_cache(6, 2, 16, 64)
    binding.TokenPools([a, c])
    room = torch.zeros((9, 2, 16, 64), dtype=torch.uint8, device=DEV)
    scales = torch.ones((9, 2), device=DEV)
    for bad in ([a, a], [(a[0], a[0], a[2], a[3])], [(a[0], a[1], a[2], a[2])],       # a pool twice; K's and V's scales in one
                [a, (c[0], c[1], a[2], c[3])], [a, (c[0], c[1], c[2], a[2])],         # two layers' scales
                [(room[:6], room[3:], a[2], a[3])], [(a[0], a[1], scales[:6], scales[2:8])],   # views that overlap
                [a, (room[:6], c[1], c[2], a[3])]):
        with pytest.raises(ValueError, match="share memory"):
            binding.TokenPools(bad)
    binding.TokenPools([(room[:4], room[5:], scales[:4], scales[4:8])])               # side by side in one allocation
    flat = torch.zeros((100, 576), dtype=torch.uint8, device=DEV)
    binding.TokenPools([flat[:48], flat[48:96]], 16)
    for bad in ([flat[:48], flat[47:95]], [flat[:48], flat[:48]]):
        with pytest.raises(ValueError, match="share memory"):
            binding.TokenPools(bad, 16)
    none = torch.zeros((0, 576), dtype=torch.uint8, device=DEV)
    binding.TokenPools([none, none], 16)
