"""smla_rope at the largest number of tokens."""
import pytest
import torch

from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu


def test_two_to_the_31_tokens_less_one():
    """One head of two columns each, in place: 26 GB."""
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    cs = binding.smla_rope_cos_sin_cache(4, 2)
    q = torch.zeros((T, 1, 2), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    pos = torch.zeros(T, dtype=torch.int64, device=DEV)
    for t in (0, 1, 2 ** 30, T - 2, T - 1):
        pos[t] = 3
    binding.smla_rope(q, None, pos, cs, q_out=q)
    want = cs[3].to(torch.bfloat16)
    for t in (0, 1, 2 ** 30, T - 2, T - 1):
        assert torch.equal(q[t, 0], want)
    assert q[5:T - 5:1000003, 0].tolist() == [[1.0, 0.0]] * len(range(5, T - 5, 1000003))
    assert binding.smla_device_error(reset=True) == 0
    del q, pos
    torch.cuda.empty_cache()
