"""smla_qk_norm_rope where a group of lanes takes several rows one after another: heads of a token, or (weights for each head)
tokens of a head. That is so for calls of more than 2048 lanes to an SM, whatever the device: the number of tokens is made from
its SMs. Odd numbers of both, so that last groups are short; rows out of range, beyond binary32, infinite and NaN among a
group's. Tolerance: test_gpu_norm_rope.py. Rows of a group are computed as by themselves: the same bits as calls of few
tokens, which take a row to a group."""
import math

import pytest
import torch

from parity import DEV
from sparse_mla_attention_04_gb300 import binding
from test_gpu_norm_rope import TYPES, _close, _problem

pytestmark = pytest.mark.gpu


def _tokens(heads, D, dtype):
    """Just more than go by single rows, three more than a multiple of eight. A lane has at most 32 bytes of a row."""
    lanes = D * (4 if dtype == "f32" else 2) // 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = sms * 2048 // (heads * lanes) + 1
    return T + (3 - T) % 8


def _few(q, k, wq, wk, pos, cs, at, **kw):
    """The tokens `at` in a call of their own: too few for groups of rows."""
    return binding.smla_qk_norm_rope(q[at], None if k is None else k[at], wq, wk, pos[at].contiguous(), cs, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hk,D,rot,off", [(9, 4, 128, 128, 0), (3, 1, 256, 64, 192), (17, 2, 64, 32, 16), (1, 1, 128, 64, 0)])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("per_head", [False, True])
def test_rows_of_a_group(dtype, wide, H, Hk, D, rot, off, neox, per_head):
    T = _tokens(H + Hk, D, dtype)
    (q, k), (wq, wk), pos, cs = _problem(T, H, Hk, D, rot, dtype, T + D, wide, per_head)
    kw = dict(eps=1e-5, weight_offset=0.5, rot_offset=off, is_neox=neox)
    qo, ko = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, **kw)
    _close(qo, q, wq, 0.5, 1e-5, pos, cs, off, neox)
    _close(ko, k, wk, 0.5, 1e-5, pos, cs, off, neox)
    at = torch.arange(T - 21, T, device=DEV)
    qf, kf = _few(q, k, wq, wk, pos, cs, at, **kw)
    assert torch.equal(qf, qo[at]) and torch.equal(kf, ko[at])
    q2, k2 = q.clone(), k.clone()
    binding.smla_qk_norm_rope(q2, k2, wq, wk, pos, cs, q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert binding.smla_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("which", ["one row", "each head", "queries only", "keys only"])
@pytest.mark.parametrize("neox", [True, False])
def test_bad_positions_and_special_rows_among_a_group(dtype, which, neox):
    binding.smla_device_error(reset=True)
    H, Hk, D, rot = 9, 4, 128, 64
    T = _tokens(H + Hk, D, dtype)
    (q, k), (wq, wk), pos, cs = _problem(T, H, Hk, D, rot, dtype, 31, True, True)
    wq, wk = (w if which in ("each head", only) else w[0] for w, only in ((wq, "queries only"), (wk, "keys only")))
    large = dtype != "f16"                                         # (its squares stay within binary32)
    if large:
        q[1::5, 2] *= 1e30
        q[2::9, 8, 7] = 3.3e38
        k[3::8, 1, 5] = -3.3e38
    q[4::11, 0], k[6::10, 3] = 0.0, 0.0
    want = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, is_neox=neox)
    _close(want[0], q, wq, 0.0, 1e-6, pos, cs, 0, neox)
    _close(want[1], k, wk, 0.0, 1e-6, pos, cs, 0, neox)
    assert binding.smla_device_error() == 0
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[2::7] = bad[T - 1] = bad[8:16] = True                      # some of a group, its last, all of one
    at = torch.where(bad, torch.where(torch.arange(T, device=DEV) % 2 == 0, -1, 1 << 40), pos)
    q[7::13, 1, 5], q[9::17, 3, 100], k[5::9, 2, 0] = math.inf, math.nan, -math.inf
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    binding.smla_qk_norm_rope(q, k, wq, wk, at, cs, is_neox=neox, q_out=qo, k_out=ko)
    assert binding.smla_device_error(reset=True) == 4
    for x, o, w in ((q, qo, want[0]), (k, ko, want[1])):
        assert bool((o[bad] == 7.0).all())
        plain = x.isfinite().all(-1) & ~bad[:, None]
        assert torch.equal(o[plain], w[plain])
        one = x.isinf().any(-1) & ~bad[:, None]
        rest = torch.where(x.isinf(), torch.zeros_like(o), o)[one]
        pair = rest[..., :rot].isnan().sum(-1)                     # what the infinity is rotated with
        assert bool((pair <= 1).all()) and float(rest.nan_to_num(0.0).abs().max()) == 0
        assert bool(o[x.isinf() & one[..., None]].isnan().all())
        assert bool(o[x.isnan().any(-1) & ~bad[:, None]].isnan().all())
    few = torch.arange(8, 40, device=DEV)
    got = [torch.full_like(x[few], 7.0) for x in (q, k)]
    binding.smla_qk_norm_rope(q[few], k[few], wq, wk, at[few].contiguous(), cs, is_neox=neox, q_out=got[0], k_out=got[1])
    binding.smla_device_error(reset=True)
    for g, o in zip(got, (qo, ko)):
        assert torch.equal(torch.nan_to_num(g, nan=9.0), torch.nan_to_num(o[few], nan=9.0))


@pytest.mark.parametrize("per_head", [False, True])
def test_strided_groups_in_place_of_one_tensor(per_head):
    """Queries and keys as slices of one projection's rows, normed where they lie; queries alone."""
    H, Hk, D = 10, 3, 128
    T = _tokens(H + Hk, D, "bf16")
    (q, k), (wq, wk), pos, cs = _problem(T, H, Hk, D, 128, "bf16", 17, True, per_head)
    want = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs)
    room = torch.zeros((T, H + 2 * Hk, D), dtype=torch.bfloat16, device=DEV)
    room[:, :H], room[:, H:H + Hk], room[:, H + Hk:] = q, k, 3.0
    qs, ks = room[:, :H], room[:, H:H + Hk]
    binding.smla_qk_norm_rope(qs, ks, wq, wk, pos, cs, q_out=qs, k_out=ks)
    assert torch.equal(room[:, :H], want[0]) and torch.equal(room[:, H:H + Hk], want[1])
    assert bool((room[:, H + Hk:] == 3.0).all())
    T2 = _tokens(H, D, "bf16")
    q2 = torch.cat([q, q])[:T2].contiguous()
    p2 = torch.cat([pos, pos])[:T2].contiguous()
    alone, _ = binding.smla_qk_norm_rope(q2, None, wq, None, p2, cs)
    assert torch.equal(alone[:T], want[0]) and torch.equal(alone[T:], want[0][:T2 - T])
