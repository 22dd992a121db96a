"""smla_qk_norm_rope against its formula in 64 bits.

Tolerance: the sum of squares adds at most D / 32 + 16 terms one after another in a lane, then five levels: its rounding is
below (D / 32 + 22) 2^-24 of it, half of that of the root; the mean, the root, the weight's sum and three products round once
each: (D / 64 + 20) 2^-24 of a value. The rotation's two products and their sum add 2 * 2^-24 of |a cos| + |b sin|. Together
below 2^-18 of the pair's size for D <= 1024; then half a step of the type. Below a type's normals its steps stay those
of the smallest normals, whatever the value: half of one is 2^-25 in fp16, 2^-134 in bf16 and 2^-150 in binary32, where a value
takes at most five such roundings (two products, then two more and a sum) that later factors below 2 may double: 2^-146."""
import math

import pytest
import torch

import branch_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _table(P, rot, g):
    a = torch.rand((P, rot // 2), generator=g, dtype=torch.float64) * 6.4
    return torch.cat([a.cos(), a.sin()], 1).float()


def _close(got, x, w, plus, eps, pos, cs, off, neox):
    want, size = ref.norm_rope(x.cpu(), None if w is None else w.cpu(), plus, eps, pos.cpu(), cs.cpu(), off, neox)
    least = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 0.0}[x.dtype] + 2.0 ** -146
    tol = size * 2.0 ** -18 + want.abs() * torch.finfo(x.dtype).eps / 2 + least
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())


def _problem(T, H, Hk, D, rot, dtype, seed, wide=False, per_head=False, P=200):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    x = [(torch.randn((T, h, D), generator=g) * torch.exp(torch.randn((T, h, 1), generator=g))).to(dt).to(DEV) for h in (H, Hk)]
    w = [(1 + 0.3 * torch.randn((h, D) if per_head else (D,), generator=g)).to(torch.float32 if wide else dt).to(DEV) for h in (H, Hk)]
    pos = torch.randint(0, P, (T,), generator=g).to(DEV)
    return x, w, pos, _table(P, rot, g).to(DEV)


@pytest.mark.parametrize("T,H,Hk,D,rot,off", [
    (1, 1, 1, 64, 64, 0), (1, 32, 8, 128, 128, 0), (3, 5, 1, 128, 64, 64), (700, 32, 8, 128, 128, 0), (513, 7, 3, 96, 32, 0),
    (64, 128, 1, 192, 64, 128), (33, 9, 2, 256, 256, 0), (5, 3, 2, 576, 64, 512), (17, 4, 4, 80, 80, 0), (9, 2, 1, 512, 128, 0),
    (40, 3, 1, 72, 16, 24), (11, 2, 1, 65, 22, 7), (6, 1, 1, 2, 2, 0), (4, 2, 1, 1000, 100, 300), (3, 130, 17, 64, 32, 16)])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype,wide,per_head,plus", [("bf16", False, False, 0.0), ("bf16", True, True, 1.0), ("f16", False, True, 0.0),
                                                      ("f16", True, False, 1.0), ("f32", True, False, -0.5),
                                                      ("f32", True, True, 0.0)])
def test_values(T, H, Hk, D, rot, off, neox, dtype, wide, per_head, plus):
    (q, k), (wq, wk), pos, cs = _problem(T, H, Hk, D, rot, dtype, D + T, wide, per_head)
    qo, ko = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, eps=1e-5, weight_offset=plus, rot_offset=off, is_neox=neox)
    _close(qo, q, wq, plus, 1e-5, pos, cs, off, neox)
    _close(ko, k, wk, plus, 1e-5, pos, cs, off, neox)
    assert binding.smla_device_error() == 0


@pytest.mark.parametrize("D,rot", [(128, 64), (72, 20)])
def test_strides_in_place_and_q_alone(D, rot):
    T, H, Hk = 37, 6, 2
    (q, k), (wq, wk), pos, cs = _problem(T, H, Hk, D, rot, "bf16", 5)
    wide = torch.zeros((T, H + Hk, 2 * D), dtype=torch.bfloat16, device=DEV)
    wide[:, :H, :D], wide[:, H:, D:] = q, k
    qs, ks = wide[:, :H, :D], wide[:, H:, D:]
    want = binding.smla_qk_norm_rope(q, k, wq, None, pos, cs)
    got = binding.smla_qk_norm_rope(qs, ks, wq, None, pos, cs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _close(want[1], k, None, 0.0, 1e-6, pos, cs, 0, True)         # no weights: factors of 1
    alone, none = binding.smla_qk_norm_rope(q, None, wq, None, pos, cs)
    assert none is None and torch.equal(alone, want[0])
    heads = q.transpose(0, 1).contiguous().transpose(0, 1)        # heads before tokens
    assert torch.equal(binding.smla_qk_norm_rope(heads, None, wq, None, pos, cs)[0], want[0])
    binding.smla_qk_norm_rope(qs, ks, wq, None, pos, cs, q_out=qs, k_out=ks)
    assert torch.equal(wide[:, :H, :D], want[0]) and torch.equal(wide[:, H:, D:], want[1])
    assert float(wide[:, :H, D:].abs().max()) == 0                # what lies between is left alone
    odd = torch.zeros(T * H * D + 1, dtype=torch.bfloat16, device=DEV)[1:].view(T, H, D)
    odd.copy_(q)                                                  # a row that is not 16-byte aligned
    _close(binding.smla_qk_norm_rope(odd, None, wq, None, pos, cs, q_out=odd)[0], q, wq, 0.0, 1e-6, pos, cs, 0, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(128, 64), (70, 20)])
def test_large_small_and_special_rows(dtype, D, rot):
    """Squares beyond binary32, rows of zeros, infinities and NaN; what stands beside them is not touched."""
    T, H = 9, 5
    (q, _), (wq, _), pos, cs = _problem(T, H, 1, D, rot, dtype, 7)
    q[0, 0] *= 1e30
    q[0, 1, 3] = 3.3e38
    q[1, 2] = 3.3e38
    q[2] = 0.0
    q[3] *= 1e-30
    got = binding.smla_qk_norm_rope(q, None, wq, None, pos, cs)[0]
    _close(got, q, wq, 0.0, 1e-6, pos, cs, 0, True)
    assert float(got[2].abs().max()) == 0
    clean = got.clone()
    q[4, 1, D - 1] = math.inf
    q[5, 0, 2] = math.nan
    got = binding.smla_qk_norm_rope(q, None, wq, None, pos, cs)[0]
    assert bool(got[5, 0].isnan().all())
    assert bool(got[4, 1, D - 1].isnan()) and float(got[4, 1, :D - 1].abs().max()) == 0
    same = torch.ones((T, H), dtype=torch.bool, device=DEV)
    same[4, 1] = same[5, 0] = False
    assert torch.equal(got[same], clean[same])


@pytest.mark.parametrize("D", [128, 70])
def test_positions_out_of_range(D):
    binding.smla_device_error(reset=True)
    (q, k), (wq, wk), pos, cs = _problem(6, 3, 2, D, 20 if D == 70 else 64, "bf16", 9)
    pos[1], pos[4] = -1, 200
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, q_out=qo, k_out=ko)
    assert binding.smla_device_error(reset=True) == 4
    for x, o, w in ((q, qo, wq), (k, ko, wk)):
        assert bool((o[[1, 4]] == 7.0).all())
        keep = [0, 2, 3, 5]
        _close(o[keep], x[keep], w, 0.0, 1e-6, pos[keep], cs, 0, True)


@pytest.mark.parametrize("T", [3, 2000])
def test_weights_for_each_head_beside_one_row(T):
    """Queries with weights for each head, keys with one row for all, or none; bad positions among eight tokens of a head."""
    binding.smla_device_error(reset=True)
    (q, k), (wq, _), pos, cs = _problem(T, 9, 4, 128, 64, "bf16", 21, True, True)
    wk = torch.rand(128, device=DEV) + 0.5
    for w in (wk, None):
        qo, ko = binding.smla_qk_norm_rope(q, k, wq, w, pos, cs, weight_offset=0.5)
        _close(qo, q, wq, 0.5, 1e-6, pos, cs, 0, True)
        _close(ko, k, w, 0.5, 1e-6, pos, cs, 0, True)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[1::7] = True
    at = torch.where(bad, 1 << 40, pos)
    q2, k2 = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    binding.smla_qk_norm_rope(q, k, wq, None, at, cs, weight_offset=0.5, q_out=q2, k_out=k2)
    assert binding.smla_device_error(reset=True) == 4
    for x, y in ((q2, qo), (k2, ko)):
        assert torch.equal(x[~bad], y[~bad]) and bool((x[bad] == 7.0).all())


def test_refusals_graph_and_stream():
    (q, k), (wq, wk), pos, cs = _problem(20, 8, 2, 128, 128, "bf16", 11)
    with pytest.raises(ValueError):
        binding.smla_qk_norm_rope(q, k, wq[:64], wk, pos, cs)
    with pytest.raises(ValueError):
        binding.smla_qk_norm_rope(q, k, wq.expand(3, 128), wk, pos, cs)
    with pytest.raises(TypeError):
        binding.smla_qk_norm_rope(q, k, wq, wk.float(), pos, cs)
    with pytest.raises(TypeError):
        binding.smla_qk_norm_rope(q, k, wq.half(), wk.half(), pos, cs)
    with pytest.raises(ValueError):
        binding.smla_qk_norm_rope(q, None, wq, wk, pos, cs)
    with pytest.raises(binding.SmlaError):
        binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, eps=0.0)
    with pytest.raises(binding.SmlaError):
        binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, rot_offset=8)
    want = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs)
    assert torch.equal(binding.smla_qk_norm_rope(q, k, wq.expand(8, 128), wk, pos, cs)[0], want[0])   # one row for all heads
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.smla_qk_norm_rope(q, k, wq, wk, pos, cs)
    q.normal_()
    pos.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    _close(got[0], q, wq, 0.0, 1e-6, pos, cs, 0, True)
    empty = binding.smla_qk_norm_rope(q[:0], k[:0], wq, wk, pos[:0], cs)
    assert empty[0].shape == (0, 8, 128)


def test_rows_past_32_bits():
    """Rows whose offsets pass 2^31 elements."""
    H, D, st = 3, 128, (1 << 30) + 128
    room = torch.empty(2 * st + H * D, dtype=torch.bfloat16, device=DEV)
    q = room.as_strided((3, H, D), (st, D, 1))
    (small, _), (wq, _), pos, cs = _problem(3, H, 1, D, 64, "bf16", 13)
    q.copy_(small)
    want = binding.smla_qk_norm_rope(small, None, wq, None, pos, cs)[0]
    binding.smla_qk_norm_rope(q, None, wq, None, pos, cs, q_out=q)
    assert torch.equal(q, want)
