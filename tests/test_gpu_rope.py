"""smla_rope_cos_sin_cache and smla_rope against their formulas in 64 bits.

Table: the angle is exact to 2^-63 of a turn, its conversion to binary32 is off
by at most 2^-24 relative (up to pi 2^-24 < 2^-22 in radians), sincospif by 2
ulp (2^-23 of 1) and the factor's product by 2^-24: under 2^-21 times the
factor. The frequencies are rounded to binary64 (2^-53 relative, a few
roundings), which at position p moves the angle by about p 2^-51 f.
Rotation: two products and their sum are rounded in binary32 (each 2^-24 of
|a| + |b|), then once to the type (half a step)."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,base,scaling,factor,orig,fast,slow", [
    (64, 1e4, "none", 1.0, 0, 32.0, 1.0), (2, 1e4, "none", 1.0, 0, 32.0, 1.0), (256, 5e5, "none", 1.0, 0, 32.0, 1.0),
    (64, 1e4, "linear", 4.0, 0, 32.0, 1.0), (128, 1e4, "ntk", 8.0, 0, 32.0, 1.0), (4, 1e4, "ntk", 2.0, 0, 32.0, 1.0),
    (64, 1e4, "yarn", 40.0, 4096, 32.0, 1.0), (96, 1e6, "yarn", 4.0, 32768, 16.0, 2.0),
    (6, 1e4, "yarn", 2.0, 7, 32.0, 1.0)])
@pytest.mark.parametrize("first,n", [(0, 1000), (1, 1), (1048575, 257), ((1 << 31) - 300, 300)])
def test_table(rot, base, scaling, factor, orig, fast, slow, first, n):
    got = binding.smla_rope_cos_sin_cache(n, rot, base=base, scaling=scaling, factor=factor,
                                          original_max_position=orig, beta_fast=fast, beta_slow=slow,
                                          first_position=first).cpu().numpy().astype(np.float64)
    f, m = ref.frequencies(rot, base, scaling, factor, orig, fast, slow)
    # the angle modulo a turn in extended steps: p f in two parts keeps the product's rounding out
    p = np.arange(first, first + n, dtype=np.float64)[:, None]
    turns = f / (2 * np.pi)
    hi = np.round(turns * 2.0 ** 21) / 2.0 ** 21         # 21 bits: p * hi is exact in binary64
    ang = (np.mod(p * hi, 1.0) + p * (turns - hi)) * 2 * np.pi
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1) * m
    tol = m * (2.0 ** -21 + (first + n) * 2.0 ** -50)
    assert np.abs(got - want).max() <= tol


def test_table_attention_factor_and_out():
    out = torch.empty((50, 64), device=DEV)
    t = binding.smla_rope_cos_sin_cache(50, 64, attention_factor=1.25, out=out)
    assert t.data_ptr() == out.data_ptr()
    plain = binding.smla_rope_cos_sin_cache(50, 64)
    assert torch.equal(t, plain * 1.25)
    assert binding.smla_rope_cos_sin_cache(0, 64).shape == (0, 64)


def _ref(x, pos, cs, off, neox, inverse):
    rot = cs.shape[1]
    n = rot // 2
    y = x.double().clone()
    row = cs.double()[pos]
    c, s = row[:, None, :n], row[:, None, n:]
    if inverse:
        s = -s
    part = y[..., off:off + rot].clone()
    a, b = (part[..., :n], part[..., n:]) if neox else (part[..., 0::2], part[..., 1::2])
    u, w = a * c - b * s, b * c + a * s
    y[..., off:off + rot] = torch.cat([u, w], -1) if neox else torch.stack([u, w], -1).flatten(-2)
    size = torch.zeros_like(y)
    t = a.abs() + b.abs()
    size[..., off:off + rot] = torch.cat([t, t], -1) if neox else torch.stack([t, t], -1).flatten(-2)
    return y, size


def _close(got, want, size, dtype, m):
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    tol = want.abs() * half + size * m * 3 * 2.0 ** -24 * (1 + half) + tiny
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T,H,Hk,D,rot,off", [
    (1, 1, 1, 64, 64, 0), (3, 16, 2, 128, 128, 0), (64, 128, 1, 192, 64, 128), (7, 5, 3, 96, 32, 64),
    (130, 4, 0, 576, 64, 512), (9, 3, 1, 65, 32, 33), (5, 2, 2, 80, 6, 10), (2, 300, 9, 256, 256, 0),
    (33, 7, 1, 128, 96, 16), (4, 2, 1, 2000, 2, 1998)])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rotation(T, H, Hk, D, rot, off, neox, dtype):
    g = torch.Generator().manual_seed(T * 1000 + D)
    q = torch.randn((T, H, D), generator=g).to(dtype)
    k = torch.randn((T, Hk, D), generator=g).to(dtype) if Hk else None
    pos = torch.randint(0, 500, (T,), generator=g)
    cs = binding.smla_rope_cos_sin_cache(500, rot, scaling="yarn", factor=4.0, original_max_position=128)
    m = 0.1 * np.log(4.0) + 1
    for inverse in (False, True):
        qo, ko = binding.smla_rope(q.to(DEV), None if k is None else k.to(DEV), pos.to(DEV), cs, rot_offset=off,
                                   is_neox=neox, inverse=inverse)
        for x, o in ((q, qo), (k, ko)):
            if x is None:
                assert o is None
                continue
            want, size = _ref(x, pos, cs.cpu(), off, neox, inverse)
            _close(o, want, size, dtype, m)
            assert torch.equal(o.cpu()[..., :off], x[..., :off]) and torch.equal(o.cpu()[..., off + rot:], x[..., off + rot:])


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("shift", [0, 1])
def test_in_place_strided_and_misaligned(neox, shift):
    """Rows inside wider rows (16-byte aligned or not), rotated in place, neighbours left alone."""
    T, H, D, rot = 11, 4, 128, 64
    g = torch.Generator().manual_seed(5)
    wide = torch.randn((T, H, 200), generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 90, (T,), generator=g).to(DEV)
    cs = binding.smla_rope_cos_sin_cache(90, rot)
    before = wide.clone()
    q = wide[:, :, 8 + shift:8 + shift + D]
    want, _ = binding.smla_rope(q.contiguous(), None, pos, cs, rot_offset=32, is_neox=neox)
    got, none = binding.smla_rope(q, None, pos, cs, rot_offset=32, is_neox=neox, q_out=q)
    assert none is None and got.data_ptr() == q.data_ptr()
    assert torch.equal(q, want)
    assert torch.equal(wide[:, :, :8 + shift], before[:, :, :8 + shift])
    assert torch.equal(wide[:, :, 8 + shift + D:], before[:, :, 8 + shift + D:])


def test_bad_positions_write_nothing():
    binding.smla_device_error(reset=True)
    q = torch.randn((4, 2, 64), device=DEV).to(torch.bfloat16)
    cs = binding.smla_rope_cos_sin_cache(10, 64)
    out = torch.full_like(q, 7.0)
    pos = torch.tensor([0, 10, -1, 9], device=DEV)
    binding.smla_rope(q, None, pos, cs, q_out=out)
    assert binding.smla_device_error(reset=True) == 4
    assert bool((out[1:3] == 7.0).all()) and torch.equal(out[0], q[0])


def test_inverse_is_the_gradient():
    """d/dx sum(w . R x) = R^T w: the inverse rotation of w, against differences."""
    T, H, D = 3, 2, 32
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn((T, H, D), generator=g).to(DEV) for _ in range(2))
    pos = torch.tensor([1, 50, 99], device=DEV)
    cs = binding.smla_rope_cos_sin_cache(100, 16, scaling="yarn", factor=8.0, original_max_position=32)
    for neox in (True, False):
        grad, _ = binding.smla_rope(w, None, pos, cs, rot_offset=8, is_neox=neox, inverse=True)
        d = torch.randn((T, H, D), generator=g).to(DEV)
        up, _ = binding.smla_rope(x + d, None, pos, cs, rot_offset=8, is_neox=neox)
        down, _ = binding.smla_rope(x - d, None, pos, cs, rot_offset=8, is_neox=neox)
        # linear: the difference quotient is exact but for binary32 roundings of values below ~8
        lhs = float(((up.double() - down.double()) * w.double()).sum() / 2)
        rhs = float((grad.double() * d.double()).sum())
        assert abs(lhs - rhs) <= x.numel() * 8 * 8 * 2.0 ** -22


def test_matches_the_fused_producer():
    """smla_rope on the 64 rope columns gives the fused producer's bits, over the new table."""
    T, H, P = 9, 16, 300
    ql, qp, kc, kp, pos, _, _ = inputs.producer_inputs(T, H, 3, P)
    cs = binding.smla_rope_cos_sin_cache(P, 64, scaling="linear", factor=2.0)
    pool = torch.zeros((64, 576), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(T, device=DEV)
    for neox in (True, False):
        q_out = binding.smla_fused_qk_rope_cache(ql.to(DEV), qp.to(DEV), kc.to(DEV), kp.to(DEV), pos.to(DEV), cs,
                                                 slots, pool, is_neox=neox)
        full = torch.cat([ql, qp], -1).to(DEV)
        kfull = torch.cat([kc, kp], -1)[:, None].contiguous().to(DEV)
        qo, ko = binding.smla_rope(full, kfull, pos.to(DEV), cs, rot_offset=512, is_neox=neox)
        assert torch.equal(qo, q_out) and torch.equal(ko[:, 0], pool[:T])
