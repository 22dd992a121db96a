"""What attention over the block-scaled cache keeps of each weight, row by row and
weight by weight, against binary64.

Tolerances, derived. A weight times its block's value scale is rounded to
binary16, relative to a reference that the row's largest such product reaches to
2^5 or above: it is off by half a step, 2^-11 of itself, where it is a normal
number (2^-14, so 2^-19 of the largest), and by 2^-25 (2^-30 of the largest)
below. Logits are off by 2^-18 of their reach scale * sum |q| |K| (partial sums
in binary32, three products, a base-2 exponential of 2^-22), which moves weights
and lse by as much, and by scale * sum |K| * 2^-17 max |q| from q's two E4M3
parts: a part's smallest step is 2^-9, where the row's largest is 2^7 or above.
out is rounded once to bf16 (2^-8)."""
import math

import pytest
import torch

import kv8_reference as ref
from parity import DEV
from sparse_mla_attention_04_gb300 import binding

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def _cache(n, hk, D, bs, g, size):
    """One request's n positions in blocks in random order: K of deviation 1, V of deviation `size`."""
    nb = -(-n // bs)
    perm = torch.randperm(nb + 2, generator=g)[:nb]
    p = dict(table=perm.int()[None].contiguous())
    for name, dev in (("k", 1.0), ("v", size)):
        x = torch.randn((nb + 2, hk, bs, D), generator=g) * dev
        s = x.abs().amax((2, 3)) / 448
        p[name + "c"] = (x / s[:, :, None, None]).to(FP8).view(torch.uint8)
        p[name + "s"] = s
    return p, perm


def _expect(p, q, n, scale, window=0):
    """(want, z, tol of out, tol of lse) of the request's last rows."""
    T, H, D = q.shape
    hk = p["kc"].shape[1]
    pages = p["table"][0].long()
    kv = [ref.values(p[x + "c"], p[x + "s"])[pages].transpose(1, 2).reshape(-1, hk, D)[:n] for x in "kv"]
    vs = p["vs"].double()[pages].repeat_interleave(p["kc"].shape[2], 0)[:n]
    want, tol = (torch.zeros((T, H, D), dtype=torch.float64) for _ in range(2))
    z, ztol = (torch.zeros((T, H), dtype=torch.float64) for _ in range(2))
    for t in range(T):
        at = n - T + t
        lo = max(0, at - window + 1) if window else 0
        for h in range(H):
            K, V, s = kv[0][lo:at + 1, h * hk // H], kv[1][lo:at + 1, h * hk // H], vs[lo:at + 1, h * hk // H]
            x = q[t, h].double()
            logit = (K @ x) * scale
            z[t, h] = torch.logsumexp(logit, 0)
            w = torch.exp(logit - z[t, h])
            off = float(((K.abs() @ x.abs()).max() * 2.0 ** -18 + K.abs().sum(1).max() * x.abs().max() * 2.0 ** -17) * scale)
            part = w * s / (w * s).max()                       # of the largest product
            each = torch.where(part >= 2.0 ** -19, torch.full_like(part, 2.0 ** -11), (2.0 ** -30 / part).clamp(max=1.0))
            want[t, h] = w @ V
            tol[t, h] = want[t, h].abs() * 2.0 ** -8 + (w * (each + 2.0 ** -17 + 2 * off)) @ V.abs()
            ztol[t, h] = 2.0 ** -18 + off
    return want, z, tol, ztol


def _run(p, q, n, scale, window=0):
    d = {k: v.to(DEV) for k, v in p.items()}
    T = q.shape[0]
    out, lse = binding.smla_kv8_attn_fwd(q.to(DEV), d["kc"], d["vc"], d["ks"], d["vs"], d["table"],
                                         torch.tensor([n], dtype=torch.int32, device=DEV),
                                         torch.tensor([0, T], dtype=torch.int32, device=DEV), scale, max_query_len=T,
                                         window=window)
    return out.cpu().double(), lse.cpu().double()


def _check(p, q, n, scale, window=0):
    out, lse = _run(p, q, n, scale, window)
    want, z, tol, ztol = _expect(p, q, n, scale, window)
    worst = float(((out - want).abs() / tol.clamp(min=1e-300)).max())
    assert bool(((out - want).abs() <= tol).all()), worst
    assert bool(((lse - z).abs() <= ztol).all())


@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-6])
@pytest.mark.parametrize("place", [0, 2, -1])
@pytest.mark.parametrize("T,n,D,bs", [(1, 400, 128, 64), (1, 130, 64, 16), (4, 300, 128, 32), (33, 200, 64, 64),
                                      (40, 330, 128, 16), (140, 290, 128, 64), (130, 140, 64, 128)])
def test_a_block_whose_scale_says_nothing(T, n, D, bs, place, size):
    """All its values are 0 under a scale of 1, the others' scales are `size` / 100: its weights count in
    the denominator only, and the others' keep their bits."""
    g = torch.Generator().manual_seed(T + n + place)
    H, hk = 4, 2
    p, perm = _cache(n, hk, D, bs, g, size)
    b = int(perm[min(place, len(perm) - 1)])
    p["vc"][b], p["vs"][b] = 0, 1.0
    q = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    _check(p, q, n, 1 / math.sqrt(D))


@pytest.mark.parametrize("T", [1, 5, 40, 150])
def test_a_large_value_that_no_row_sees(T):
    """It sets its block's scale: the block's other values are 0, as the write gives them."""
    H, hk, D, bs, n, window = 4, 2, 128, 64, 300, 120
    g = torch.Generator().manual_seed(T)
    p, perm = _cache(n, hk, D, bs, g, 1e-4)
    first = max(0, n - T - window + 1)                         # of the positions that a row sees
    b = int(perm[first // bs])
    if first % bs:
        p["vc"][b], p["vs"][b] = 0, 2.0
        p["vc"][b, :, 0] = 0x7E
    q = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    _check(p, q, n, 1 / math.sqrt(D), window)


@pytest.mark.parametrize("T", [1, 40, 140])
def test_rows_of_zeros_written_by_the_append(T):
    """A prompt whose first tokens have no values (then blocks of them), written by the library."""
    H, hk, D, bs, n = 4, 2, 128, 64, 300
    g = torch.Generator().manual_seed(T)
    k = torch.randn((n, hk, D), generator=g).to(torch.bfloat16)
    v = (torch.randn((n, hk, D), generator=g) * 1e-5).to(torch.bfloat16)
    v[:70], v[128:200] = 0.0, 0.0
    cache = binding.new_kv8_cache(6, hk, bs, D)
    binding.smla_kv8_append(k.to(DEV), v.to(DEV), torch.arange(n, device=DEV), *cache)
    p = dict(zip(("kc", "vc", "ks", "vs"), (x.cpu() for x in cache)), table=torch.arange(5, dtype=torch.int32)[None])
    q = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    _check(p, q, n, 1 / math.sqrt(D))


@pytest.mark.parametrize("T", [1, 50])
def test_logits_that_grow_along_the_context(T):
    """The reference has to move again and again, by little and by much; values of two sizes."""
    H, hk, D, bs, n = 4, 2, 128, 32, 512
    for step in (0.3, 2.0, 40.0):
        g = torch.Generator().manual_seed(int(step * 10))
        p, perm = _cache(n, hk, D, bs, g, 1.0)
        p["vs"][perm[1::2]] *= 2.0 ** -12
        q = torch.ones((T, H, D), dtype=torch.bfloat16)
        kc = torch.full((n, D), 1.0).to(FP8).view(torch.uint8)
        for j, blk in enumerate(perm.tolist()):                # every key of a block alike, the next one's larger
            p["kc"][blk] = kc[:bs]
            p["ks"][blk] = (j + 1) * step * math.log(2.0) / math.sqrt(D)
        _check(p, q, n, 1 / math.sqrt(D))


@pytest.mark.parametrize("T", [1, 3, 50])
def test_large_and_tiny_queries_row_by_row(T):
    H, hk, D, bs, n = 8, 2, 64, 32, 90
    g = torch.Generator().manual_seed(T)
    p, _ = _cache(n, hk, D, bs, g, 1.0)
    q = torch.randn((T, H, D), generator=g)
    q[:, 1] *= 1e-30
    q[:, 2] = 0.0
    q[:, 3, 0] = 300.0
    q[:, 4] *= 30.0
    q[:, 5, 1:] *= 2.0 ** -12                                  # one element alone
    _check(p, q.to(torch.bfloat16), n, 1 / math.sqrt(D))


@pytest.mark.parametrize("T", [1, 7, 60, 200])
def test_a_context_without_values(T):
    """Blocks of zeros at the smallest scale: out 0, and the lse as ever. There the logits in log2 units have -60
    added and the denominator is about 2^66: a rounding of 2^-19 and a logarithm of 2^-22 times 66, times ln 2."""
    H, hk, D, bs, n = 4, 2, 64, 16, 200
    g = torch.Generator().manual_seed(T)
    k = torch.randn((n, hk, D), generator=g).to(torch.bfloat16)
    cache = binding.new_kv8_cache(14, hk, bs, D)
    binding.smla_kv8_append(k.to(DEV), torch.zeros_like(k).to(DEV), torch.arange(n, device=DEV), *cache)
    p = dict(zip(("kc", "vc", "ks", "vs"), (x.cpu() for x in cache)), table=torch.arange(14, dtype=torch.int32)[None])
    q = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    out, lse = _run(p, q, n, 0.125)
    assert bool((out == 0).all())
    p["table"] = p["table"][:, :-(-n // bs)]
    _, z, _, ztol = _expect(p, q, n, 0.125)
    assert bool(((lse - z).abs() <= ztol + 2.0 ** -16).all()), float((lse - z).abs().max())
