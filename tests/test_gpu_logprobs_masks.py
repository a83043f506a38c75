"""Scores of rows that hold finite masks of any size, maxima far from zero, and very small
temperatures, against the definition in 64 bits.

Tolerances are those of test_gpu_logprobs.py: every difference from the row's maximum is taken
before it is scaled or is the exact result of a fused product, so they do not grow with the
mask, and with the maximum only where lse itself does.

Gradients: below |lse| = 4096, lp = x - lse is off by lse's own error (e and 2^-23 |lse|), by
2^-24 |x| of 1 / temp's rounding with |x| <= |lse| + |lp|, and by 2^-24 of itself. From there
on the sum is formed again: lp = (l - m) / temp - ln s is off by e of ln s and less than 2^-21
of itself. Both enter as p times that error; p below 2^-126 is 0.
"""
import math

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn
from test_gpu_logprobs import BF16, F32, compare, grad, rows, score

pytestmark = pytest.mark.gpu

MASKS = [-1e5, -1e9, -2e9, -3e9, -1e10, -1e12, -1e15, -1e20, -1e30, -1e36]


def patterns(logits, mask):
    """Rows of every kind of masking: all but 1, 10 and 300 entries, a prefix, a suffix, every
    other entry, a whole row (uniform), one allowed entry at the end."""
    V = logits.shape[-1]
    logits[0, 0, 1:] = mask
    logits[1, 0, 10:] = mask
    logits[2, 0, 300:] = mask
    logits[3, 0, :V - 20] = mask
    logits[4, 0, 20:] = mask
    logits[5, 0, ::2] = mask
    logits[6, 0, :] = mask
    logits[7, 0, :V - 1] = mask
    return logits


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("V,n", [(2056, 0), (5000, 8), (40000, 20)])
def test_finite_masks(cuda_ok, dtype, mask, V, n):
    logits, tok, _ = rows(8, 1, V, dtype, seed=21)
    logits = patterns(logits, mask)
    tok[:4] = torch.tensor([0, 3, 17, V - 5], device="cuda", dtype=torch.int32)[:, None]
    for temp in ([0.6] * 8, [1.0] * 8, [0.8, 1.7, 0.0, 0.3, 1.0, 2.0, 0.5, 1.0]):
        temp = torch.tensor(temp, device="cuda")
        out, status = score(logits, tok, temp, n)
        assert status == (0, -1)
        compare(out, logits, tok, temp, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_finite_masks_with_a_cta_per_row(cuda_ok, dtype):
    """As many rows as leave one CTA to each, a different mask in every group of eight."""
    V, n = 2056, 8
    few, _, _ = rows(8, 1, V, dtype, seed=22)
    logits = torch.cat([patterns(few.clone(), m) for m in MASKS] * 8)
    B = logits.shape[0]
    tok = (torch.arange(B, device="cuda", dtype=torch.int32) * 37 % V)[:, None]
    temp = torch.tensor([0.6, 1.0, 1.7, 0.0], device="cuda")[torch.arange(B, device="cuda") // 8 % 4]
    out, status = score(logits, tok, temp, n)
    assert status == (0, -1)
    compare(out, logits, tok, temp, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1000, 40000])
@pytest.mark.parametrize("size", [1e3, 1e6, 3e6, 5e6, 1e7, 1e10, 1e20, 1e35])
def test_maxima_far_from_zero(cuda_ok, dtype, V, size):
    """Rows near +size and -size, rows that reach from one to the other, and rows of which
    every entry but one or a few is smaller by a size."""
    logits, tok, _ = rows(6, 1, V, dtype, seed=23)
    logits[0] = (logits[0].float() + size).to(dtype)
    logits[1] = (logits[1].float() - size).to(dtype)
    logits[2] = torch.linspace(-size, size, V, device="cuda").to(dtype)
    logits[3] = (logits[3].float() * size / 4).to(dtype)
    logits[4, 0, 7] = size
    logits[5] = (logits[5].float() - size).to(dtype)
    logits[5, 0, V - 3:] = -size / 2
    temp = torch.tensor([1.0, 1.0, 0.7, 1.0, 2.0, 1.0], device="cuda")
    for t in (None, temp):
        out, status = score(logits, tok, t, 8)
        assert status == (0, -1)
        compare(out, logits, tok, t, 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,n", [(1000, 5), (40000, 0)])
@pytest.mark.parametrize("temp", [1e-3, 1e-5, 4e-6, 1e-6, 1e-8, 1e-9, 1e-12, 1e-20, 1e-30])
def test_small_temperatures(cuda_ok, dtype, V, n, temp):
    logits, tok, _ = rows(6, 1, V, dtype, seed=24)
    logits[1] *= 10
    logits[2, 0, 40:] = -1e4                 # few allowed
    logits[3] -= 30
    logits[4] = 3.5                          # uniform
    logits[5, 0, 11] = logits[5, 0, V - 2] = 40.0  # two certain tokens
    tok[5] = 11
    t = torch.full((6,), temp, device="cuda")
    out, status = score(logits, tok, t, n)
    assert status == (0, -1)
    compare(out, logits, tok, t, n)
    assert abs(out["logp"][5, 0].item() + math.log(2)) < 1e-6


def check_gradient(logits, tok, temp, with_entropy, in_place=False):
    V = logits.shape[-1]
    out, status = score(logits, tok, temp)
    assert status == (0, -1)
    g = torch.Generator(device="cuda").manual_seed(2)
    gl = torch.randn(tok.shape, generator=g, device="cuda")
    gh = torch.randn(tok.shape, generator=g, device="cuda") if with_entropy else None
    live = logits.clone()
    d, status = grad(live, tok, temp, out["lse"], out["entropy"], gl, gh, out=live if in_place else None)
    assert status == (0, -1)
    one = torch.ones(tok.shape[0], device="cuda")
    tau = one if temp is None else torch.where(temp > 0, temp, one)
    tau = tau.double()[:, None, None]
    x = logits.double() / tau
    top = x.amax(-1, keepdim=True)
    ln_s = torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    lp = x - top - ln_s
    p = lp.exp()
    lpf = torch.where(p > 0, lp, torch.zeros_like(lp))   # p ln p is 0 where p is
    ent = -(p * lpf).sum(-1, keepdim=True)
    a = gl.double()[..., None]
    h = gh.double()[..., None] if with_entropy else torch.zeros_like(a)
    want = -p * (a + h * (lpf + ent))
    want = want.scatter_add(-1, tok.long()[..., None], a) / tau
    e = 2.0 ** -24 * (V / 256 + 16) + 2.0 ** -22 + 2.0 ** -23 * 30
    lse = (top + ln_s).abs()
    rel = torch.where(out["lse"].abs()[..., None] < 4096, 2.0 ** -22 * lse, 0 * lse) + e + 2.0 ** -21 + 2.0 ** -21 * lpf.abs()
    a, h = a.abs(), h.abs()
    e_h = e * (2 + 2 * math.log(V)) + 2.0 ** -22 * ent
    tol = torch.finfo(logits.dtype).eps / 2 * want.abs() + 2.0 ** -21 * want.abs()
    tol = tol + p * (a + h * (1 + lpf.abs() + ent)) / tau * (rel + 2.0 ** -21) + h * p * e_h / tau
    tol = tol + 2.0 ** -126 * (a + h * (200 + ent)) / tau + 1e-38
    tol = tol.scatter_add(-1, tok.long()[..., None], 2.0 ** -22 * a / tau)  # a difference of two terms of size a
    err = (d.double() - want).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()


@pytest.mark.parametrize("with_entropy", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [1e-3, 1e-5, 1e-6, 1e-9, 1e-30])
@pytest.mark.parametrize("V", [1000, 40000])
def test_gradient_at_small_temperatures(cuda_ok, dtype, temp, V, with_entropy):
    logits, tok, _ = rows(7, 1, V, dtype, seed=25)
    logits[1] *= 10
    logits[2, 0, 40:] = -1e4
    logits[3] -= 30
    logits[4] = 3.5                          # uniform
    logits[5, 0, 11] = logits[5, 0, V - 2] = 40.0
    logits[6] *= temp                        # an ordinary row at this temperature
    tok[5] = 11
    check_gradient(logits, tok, torch.full((7,), temp, device="cuda"), with_entropy)


@pytest.mark.parametrize("with_entropy", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e3, 4e3, 5e3, 1e6, 1e10, 1e30])
def test_gradient_of_far_maxima_and_masks(cuda_ok, dtype, size, with_entropy):
    V = 5000
    logits, tok, _ = rows(7, 1, V, dtype, seed=26)
    logits[0] = (logits[0].float() + size).to(dtype)
    logits[1] = (logits[1].float() - size).to(dtype)
    logits[2] = torch.linspace(-size, size, V, device="cuda").to(dtype)
    logits[3, 0, 10:] = -size                # few allowed
    logits[4] = -size                        # uniform
    logits[5, 0, 7] = size
    logits[6] = -math.inf
    logits[6, 0, 100:110] = -size
    tok[6], tok[5] = 104, 7
    temp = torch.tensor([1.0, 0.6, 1.0, 0.8, 1.0, 2.0, 1.0], device="cuda")
    for in_place in (False, True):
        check_gradient(logits, tok, temp, with_entropy, in_place)
    check_gradient(logits, tok, None, with_entropy)


def test_gradient_of_a_far_row_that_is_not_finite(cuda_ok):
    """The logits have changed since lse was made: zeros and a status, as for other rows in error."""
    logits, tok, _ = rows(3, 2, 2000, BF16, seed=27)
    logits += 1e6
    out, _ = score(logits, tok)
    ones = torch.ones(3, 2, device="cuda")
    for bad in (math.nan, math.inf):
        now = logits.clone()
        now[1, 1, 1234] = bad
        d, status = grad(now, tok, None, out["lse"], out["entropy"], ones, ones)
        assert status == (bn.STATUS_BAD_ROW, 1)
        assert bool((d[1, 1] == 0).all()) and bool(torch.isfinite(d.float()).all()) and bool((d[1, 0] != 0).any())
