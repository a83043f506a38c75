"""Scores of rows that hold finite masks of any size, maxima far from zero, and very small
temperatures, against the definition in 64 bits.

Tolerances are those of test_gpu_logprobs.py: every difference from the row's maximum is taken
before it is scaled or is the exact result of a fused product, so they do not grow with the
mask, and with the maximum only where lse itself does.
"""
import math

import pytest
import torch

from test_gpu_logprobs import BF16, F32, compare, rows, score

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
