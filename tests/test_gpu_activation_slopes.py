"""act'(pre) of dspark_linear_grad over the whole range of pre, by way of dbias of a single row
(its sums are not rounded to bf16).

Tolerances. With v the gate's argument and g = 1 / (1 + exp(-v)): exp by a power of two is off
by 2^-23 |v| (the argument's two roundings) and 2^-22 of itself, the division by 2^-22, so g by
d = (2^-23 |v| + 2^-21) of itself and 1 - g by d g + 2^-24. gelu's v and its slope carry another
2^-22 of their own size. Past 2^126 the division gives 0.
"""
import math

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def slopes(pre, act):
    N, K = pre.numel(), 8
    x, w = torch.zeros(1, K, device="cuda", dtype=BF16), torch.zeros(N, K, device="cuda", dtype=BF16)
    ws = torch.zeros(bn.workspace_bytes(bn.OP_LINEAR, 1, 1, N, K, bn.BF16), dtype=torch.uint8, device="cuda")
    out = torch.full((N,), 7.0, device="cuda")
    bn.linear_grad(x, w, torch.ones(1, N, device="cuda", dtype=BF16), ws, dbias=out, pre=pre.view(1, N), act=act)
    assert bn.read_status(ws) == (0, -1)
    return out.double()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_everywhere(cuda_ok, act):
    z = torch.cat([torch.linspace(0, 12, 400), torch.linspace(12, 210, 1000),
                   torch.tensor([1e3, 1e4, 1e10, 1e20, 1e30, 3.3e38, 0, 1e-30])]).to(BF16)
    z = torch.cat([z, -z]).cuda()
    got, z = slopes(z, act), z.double()
    if act == "relu":
        assert torch.equal(got, (z > 0).double())
        return
    c = 2 * math.sqrt(2 / math.pi)
    v = z if act == "silu" else c * (z + 0.044715 * z ** 3)
    dv = torch.ones_like(z) if act == "silu" else c * (1 + 3 * 0.044715 * z ** 2)
    g, h = torch.sigmoid(v), torch.sigmoid(-v)
    zd = torch.where(g * h > 0, (z * dv).abs(), torch.zeros_like(z))   # times g h, which is 0 far out
    want = g + torch.where(g * h > 0, z * dv * g * h, torch.zeros_like(z))
    own = 2.0 ** -22 if act == "gelu" else 0.0
    d = (2.0 ** -23 + own) * v.abs().clamp(max=200) + 2.0 ** -21
    near = z.abs().clamp(max=128)
    slope = near if act == "silu" else near * c * (1 + 3 * 0.044715 * near ** 2)
    tol = g * d * (1 + zd * h) + zd * g * (d * g + 2.0 ** -24).clamp(max=1) + (2.0 ** -21 + own) * (g + zd * g * h)
    tol = tol + 2.0 ** -125 * (1 + slope)
    err = (got - want).abs()
    worst = (err - tol).argmax()
    assert bool((err <= tol).all()), (z[worst].item(), got[worst].item(), want[worst].item(), tol[worst].item())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_at_infinity_and_nan(cuda_ok, act):
    got = slopes(torch.tensor([math.inf, -math.inf, math.nan, 0.0, 70, -70, 1e4, -1e4], device="cuda").to(BF16), act)
    assert got[0] == 1 and got[1] == 0 and got[2].isnan() and got[3] == 0.5
    assert got[4] == 1 and got[6] == 1 and got[7] == 0
    assert abs(got[5].item()) <= 3e-29      # exp(-70) (1 - 70) = -2.7e-29 for silu, nothing for gelu
