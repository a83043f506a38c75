"""dspark_residual_norm and its gradient against the definition in 64 bits.

Tolerances. sum v^2 of H terms: a thread adds at most 64 of them and about 10 joining
steps follow, each off by at most 2^-24 (fp32, relative, all terms positive), the
squares by 2^-24; v itself by 2^-24. rstd halves that and adds a division and a root:
below e = 2^-24 * 60 in all. y adds two products and the rounding to its type (half a
step). e4m3: half a step is 2^-4 of the value, 2^-10 of the scale below its normal
range; the scale carries e.
"""
import math

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
E = 2.0 ** -24 * 60


def half(dtype):
    return torch.finfo(dtype).eps / 2


def inputs(M, H, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (mk(M, H) * 3).to(dtype), mk(M, H).to(dtype), (1 + 0.3 * mk(H)).to(dtype)


def workspace(M, H):
    return torch.zeros(bn.workspace_bytes(bn.OP_NORM, M, 0, H, 0, 0), dtype=torch.uint8, device="cuda")


def norm(x, delta, weight, eps=1e-6, e4m3=False, sum_out=None, stream=None):
    M, H = x.shape
    ws = workspace(M, H)
    out = dict(sum=torch.full_like(x, 7) if sum_out is None else sum_out, rstd=torch.full((M,), 7.0, device="cuda"),
               y=torch.empty(M, H, device="cuda", dtype=E4M3 if e4m3 else x.dtype),
               y_scale=torch.full((M,), 7.0, device="cuda") if e4m3 else None)
    y = out["y"]
    bn.residual_norm(x, delta, weight, eps, y, ws, **{k: v for k, v in out.items() if k != "y"}, stream=stream)
    torch.cuda.synchronize()
    return out, bn.read_status(ws)


def check(out, x, delta, weight, eps=1e-6):
    v = x.double() + (delta.double() if delta is not None else 0)
    rstd = 1 / torch.sqrt((v * v).mean(1) + eps)
    y = v * rstd[:, None] * weight.double()
    assert bool(((out["sum"].double() - v).abs() <= half(x.dtype) * v.abs() * 1.0001 + 2.0 ** -24 * v.abs()).all())
    assert bool(((out["rstd"].double() - rstd).abs() <= E * rstd).all())
    if out["y_scale"] is None:
        err, tol = (out["y"].double() - y).abs(), (half(x.dtype) + 2 * E) * y.abs()
    else:
        scale = torch.clamp(y.abs().amax(1) / 448, min=2.0 ** -126)
        assert bool(((out["y_scale"].double() - scale).abs() <= 2 * E * scale).all())
        s = out["y_scale"].double()[:, None]
        err, tol = (out["y"].double() * s - y).abs(), (2.0 ** -4 + 4 * E) * y.abs() + 2.0 ** -10 * s
    assert bool((err <= tol).all()), (err - tol).max().item()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,H", [(1, 8), (1, 4096), (3, 40), (5, 264), (130, 1032), (2, 7168), (3, 8200), (2, 16384),
                                 (700, 2048)])
def test_norm_matches(cuda_ok, dtype, M, H, e4m3):
    x, delta, weight = inputs(M, H, dtype, seed=H)
    out, status = norm(x, delta, weight, e4m3=e4m3)
    assert status == (0, -1)
    check(out, x, delta, weight)


@pytest.mark.parametrize("e4m3", [False, True])
def test_without_residual_and_outputs_left_out(cuda_ok, e4m3):
    x, delta, weight = inputs(9, 512, BF16, seed=1)
    out, _ = norm(x, None, weight, e4m3=e4m3)
    check(out, x, None, weight)
    y = torch.empty_like(out["y"])
    scale = torch.empty(9, device="cuda") if e4m3 else None
    bn.residual_norm(x, None, weight, 1e-6, y, workspace(9, 512), y_scale=scale)
    assert torch.equal(y.view(torch.uint8), out["y"].view(torch.uint8))


@pytest.mark.parametrize("which", ["x", "delta"])
def test_sum_in_place(cuda_ok, which):
    x, delta, weight = inputs(17, 2056, BF16, seed=2)
    want, _ = norm(x, delta, weight)
    a, b = x.clone(), delta.clone()
    out, _ = norm(a, b, weight, sum_out=a if which == "x" else b)
    assert torch.equal(out["y"], want["y"]) and torch.equal(out["sum"], want["sum"])


def test_rows_of_zeros_tiny_huge_and_not_finite(cuda_ok):
    x, _, weight = inputs(8, 1024, BF16, seed=3)
    x[0] = 0
    x[1] = 1e-30
    x[2] *= 1e15
    x[4, 3] = math.nan
    x[5, 1000] = math.inf
    x[6, 7] = 1e30                           # its square leaves fp32
    for e4m3 in (False, True):
        out, status = norm(x, None, weight, e4m3=e4m3)
        assert status == (bn.STATUS_BAD_ROW, 4)
        ok = torch.tensor([0, 1, 2, 3, 7], device="cuda")
        check({k: (v[ok] if v is not None else None) for k, v in out.items()}, x[ok], None, weight)
        for r in (4, 5, 6):
            assert bool(out["y"][r].float().isnan().all() and out["rstd"][r].isnan())
            assert out["y_scale"] is None or bool(out["y_scale"][r].isnan())
        assert bool((out["y"][0].float() == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,H", [(1, 8), (1, 4096), (5, 40), (33, 1032), (700, 2048), (4, 8200), (3, 16384), (1000, 264)])
def test_gradient_matches(cuda_ok, dtype, M, H):
    s, dsum, weight = inputs(M, H, dtype, seed=H + 1)
    g = torch.Generator(device="cuda").manual_seed(4)
    dy = torch.randn(M, H, generator=g, device="cuda").to(dtype)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    for with_sum in (True, False):
        dx, dw = torch.full_like(s, 7), torch.full((H,), 7.0, device="cuda")
        ws = workspace(M, H)
        bn.residual_norm_grad(s, weight, rstd, dy, dx, ws, dsum=dsum if with_sum else None, dweight=dw)
        v = s.double().requires_grad_()
        w = weight.double().requires_grad_()
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * w
        loss = (y * dy.double()).sum() + ((v * dsum.double()).sum() if with_sum else 0)
        want, wantw = torch.autograd.grad(loss, (v, w))
        wd, r = (weight.double() * dy.double()).abs(), rstd.double()[:, None]
        # the terms of dx, each with a few fp32 roundings; the mean adds its terms' sizes
        size = r * (wd + s.double().abs() * r * r * (wd * s.double().abs()).mean(1, keepdim=True))
        tol = half(dtype) * want.abs() * 1.0001 + 2 * E * size + (2.0 ** -23 * dsum.double().abs() if with_sum else 0)
        assert bool(((dx.double() - want).abs() <= tol).all())
        # M terms: at most M / 296 + 1 in a CTA, then 296 / 8 + 8 partial sums
        terms = (dy.double() * s.double() * r).abs().sum(0)
        tolw = 2.0 ** -24 * (M / 296 + 50) * terms + 1e-30
        assert bool(((dw.double() - wantw).abs() <= tolw).all())
    for dst in (dy.clone(), dsum.clone()):  # in place
        a = dict(dy=dy, dsum=dsum)
        a["dy" if torch.equal(dst, dy) else "dsum"] = dst
        bn.residual_norm_grad(s, weight, rstd, a["dy"], dst, workspace(M, H), dsum=a["dsum"])
        want = torch.empty_like(s)
        bn.residual_norm_grad(s, weight, rstd, dy, want, workspace(M, H), dsum=dsum)
        assert torch.equal(dst, want)


def test_gradient_against_differences(cuda_ok):
    """Central differences of the forward kernel in fp32: step 2^-5 on values of size 1, the
    third-order term below h^2 times the loss's scale, the forward's error over the step."""
    H = 32
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(1, H, generator=g, device="cuda")
    weight = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    dy = torch.randn(1, H, generator=g, device="cuda")
    h = 2.0 ** -5
    eye = h * torch.eye(H, device="cuda")
    out, _ = norm(torch.cat([x + eye, x - eye]), None, weight)
    loss = (out["y"].double() * dy.double()).sum(1)
    diff = (loss[:H] - loss[H:]) / (2 * h)
    one, _ = norm(x, None, weight)
    dx = torch.empty_like(x)
    bn.residual_norm_grad(x, weight, one["rstd"], dy, dx, workspace(1, H))
    scale = (dy.abs() * weight.abs()).sum().item()
    assert (diff - dx[0].double()).abs().max().item() <= h * h * scale + 2.0 ** -19 / h * scale / H


def test_same_result_every_time_and_captured(cuda_ok):
    s, dsum, weight = inputs(900, 1536, BF16, seed=6)
    dy = dsum.roll(1, 0).contiguous()
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-6)
    ws = workspace(900, 1536)
    dx, dw = torch.empty_like(s), torch.empty(1536, device="cuda")
    bn.residual_norm_grad(s, weight, rstd, dy, dx, ws, dsum=dsum, dweight=dw)
    first, firstw = dx.clone(), dw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bn.residual_norm_grad(s, weight, rstd, dy, dx, ws, dsum=dsum, dweight=dw)
    for _ in range(3):
        dx.zero_()
        dw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, first) and torch.equal(dw, firstw)


@pytest.mark.parametrize("M,H", [(5, 1024), (300, 272), (700, 4096)])
def test_launches_in_a_row_see_each_other(cuda_ok, M, H):
    """A launch may start before the one before it has ended: every call here reads what the
    call before wrote, in eager mode and replayed, and a copy follows the last."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    ws = workspace(M, H)
    a, b, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(M, device="cuda")
    dw, out = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")

    def chain(sync=lambda: None):
        a.copy_(x)
        for _ in range(3):
            sync()
            bn.residual_norm(a, None, w, 1e-6, b, ws, rstd=rstd)
            sync()
            bn.residual_norm(b, x, w, 1e-6, a, ws, sum=b, rstd=rstd)
            sync()
        bn.residual_norm_grad(b, w, rstd, a, dx, ws, dsum=b, dweight=dw)
        sync()
        out.copy_(dw)
        sync()
        bn.residual_norm_grad(b, w, rstd, dx, dx, ws, dweight=dw)
        sync()
        out.add_(dw)

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in (a, b, dx, rstd, dw, out)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
        chain()
    for run in (chain, graph.replay, chain, graph.replay):
        for t in (a, b, dx, rstd, dw, out):
            t.fill_(7)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip((a, b, dx, rstd, dw, out), want))
    assert bn.read_status(ws) == (0, -1)
