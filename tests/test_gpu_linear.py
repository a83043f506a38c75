"""dspark_linear and its gradient against the definition in 64 bits.

Tolerances. The products of bf16 or e4m3 factors are exact in fp32; the accumulator
takes 16 (bf16) or 32 (e4m3) of them at a time, each step at most one unit of 2^-23 of
the sum of magnitudes S = sum |x| |w| off (whether it rounds or truncates), so the sum
is within 2^-23 (K / 16 + 8 + splits) S; splits are at most 148. Activations have
slopes below 1.13 and their own error of 2^-21; the result is rounded once.
"""
import math

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def act64(z, act):
    return {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu,
            "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act](z)


def operand(rows, K, e4m3, g, std=1.0):
    v = torch.randn(rows, K, generator=g, device="cuda") * std
    if not e4m3:
        return v.to(BF16), None
    scale = v.abs().amax(1) / 448
    return (v / scale[:, None]).to(E4M3), scale


def workspace(M, N, K, code=bn.BF16, mode=0):
    n = bn.workspace_bytes(bn.OP_LINEAR, M, mode, N, K, code)
    assert n > 0
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda").index_fill_(0, torch.arange(256, device="cuda"), 0)


def run(M, N, K, e4m3=False, act="none", bias=False, residual=False, out=BF16, pre=False, seed=0, in_place=False,
        stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, xs = operand(M, K, e4m3, g)
    w, wsc = operand(N, K, e4m3, g, K ** -0.5)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(out) if residual else None
    guard = torch.full((M * N + 64,), 7.0, device="cuda", dtype=out)   # rows behind the last are left as they were
    y = guard[:M * N].view(M, N)
    if in_place:
        y.copy_(r)
    p = torch.full((M, N), 7.0, device="cuda", dtype=out) if pre else None
    ws = workspace(M, N, K, bn.E4M3 if e4m3 else bn.BF16)
    bn.linear(x, w, y, ws, x_scale=xs, w_scale=wsc, bias=b, residual=y if in_place else r, pre=p, act=act, stream=stream)
    torch.cuda.synchronize()
    assert bn.read_status(ws) == (0, -1)
    assert bool((guard[M * N:] == 7).all())
    xd, wd = x.double(), w.double()
    if e4m3:
        xd, wd = xd * xs.double()[:, None], wd * wsc.double()[:, None]
    z = xd @ wd.t() + (b.double() if bias else 0)
    S = xd.abs() @ wd.abs().t() + (b.double().abs() if bias else 0)
    want = act64(z, act) + (r.double() if residual else 0)
    acc = 1.13 * 2.0 ** -23 * (K / 16 + 8 + 148) * S + 2.0 ** -21 * act64(z, act).abs()
    eps = torch.finfo(out).eps / 2
    tol = acc + (eps + 2.0 ** -23) * (want.abs() + acc) + 2.0 ** -23 * (r.double().abs() if residual else 0)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()
    if pre:
        assert bool(((p.double() - z).abs() <= acc + eps * (z.abs() + acc)).all())
    return y


SIZES = [(1, 1, 8), (1, 8, 64), (1, 4096, 4096), (3, 130, 72), (16, 1000, 2048), (17, 257, 1000), (64, 5, 520),
         (100, 300, 64), (130, 129, 200), (256, 256, 256), (257, 1001, 136), (500, 2056, 4104), (1283, 517, 96)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_bf16_sizes(cuda_ok, M, N, K):
    run(M, N, K, seed=K)


@pytest.mark.parametrize("M,N,K", [(m, n, (k + 15) // 16 * 16) for m, n, k in SIZES])
def test_e4m3_sizes(cuda_ok, M, N, K):
    run(M, N, K, e4m3=True, seed=K, out=F32 if M % 2 else BF16)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("M,N", [(5, 300), (300, 203)])
def test_epilogue(cuda_ok, act, out, e4m3, M, N):
    run(M, N, 320, e4m3=e4m3, act=act, bias=True, residual=True, out=out, pre=True, seed=3)
    run(M, N, 320, e4m3=e4m3, act=act, residual=True, out=out, in_place=True, seed=4)


def test_wide_outputs_and_many_tiles(cuda_ok):
    run(16, 129280, 128, seed=5)
    run(600, 20000, 192, seed=6, bias=True)


@pytest.mark.parametrize("M,N,K", [(70, 264, 64), (33, 517, 2048), (300, 1001, 128)])
@pytest.mark.parametrize("offs", [(0, 0, 0), (1, 1, 1), (3, 3, 0), (0, 5, 0), (0, 0, 1), (7, 0, 2)])
def test_outputs_of_any_alignment(cuda_ok, M, N, K, offs):
    """y, residual and pre start at any 2-byte boundary, alike or not."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x, _ = operand(M, K, False, g)
    w, _ = operand(N, K, False, g, K ** -0.5)
    r = torch.randn(M, N, generator=g, device="cuda").to(BF16)
    want, wpre = torch.empty(M, N, device="cuda", dtype=BF16), torch.empty(M, N, device="cuda", dtype=BF16)
    bn.linear(x, w, want, workspace(M, N, K), residual=r, pre=wpre, act="gelu")

    def at(off):
        flat = torch.full((M * N + 16,), 7.0, device="cuda", dtype=BF16)
        return flat, flat[off:off + M * N].view(M, N)

    (fy, y), (_, rr), (fp, p) = at(offs[0]), at(offs[1]), at(offs[2])
    rr.copy_(r)
    bn.linear(x, w, y, workspace(M, N, K), residual=rr, pre=p, act="gelu")
    assert torch.equal(y, want) and torch.equal(p, wpre)
    for flat, off in ((fy, offs[0]), (fp, offs[2])):
        assert bool((flat[:off] == 7).all() and (flat[off + M * N:] == 7).all())
    bn.linear(x, w, rr, workspace(M, N, K), residual=rr, act="gelu")
    assert torch.equal(rr, want)


def test_split_contraction_is_deterministic(cuda_ok):
    a = run(8, 200, 8192, seed=7, bias=True, act="silu")
    for _ in range(5):
        assert torch.equal(a, run(8, 200, 8192, seed=7, bias=True, act="silu"))


def test_infinities_and_nan_pass(cuda_ok):
    x, w = torch.zeros(3, 64, device="cuda", dtype=BF16), torch.ones(20, 64, device="cuda", dtype=BF16)
    x[0, 3], x[1, 5] = math.inf, math.nan
    y = torch.empty(3, 20, device="cuda", dtype=BF16)
    for act in ("none", "relu"):
        bn.linear(x, w, y, workspace(3, 20, 64), act=act)
        assert bool((y[0] == math.inf).all() and y[1].isnan().all() and (y[2] == 0).all())


GRAD_SIZES = [(1, 8, 8), (1, 1000, 64), (3, 136, 72), (70, 64, 200), (128, 256, 128), (257, 1032, 136), (600, 520, 1000),
              (40, 8000, 256), (2048, 64, 72)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K", GRAD_SIZES)
def test_gradient_matches(cuda_ok, M, N, K, act):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, _ = operand(M, K, False, g)
    w, _ = operand(N, K, False, g, K ** -0.5)
    dy = torch.randn(M, N, generator=g, device="cuda").to(BF16)
    pre = (torch.randn(M, N, generator=g, device="cuda") * 2).to(BF16)
    pre[0, 0] = 0
    dx, dw = torch.full_like(x, 7), torch.full_like(w, 7)
    db = torch.full((N,), 7.0, device="cuda")
    ws = workspace(M, N, K, mode=1 if act != "none" else 2)
    bn.linear_grad(x, w, dy, ws, dx=dx, dw=dw, dbias=db, pre=pre if act != "none" else None, act=act)
    torch.cuda.synchronize()
    assert bn.read_status(ws) == (0, -1)
    z = pre.double().requires_grad_()
    d = torch.autograd.grad((act64(z, act) * dy.double()).sum(), z)[0]
    # dpre: fp32 error 2^-20 of dy, then one rounding to bf16 (none without an activation)
    e_d = 2.0 ** -20 * dy.double().abs() if act != "none" else 0 * d
    e_r = e_d + (2.0 ** -9 * 2 * d.abs() if act != "none" else 0)
    for got, a, ea, b, n in ((dx, d, e_r, w.double(), N), (dw, d.t(), e_r.t() if act != "none" else e_r.t(), x.double(), M)):
        want = a @ b
        S = a.abs() @ b.abs()
        acc = 2.0 ** -23 * (n / 16 + 8 + 148) * S + ea @ b.abs()
        tol = acc + 2.0 ** -8 * (want.abs() + acc) * 0.5 * 2
        assert bool(((got.double() - want).abs() <= tol).all())
    tolb = (2.0 ** -24 * (M / 8 + 20) * (d.abs() + e_d)).sum(0) + (e_d.sum(0) if act != "none" else 0) + 1e-30
    assert bool(((db.double() - d.sum(0)).abs() <= tolb).all())


def test_gradient_parts_alone(cuda_ok):
    M, N, K = 50, 264, 104
    g = torch.Generator(device="cuda").manual_seed(2)
    x, _ = operand(M, K, False, g)
    w, _ = operand(N, K, False, g)
    dy = torch.randn(M, N, generator=g, device="cuda").to(BF16)
    every = dict(dx=torch.empty_like(x), dw=torch.empty_like(w), dbias=torch.empty(N, device="cuda"))
    ws = workspace(M, N, K, mode=1)
    bn.linear_grad(x, w, dy, ws, pre=dy, act="gelu", **every)
    for k, v in every.items():
        one = torch.full_like(v, 7)
        bn.linear_grad(x, w, dy, ws, pre=dy, act="gelu", **{k: one})
        assert torch.equal(one, v), k


def test_gradient_against_differences(cuda_ok):
    """The forward kernel in fp32 output; bf16 inputs move by 2^-4, exactly representable here."""
    M, N, K = 1, 16, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randint(-8, 9, (M, K), generator=g, device="cuda") / 8).to(BF16)
    w = (torch.randint(-8, 9, (N, K), generator=g, device="cuda") / 8).to(BF16)
    dy = (torch.randint(-8, 9, (M, N), generator=g, device="cuda") / 8).to(BF16)
    h = 2.0 ** -4
    eye = h * torch.eye(K, device="cuda")
    pts = torch.cat([x.float() + eye, x.float() - eye]).to(BF16)
    y = torch.empty(2 * K, N, device="cuda")
    bn.linear(pts, w, y, workspace(2 * K, N, K), act="silu")
    loss = (y.double() * dy.double()).sum(1)
    diff = (loss[:K] - loss[K:]) / (2 * h)
    out, pre = torch.empty(M, N, device="cuda", dtype=BF16), torch.empty(M, N, device="cuda", dtype=BF16)
    bn.linear(x, w, out, workspace(M, N, K), pre=pre, act="silu")
    dx = torch.empty_like(x)
    bn.linear_grad(x, w, dy, workspace(M, N, K, mode=1), dx=dx, pre=pre, act="silu")
    S = (dy.double().abs() @ w.double().abs())[0]
    # silu'' and silu''' stay below 0.6; pre moved by 2^-9 of its size (at most 8); two roundings of 2^-8
    tol = S * (h * h / 6 * 0.6 + 0.6 * 8 * 2.0 ** -9 + 2 * 2.0 ** -8) + 1e-4
    assert bool(((diff - dx[0].double()).abs() <= tol).all())


def test_captured_shared_workspace_and_side_stream(cuda_ok):
    M, N, K = 12, 300, 4096                  # the contraction is split over a cluster
    g = torch.Generator(device="cuda").manual_seed(4)
    x, _ = operand(M, K, False, g)
    w, _ = operand(N, K, False, g)
    ws = workspace(M, N, K)
    a, b = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = torch.empty(M, N, device="cuda")
    bn.linear(x, w, want, ws, stream=side)
    side.synchronize()
    x2 = x.roll(1, 0).contiguous()
    graphs = []
    for src, dst in ((x, a), (x2, b)):       # two graphs, one workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bn.linear(src, w, dst, ws)
        graphs.append(graph)
    for _ in range(3):
        a.zero_()
        b.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want.roll(1, 0))


@pytest.mark.parametrize("M,N,K", [(5, 1456, 1640), (300, 1000, 520), (1000, 4096, 1024)])
def test_gradient_captured_and_followed(cuda_ok, M, N, K):
    """dx and dw run beside each other; what follows in the stream sees both complete."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x, _ = operand(M, K, False, g)
    w, _ = operand(N, K, False, g, K ** -0.5)
    dy = torch.randn(M, N, generator=g, device="cuda").to(BF16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    ws = workspace(M, N, K, mode=1)
    copies = [torch.empty_like(t) for t in (dx, dw, db)]

    def step():
        bn.linear_grad(x, w, dy, ws, dx=dx, dw=dw, dbias=db, pre=dy, act="silu")
        for c, t in zip(copies, (dx, dw, db)):
            c.copy_(t)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dx, dw, db)]
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for run_once in (step, graph.replay, graph.replay, step):
        for t in (dx, dw, db, *copies):
            t.fill_(7)
        run_once()
        torch.cuda.synchronize()
        for a, b, c in zip(copies, want, (dx, dw, db)):
            assert torch.equal(a, b) and torch.equal(c, b)
    assert bn.read_status(ws) == (0, -1)
