"""dspark_token_logprobs and its gradient against the definition in 64 bits.

Tolerances. The kernel sums V positive terms 2^z in fp32: a thread adds at most
V / 256 of them one after the other and the partial sums are joined in about 16
more steps, each step at most half an fp32 step (2^-24) off; 2^z itself is 2 units
of 2^-23 off; z carries two roundings of 2^-24 |z|, and terms past |z| = 30 weigh
less than 2^-30. So ln s is off by at most
    e = 2^-24 (V / 256 + 16) + 2^-22 + 2^-23 * 30,
and x - M or M / temp add 2^-23 of their own size. Gradients: exp(lp) with lp off
by 2^-23 (|x| + |lse|), rounded once to the logits' type.
"""
import math

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def score(logits, tok, temp=None, n=0, stream=None):
    B, J, V = logits.shape
    f = dict(device="cuda", dtype=F32)
    out = dict(logp=torch.full((B, J), 7.0, **f), entropy=torch.full((B, J), 7.0, **f),
               lse=torch.full((B, J), 7.0, **f))
    if n:
        out.update(top_idx=torch.full((B, J, n), -7, device="cuda", dtype=torch.int32),
                   top_logp=torch.full((B, J, n), 7.0, **f))
    ws = torch.zeros(bn.workspace_bytes(bn.OP_LOGPROBS, B, J, V, 0, bn._dtype_code(logits)), dtype=torch.uint8,
                     device="cuda")
    logp = out["logp"]
    bn.token_logprobs(logits, tok, temp, logp, ws, **{k: v for k, v in out.items() if k != "logp"}, stream=stream)
    torch.cuda.synchronize()
    return out, bn.read_status(ws)


def exact(logits, tok, temp, n):
    x = logits.double()
    if temp is not None:
        x = x / torch.where(temp > 0, temp, torch.ones_like(temp)).double()[:, None, None]
    top = x.amax(-1, keepdim=True)
    lse = torch.logsumexp(x, -1)
    lp = (x - top) - torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    order = torch.sort(logits.double(), dim=-1, descending=True, stable=True).indices[..., :n]
    return dict(logp=lp.gather(-1, tok.clamp(min=0).long()[..., None])[..., 0], entropy=ent, lse=lse,
                top_idx=order.int(), top_logp=lp.gather(-1, order)), top[..., 0]


def compare(out, logits, tok, temp, n):
    V = logits.shape[-1]
    ref, top = exact(logits, tok, temp, n)
    e = 2.0 ** -24 * (V / 256 + 16) + 2.0 ** -22 + 2.0 ** -23 * 30
    keep = tok >= 0

    def near(name, tol):
        got, want = out[name].double(), ref[name]
        k = keep if got.dim() == 2 else keep[..., None].expand_as(got)
        got, want = got[k], want[k]
        fin = torch.isfinite(want)
        assert torch.equal(got[~fin], want[~fin]), name
        err = (got - want).abs()[fin]
        lim = (tol + 2.0 ** -22 * want.abs())[fin] if not torch.is_tensor(tol) else (tol[k] + 2.0 ** -22 * want.abs())[fin]
        assert bool((err <= lim).all()), (name, (err - lim).max().item())

    near("logp", e)
    near("lse", e + 2.0 ** -23 * top.abs())
    # t / s carries e of its own size (at most H + ln s <= H + ln V) and the terms' z
    near("entropy", e * (2 + 2 * math.log(V)))
    if n:
        assert torch.equal(out["top_idx"][keep], ref["top_idx"][keep])
        near("top_logp", e)
    assert bool((out["logp"][~keep] == 0).all() and (out["entropy"][~keep] == 0).all())
    assert bool((out["lse"][~keep] == 0).all())
    if n:
        assert bool((out["top_idx"][~keep] == -1).all() and (out["top_logp"][~keep] == -math.inf).all())


def rows(B, J, V, dtype, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(B, J, V, generator=g, device="cuda") * std).to(dtype)
    tok = torch.randint(0, V, (B, J), generator=g, device="cuda", dtype=torch.int32)
    temp = torch.tensor([0.6, 1.0, 1.7, 0.0], device="cuda")[torch.arange(B, device="cuda") % 4]
    return logits, tok, temp


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,J,V,n", [
    (1, 1, 8, 8), (1, 1, 16, 0), (3, 2, 40, 5), (1, 3, 2048, 1), (2, 2, 2056, 32), (5, 7, 10000, 20),
    (1, 1, 151936, 20), (1, 2, 4104, 32), (300, 1, 1032, 3), (64, 5, 32000, 5)])
def test_scores_match(cuda_ok, dtype, B, J, V, n):
    logits, tok, temp = rows(B, J, V, dtype, seed=V + n)
    out, status = score(logits, tok, temp, n)
    assert status == (0, -1)
    compare(out, logits, tok, temp, n)


def test_peaked_flat_and_wide_rows(cuda_ok):
    V = 5000
    logits, tok, _ = rows(6, 1, V, F32, seed=3)
    logits[0] = 0.25                         # uniform: H = ln V, alternatives 0, 1, 2, ...
    logits[1, 0, 17] = 200.0                 # one certain token
    logits[2] *= 1000.0
    logits[3] = torch.linspace(-5, 5, V, device="cuda")
    logits[4] = torch.linspace(5, -5, V, device="cuda")
    logits[5] = -logits[5].abs() - 3e4
    tok[1, 0] = 17
    out, status = score(logits, tok, None, 32)
    assert status == (0, -1)
    compare(out, logits, tok, None, 32)
    assert out["logp"][1, 0] == 0 and out["entropy"][1, 0] == 0
    assert torch.equal(out["top_idx"][0, 0].cpu(), torch.arange(32, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_rows(cuda_ok, dtype):
    V = 3000
    low = torch.finfo(dtype).min
    logits, tok, _ = rows(7, 1, V, dtype, seed=5)
    temp = torch.tensor([0.3, 1.0, 2.0, 0.5, 1.0, 1.0, 1.0], device="cuda")
    logits[0, 0, 10:] = -math.inf            # few allowed
    logits[1, 0, 10:] = low
    logits[2, 0, :] = -math.inf
    logits[2, 0, 777] = -4.0                 # exactly one allowed
    logits[3, 0, :] = low                    # a whole row of the lowest value: uniform
    logits[4, 0, ::2] = -math.inf
    logits[5, 0, 1:] = low
    logits[6, 0, 5] = -0.0
    logits[6, 0, :5] = -1.0
    logits[6, 0, 6:] = -1.0
    logits[6, 0, 9] = 0.0                    # equal to -0: the lower index first
    tok[0, 0], tok[2, 0] = 2000, 777
    out, status = score(logits, tok, temp, 8)
    assert status == (0, -1)
    ref, _ = exact(logits, tok, temp, 8)
    assert out["logp"][0, 0] == -math.inf and out["logp"][2, 0] == 0 and out["entropy"][2, 0] == 0
    assert torch.equal(out["top_idx"], ref["top_idx"])
    e = 2.0 ** -24 * (V / 256 + 16) + 2.0 ** -22 + 2.0 ** -23 * 30
    for b in (0, 1, 2, 4, 6):
        assert abs(out["entropy"][b, 0].item() - ref["entropy"][b, 0].item()) <= e * (2 + 2 * math.log(V))
    assert abs(out["entropy"][3, 0].item() - math.log(V)) <= e * (2 + 2 * math.log(V))
    assert abs(out["logp"][3, 0].item() + math.log(V)) <= e
    assert out["top_logp"][2, 0, 1] == -math.inf and out["top_idx"][6, 0, 0] == 5


def test_rows_in_error_are_reported_and_defined(cuda_ok):
    V = 2000
    logits, tok, temp = rows(8, 2, V, BF16, seed=6)
    temp[:] = 1.0
    cases = [(bn.STATUS_BAD_ROW, lambda l, k, t: l[3, 1].fill_(-math.inf)),
             (bn.STATUS_BAD_ROW, lambda l, k, t: l[3, 1, 1999:].fill_(math.nan)),
             (bn.STATUS_BAD_ROW, lambda l, k, t: l[3, 1, 5:6].fill_(math.inf)),
             (bn.STATUS_BAD_TOKEN, lambda l, k, t: k[3, 1:].fill_(V)),
             (bn.STATUS_BAD_TOKEN, lambda l, k, t: k[3, 1:].fill_(-2))]
    for bit, spoil in cases:
        l, k, t = logits.clone(), tok.clone(), temp.clone()
        spoil(l, k, t)
        out, status = score(l, k, t, 4)
        assert status == (bit, 3)
        assert out["logp"][3, 1] == 0 and out["entropy"][3, 1] == 0 and out["lse"][3, 1] == 0
        assert bool((out["top_idx"][3, 1] == -1).all() and (out["top_logp"][3, 1] == -math.inf).all())
        k[3, 1] = -1
        if bit == bn.STATUS_BAD_TOKEN:
            compare(out, l, k, t, 4)
    for bad in (-1.0, math.nan):
        t = temp.clone()
        t[5] = bad
        out, status = score(logits, tok, t, 0)
        assert status == (bn.STATUS_BAD_TEMP, 5) and bool((out["logp"][5] == 0).all())


def test_padding_reads_nothing(cuda_ok):
    logits, tok, temp = rows(6, 4, 4096, BF16, seed=8)
    logits[:, 2:] = math.nan                 # never looked at
    tok[:, 2:] = -1
    out, status = score(logits, tok, temp, 5)
    assert status == (0, -1)
    ok = logits.clone()
    ok[:, 2:] = 0
    compare(out, ok, tok, temp, 5)


def test_many_entries_above_the_threshold(cuda_ok):
    """Large values in few of the row's vector columns: the candidate list overflows."""
    V, n = 65536, 32
    logits = torch.randn(2, 1, V, device="cuda").to(BF16)
    v = logits.view(2, 1, -1, 256, 8)        # [.., vector row, thread, entry]
    v[:, :, :, 30:62] = (100 + torch.arange(32, device="cuda") / 2).to(BF16)[:, None]
    v[1, 0, :, 40] += torch.rand(v.shape[2], 8, device="cuda").to(BF16)
    tok = torch.zeros(2, 1, device="cuda", dtype=torch.int32)
    out, status = score(logits, tok, None, n)
    assert status == (0, -1)
    compare(out, logits, tok, None, n)
    big = logits.repeat(400, 1, 1)           # one CTA per row: the columns are longest
    k = torch.zeros(800, 1, device="cuda", dtype=torch.int32)
    out, _ = score(big, k, None, n)
    compare(out, big, k, None, n)


def test_ties_go_to_the_lowest_index(cuda_ok):
    g = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.randint(0, 3, (4, 3, 20000), generator=g, device="cuda").to(BF16)
    tok = torch.zeros(4, 3, device="cuda", dtype=torch.int32)
    out, _ = score(logits, tok, None, 32)
    compare(out, logits, tok, None, 32)


def grad(logits, tok, temp, lse, ent, gl, gh, out=None, stream=None):
    B, J, V = logits.shape
    d = torch.full_like(logits, 7.0) if out is None else out
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bn.token_logprobs_grad(logits, tok, temp, lse, gl, d, ws, entropy=ent if gh is not None else None, g_entropy=gh,
                           stream=stream)
    torch.cuda.synchronize()
    return d, bn.read_status(ws)


@pytest.mark.parametrize("with_entropy", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,J,V", [(1, 1, 8), (2, 3, 1000), (5, 2, 8200), (3, 1, 151936), (200, 2, 1024)])
def test_gradient_matches(cuda_ok, dtype, B, J, V, with_entropy):
    logits, tok, temp = rows(B, J, V, dtype, seed=V)
    logits[0, 0, :4] = -math.inf
    tok[-1, -1] = -1 if B * J > 1 else tok[-1, -1]
    tok[0, 0] = 5
    out, _ = score(logits, tok, temp)
    g = torch.Generator(device="cuda").manual_seed(1)
    gl = torch.randn(B, J, generator=g, device="cuda")
    gh = torch.randn(B, J, generator=g, device="cuda") if with_entropy else None
    d, status = grad(logits, tok, temp, out["lse"], out["entropy"], gl, gh)
    assert status == (0, -1)
    tau = torch.where(temp > 0, temp, torch.ones_like(temp)).double()[:, None, None]
    z = logits.double().requires_grad_()
    # -1e4 has p = 0 in 64 bits as -inf has, without inf * 0 in autograd's products
    lp = torch.log_softmax(z.clamp(min=-1e4) / tau, -1)
    keep = tok >= 0
    loss = (lp.gather(-1, tok.clamp(min=0).long()[..., None])[..., 0] * gl.double())[keep].sum()
    p = lp.exp()
    ent = -torch.where(torch.isfinite(lp), p * lp, torch.zeros_like(p)).sum(-1)
    if gh is not None:
        loss = loss + (ent * gh.double())[keep].sum()
    want = torch.autograd.grad(loss, z)[0].nan_to_num(0.0)
    with torch.no_grad():
        x, lse = (logits.double() / tau), out["lse"].double()[..., None]
        rel = 2.0 ** -22 + 2.0 ** -23 * (x.abs().nan_to_num(0, 0, 0) + lse.abs() + 4)
        a = gl.double().abs()[..., None]
        h = gh.double().abs()[..., None] if gh is not None else torch.zeros_like(a)
        lpf = torch.where(p > 0, lp, 0.0).abs()
        size = p * (a + h * (1 + lpf + ent[..., None])) / tau
        # the entropy's own error (see above) times p
        e_h = (2.0 ** -24 * (V / 256 + 16) + 2.0 ** -22 + 2.0 ** -23 * 30) * (2 + 2 * math.log(V)) + 2.0 ** -22 * ent[..., None]
        tol = torch.finfo(dtype).eps / 2 * want.abs() + rel * size + h * p * e_h / tau + 2.0 ** -22 * want.abs() + 1e-38
        # the token's own entry is a difference of two terms of size g
        tol.scatter_add_(-1, tok.clamp(min=0).long()[..., None], (2.0 ** -22 * a / tau).expand(B, J, 1))
        err = (d.double() - want).abs()
    assert bool((err[keep] <= tol[keep]).all()), (err - tol).max().item()
    assert bool((d[~keep] == 0).all())


def test_gradient_against_differences(cuda_ok):
    """Central differences of the forward kernel's own fp32 outputs: with steps of 2^-4 the
    third-order term is h^2 / 6 times at most 4 of the gradient's scale, and the forward's
    error of 2^-19 is divided by the step."""
    V = 64
    g = torch.Generator(device="cuda").manual_seed(11)
    base = torch.randn(1, 1, V, generator=g, device="cuda")
    h = 2.0 ** -4
    steps = torch.cat([base + h * torch.eye(V, device="cuda")[:, None], base - h * torch.eye(V, device="cuda")[:, None]])
    tok = torch.full((2 * V, 1), 7, device="cuda", dtype=torch.int32)
    out, _ = score(steps, tok)
    gl, gh = 0.7, -0.3
    loss = (gl * out["logp"] + gh * out["entropy"])[:, 0].double()
    diff = (loss[:V] - loss[V:]) / (2 * h)
    one, _ = score(base, tok[:1])
    d, _ = grad(base, tok[:1], None, one["lse"], one["entropy"], torch.tensor([[gl]], device="cuda"),
                torch.tensor([[gh]], device="cuda"))
    tol = h * h / 6 * 4 * (abs(gl) + abs(gh) * 8) + 2.0 ** -19 / h
    assert (diff - d[0, 0].double()).abs().max().item() <= tol


def test_gradient_in_place_and_rows_in_error(cuda_ok):
    logits, tok, temp = rows(4, 2, 3000, BF16, seed=12)
    out, _ = score(logits, tok, temp)
    gl = torch.ones(4, 2, device="cuda")
    apart, _ = grad(logits, tok, temp, out["lse"], out["entropy"], gl, gl)
    same = logits.clone()
    grad(same, tok, temp, out["lse"], out["entropy"], gl, gl, out=same)
    assert torch.equal(apart, same)
    lse = out["lse"].clone()
    lse[2, 1] = math.nan
    d, status = grad(logits, tok, temp, lse, out["entropy"], gl, None)
    assert status == (bn.STATUS_BAD_ROW, 2) and bool((d[2, 1] == 0).all()) and bool((d[2, 0] != 0).any())
    k = tok.clone()
    k[1, 0] = 3000
    d, status = grad(logits, k, temp, out["lse"], out["entropy"], gl, None)
    assert status == (bn.STATUS_BAD_TOKEN, 1) and bool((d[1, 0] == 0).all())


def test_captured_and_on_another_stream(cuda_ok):
    logits, tok, temp = rows(8, 3, 9000, BF16, seed=13)
    want, _ = score(logits, tok, temp, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, status = score(logits, tok, temp, 5, stream=side)
    assert status == (0, -1)
    for k in want:
        assert torch.equal(want[k], got[k])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    logp, idx, lp = torch.zeros(8, 3, device="cuda"), torch.zeros(8, 3, 5, device="cuda", dtype=torch.int32), \
        torch.zeros(8, 3, 5, device="cuda")
    live = logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bn.token_logprobs(live, tok, temp, logp, ws, top_idx=idx, top_logp=lp)
    for shift in (0, 1):
        live.copy_(logits.roll(shift, 0))
        graph.replay()
        torch.cuda.synchronize()
        again, _ = score(live, tok, temp, 5)
        assert torch.equal(logp, again["logp"]) and torch.equal(idx, again["top_idx"])
