"""The operators together, as a round uses them: hidden states -> logits -> round -> scores,
and the gradient back to the hidden states.

Tolerances of the head: y carries half a step of its type (bf16 2^-9 of the value; e4m3
2^-4, 2^-10 of its scale below the normal range), each of the H products brings that
share, the accumulator 2^-23 (H / 16 + 156) of the sum of magnitudes, the logit half a
step of its own type.
"""
import pytest
import torch

from parity import SEED
from speculative_decoding_draft_sample_b200 import binding as bn
from speculative_decoding_draft_sample_b200 import workloads as wl
from speculative_decoding_draft_sample_b200.heads import LogitHead, TokenScores, quantize_rows
from speculative_decoding_draft_sample_b200.spec_round import SpecRound, run_host, to_device

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
H = 512


def parts(V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    norm_w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    w = (torch.randn(V, H, generator=g, device="cuda") * 2 * H ** -0.5).to(BF16)
    return norm_w, w, g


def hidden(g, *shape):
    return (torch.randn(*shape, H, generator=g, device="cuda") * 3).to(BF16)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,J", [(1, 1), (3, 5), (40, 6)])
def test_head_matches_the_definition(cuda_ok, B, J, e4m3, out):
    V = 1000
    norm_w, w, g = parts(V)
    x, delta = hidden(g, B, J), hidden(g, B, J)
    bias = torch.randn(V, generator=g, device="cuda")
    q, scale = quantize_rows(w) if e4m3 else (w, None)
    head = LogitHead(norm_w, q, B * J + 7, w_scale=scale, bias=bias)
    logits = torch.empty(B, J, V, device="cuda", dtype=out)
    head.run(x, logits, delta=delta)
    assert head.status() == (0, -1)
    v = (x.double() + delta.double()).view(B * J, H)
    y = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * norm_w.double()
    wd = q.double() * (scale.double()[:, None] if e4m3 else 1)
    want = (y @ wd.t() + bias.double()).view(B, J, V)
    S = (y.abs() @ wd.abs().t()).view(B, J, V)
    step = 2.0 ** -4 if e4m3 else 2.0 ** -9
    low = 2.0 ** -10 * (y.abs().amax(1) / 448).view(B, J, 1) * wd.abs().sum(1) if e4m3 else 0
    tol = (step + 2.0 ** -17 + 2.0 ** -23 * (H / 16 + 156)) * S + low
    tol = tol + (torch.finfo(out).eps / 2 + 2.0 ** -22) * (want.abs() + tol + bias.double().abs())
    assert bool(((logits.double() - want).abs() <= tol).all())
    assert torch.equal(head.sum[:B * J], (x.float() + delta.float()).to(BF16).view(-1, H))


def round_inputs(e4m3=False, greedy=0.0):
    w = wl.scaled(wl.DSPARK5, name="heads", B=24, K=4, V=4096, greedy_frac=greedy)
    inp = wl.generate(w)
    norm_w, weight, g = parts(w.V, seed=3)
    q, scale = quantize_rows(weight) if e4m3 else (weight, None)
    th, dh = LogitHead(norm_w, q, w.B * (w.K + 1), w_scale=scale), LogitHead(norm_w, q, w.B * w.K, w_scale=scale)
    host = {k: v for k, v in inp.items() if k not in ("target", "base")}
    t = hidden(g, w.B, w.K + 1)
    host["target_hidden"] = t.cpu()
    host["target_delta"] = hidden(g, w.B, w.K + 1).cpu()
    host["base_hidden"] = (t[:, :w.K].float() + torch.randn(w.B, w.K, H, generator=g, device="cuda")).to(BF16).cpu()
    return w, host, th, dh


@pytest.mark.parametrize("e4m3", [False, True])
def test_round_from_hidden_states(cuda_ok, e4m3):
    w, host, th, dh = round_inputs(e4m3, greedy=0.25)
    dev = to_device(host)
    rnd = SpecRound(w.B, w.K, w.V, w.r)
    rnd.run(dev, SEED, 2, target_head=th, draft_head=dh)
    # the same round from logits that the heads made on their own
    target = torch.empty(w.B, w.K + 1, w.V, device="cuda", dtype=BF16)
    base = torch.empty(w.B, w.K, w.V, device="cuda", dtype=BF16)
    th.run(dev["target_hidden"], target, delta=dev["target_delta"])
    dh.run(dev["base_hidden"], base)
    plain = SpecRound(w.B, w.K, w.V, w.r)
    plain.run(dict(dev, target=target, base=base), SEED, 2)
    torch.cuda.synchronize()
    assert rnd.status() == (0, -1) and plain.status() == (0, -1)
    for name in ("x", "d", "cut", "accepted", "out", "n_emit"):
        assert torch.equal(getattr(rnd, name), getattr(plain, name)), name
    assert int(rnd.accepted.sum()) > 0
    # from pinned host memory, the statistics on a side stream
    pinned = to_device(host, pin=True)
    live = {k: torch.zeros_like(v, device="cuda") if torch.is_tensor(v) else v for k, v in pinned.items()}
    out_h, n_h = torch.empty(w.B, w.K + 1, dtype=torch.int32).pin_memory(), torch.empty(w.B, dtype=torch.int32).pin_memory()
    side = torch.cuda.Stream()
    run_host(rnd, pinned, live, SEED, 2, out_h, n_h, side_stream=side, target_head=th, draft_head=dh)
    torch.cuda.synchronize()
    assert torch.equal(out_h, plain.out.cpu()) and torch.equal(n_h, plain.n_emit.cpu())


def test_scores_of_the_emitted_tokens(cuda_ok):
    w, host, th, dh = round_inputs(greedy=0.25)
    dev = to_device(host)
    rnd = SpecRound(w.B, w.K, w.V, w.r)
    with pytest.raises(bn.DSparkError, match="needs a run"):
        rnd.score(dev["temp"])
    rnd.run(dev, SEED, 5, target_head=th, draft_head=dh)
    s = rnd.score(dev["temp"], n_top=6)
    torch.cuda.synchronize()
    assert s.status() == (0, -1)
    emitted = torch.arange(w.K + 1, device="cuda") < rnd.n_emit[:, None]
    assert torch.equal(rnd.out >= 0, emitted)
    temp = torch.where(dev["temp"] > 0, dev["temp"], torch.ones_like(dev["temp"])).double()
    lp = torch.log_softmax(rnd.verified.double() / temp[:, None, None], -1)
    want = lp.gather(-1, rnd.out.clamp(min=0).long()[..., None])[..., 0]
    e = 2.0 ** -24 * (w.V / 256 + 16) + 2.0 ** -22 + 2.0 ** -23 * 30
    err = (s.logp.double() - want).abs()
    assert bool((err[emitted] <= e + 2.0 ** -22 * want.abs()[emitted]).all())
    assert bool((s.logp[~emitted] == 0).all() and (s.top_idx[~emitted] == -1).all())
    order = torch.sort(rnd.verified.double(), dim=-1, descending=True, stable=True).indices[..., :6].int()
    assert torch.equal(s.top_idx[emitted], order[emitted])
    # greedy requests emit the most likely token of every row
    greedy = (dev["temp"] == 0)[:, None] & emitted
    assert torch.equal(rnd.out[greedy], s.top_idx[..., 0][greedy])


def test_round_with_heads_and_scores_in_a_graph(cuda_ok):
    w, host, th, dh = round_inputs()
    dev = to_device(host)
    rnd = SpecRound(w.B, w.K, w.V, w.r)
    rnd.run(dev, SEED, 1, target_head=th, draft_head=dh)
    s = rnd.score(dev["temp"], n_top=3)
    torch.cuda.synchronize()
    want = [t.clone() for t in (rnd.out, s.logp, s.entropy, s.top_idx)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rnd.run(dev, SEED, 1, target_head=th, draft_head=dh)
        rnd.score(dev["temp"], n_top=3)
    for _ in range(2):
        for t in (rnd.out, s.logp, s.entropy, s.top_idx):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, v in zip((rnd.out, s.logp, s.entropy, s.top_idx), want):
            assert torch.equal(t, v)


def test_gradient_from_scores_to_hidden_states(cuda_ok):
    """The chain scores -> head against autograd in 64 bits. dlogits is rounded to bf16 (2^-9 of
    each entry), the normalised y that enters dweight too; dx is rounded to bf16 between the two
    calls and at the end. Errors are taken relative to the norm of each output, where independent
    half steps of 2^-9 stay below 2^-9 each: 4 of them, and 2^-12 for everything in fp32."""
    B, J, V = 6, 4, 2048
    norm_w, w, g = parts(V, seed=7)
    x, delta = hidden(g, B, J), hidden(g, B, J)
    tok = torch.randint(0, V, (B, J), generator=g, device="cuda", dtype=torch.int32)
    tok[2, 2:] = -1
    temp = torch.tensor([0.7, 1.0, 1.3, 0.9, 1.0, 2.0], device="cuda")
    gl, gh = torch.randn(B, J, generator=g, device="cuda"), 0.1 * torch.randn(B, J, generator=g, device="cuda")
    head, scores = LogitHead(norm_w, w, B * J), TokenScores(B, J, V, dtype=BF16)
    logits = torch.empty(B, J, V, device="cuda", dtype=BF16)
    head.run(x, logits, delta=delta)
    scores.run(logits, tok, temp)
    dlogits = torch.empty_like(logits)
    scores.gradient(logits, tok, temp, gl, dlogits, g_entropy=gh)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db, dn = torch.empty(V, device="cuda"), torch.empty(H, device="cuda")
    head.gradient(dlogits, dx, dweight=dw, dbias=db, dnorm_weight=dn)
    assert head.status() == (0, -1) and scores.status() == (0, -1)
    frozen = torch.empty_like(x)
    head.gradient(dlogits, frozen)
    assert torch.equal(frozen, dx)

    xs = head.sum.double().view(B, J, H).requires_grad_()
    nw, ww = norm_w.double().requires_grad_(), w.double().requires_grad_()
    bias = torch.zeros(V, device="cuda", dtype=torch.float64, requires_grad=True)
    y = xs / torch.sqrt(xs.square().mean(-1, keepdim=True) + 1e-6) * nw
    z = y @ ww.t() + bias
    z = z + (logits.double() - z).detach()      # the stored logits are what was scored
    lp = torch.log_softmax(z / temp.double()[:, None, None], -1)
    keep = tok >= 0
    loss = ((lp.gather(-1, tok.clamp(min=0).long()[..., None])[..., 0] * gl.double())[keep].sum()
            - ((lp.exp() * lp).sum(-1) * gh.double())[keep].sum())
    want = torch.autograd.grad(loss, (xs, ww, bias, nw))
    for got, ref in zip((dx, dw, db, dn), want):
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert rel <= 4 * 2.0 ** -9 + 2.0 ** -12, rel
    assert bool((dx[2, 2:] == 0).all())


def test_heads_refuse_what_does_not_fit(cuda_ok):
    norm_w, w, g = parts(256)
    q, scale = quantize_rows(w)
    with pytest.raises(bn.DSparkError, match="w_scale goes"):
        LogitHead(norm_w, q, 4)
    with pytest.raises(bn.DSparkError, match="norm_weight must have shape"):
        LogitHead(norm_w[:8], w, 4)
    with pytest.raises(bn.DSparkError, match="bfloat16 or float8"):
        LogitHead(norm_w, w.float(), 4)
    head = LogitHead(norm_w, w, 4)
    with pytest.raises(bn.DSparkError, match="do not fit"):
        head.run(hidden(g, 5), torch.empty(5, 256, device="cuda", dtype=BF16))
    with pytest.raises(bn.DSparkError, match="do not fit"):
        head.run(hidden(g, 4), torch.empty(4, 264, device="cuda", dtype=BF16))
    with pytest.raises(bn.DSparkError, match="contiguous"):
        head.run(hidden(g, 8)[::2], torch.empty(4, 256, device="cuda", dtype=BF16))
    with pytest.raises(bn.DSparkError, match="no gradient"):
        LogitHead(norm_w, q, 4, w_scale=scale).gradient(torch.empty(4, 256, device="cuda", dtype=BF16), hidden(g, 4))
    with pytest.raises(bn.DSparkError, match="n_top"):
        TokenScores(2, 2, 64, n_top=33)
    rnd = SpecRound(4, 2, 512, 64)
    with pytest.raises(bn.DSparkError, match="vocabulary"):
        rnd.run({"target_hidden": hidden(g, 4, 3)}, SEED, 0, target_head=head)


def test_calls_at_once_on_two_streams(cuda_ok):
    """Every operator on two streams at the same time, each with its own workspace."""
    V, M = 20000, 40
    norm_w, w, g = parts(V, seed=9)
    xs = [hidden(g, M) for _ in range(2)]
    toks = [torch.randint(0, V, (M, 1), generator=g, device="cuda", dtype=torch.int32) for _ in range(2)]

    def issue(i, stream, bufs):
        head, scores, logits, dlogits, dx = bufs
        head.run(xs[i], logits, stream=stream)
        rows = logits.view(M, 1, V)
        scores.run(rows, toks[i], None, stream=stream)
        scores.gradient(rows, toks[i], None, torch.ones_like(scores.logp), dlogits, stream=stream)
        head.gradient(dlogits, dx, stream=stream)

    def buffers():
        return (LogitHead(norm_w, w, M), TokenScores(M, 1, V, 5), torch.empty(M, V, device="cuda", dtype=BF16),
                torch.empty(M, 1, V, device="cuda", dtype=BF16), torch.empty(M, H, device="cuda", dtype=BF16))

    want = []
    for i in range(2):
        b = buffers()
        issue(i, None, b)
        want.append((b[1].logp, b[1].top_idx, b[4]))
    streams, bufs = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            issue(i, streams[i], bufs[i])
    torch.cuda.synchronize()
    for i in range(2):
        got = (bufs[i][1].logp, bufs[i][1].top_idx, bufs[i][4])
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        assert bufs[i][0].status() == (0, -1) and bufs[i][1].status() == (0, -1)


def test_offsets_past_32_bits(cuda_ok):
    """More than 2^31 entries in a tensor: the last rows against the same rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, V, n = 16500, 131072, 6              # 2.16e9 logits
    few = torch.randn(n, 1, V, generator=g, device="cuda").to(BF16)
    logits = torch.empty(B, 1, V, device="cuda", dtype=BF16)
    logits[-n:] = few
    tok = torch.full((B, 1), -1, device="cuda", dtype=torch.int32)
    tok[-n:] = torch.randint(0, V, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    many, alone = TokenScores(B, 1, V, 3), TokenScores(n, 1, V, 3)
    many.run(logits, tok, None)
    alone.run(few, tok[-n:].contiguous(), None)
    # a row shared by a cluster adds its sums in another order than a CTA of its own
    assert (many.logp[-n:] - alone.logp).abs().max().item() <= 2.0 ** -24 * (V / 256 + 16) * 2 + 2.0 ** -20
    assert torch.equal(many.top_idx[-n:], alone.top_idx) and bool((many.logp[:-n] == 0).all())
    ones = torch.ones(B, 1, device="cuda")
    many.gradient(logits, tok, None, ones, logits)
    d = torch.empty_like(few)
    bn.token_logprobs_grad(few, tok[-n:].contiguous(), None, many.lse[-n:].contiguous(), ones[-n:].contiguous(), d, alone.ws)
    assert torch.equal(logits[-n:], d) and bool((logits[0] == 0).all())

    K = 64                                  # the same buffer as a product's output
    x, w = torch.randn(B, K, generator=g, device="cuda").to(BF16), torch.randn(V, K, generator=g, device="cuda").to(BF16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bn.linear(x, w, logits.view(B, V), ws)
    want = x[-n:].double() @ w.double().t()
    S = x[-n:].double().abs() @ w.double().abs().t()
    err = (logits.view(B, V)[-n:].double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -23 * (K / 16 + 156) * S).all())

    M, W = 131500, 16384                    # and as rows of a norm, in place
    rows = logits.view(-1)[:M * W].view(M, W)
    last = torch.randn(n, W, generator=g, device="cuda").to(BF16)
    rows[-n:] = last
    weight = torch.ones(W, device="cuda", dtype=BF16)
    rstd = torch.empty(M, device="cuda")
    y = torch.empty(M, W, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.empty(M, device="cuda")
    nws = torch.zeros(bn.workspace_bytes(bn.OP_NORM, M, 0, W, 0, 0), dtype=torch.uint8, device="cuda")
    bn.residual_norm(rows, rows, weight, 1e-6, y, nws, sum=rows, y_scale=scale, rstd=rstd)
    v = 2 * last.double()
    exact = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    tol = (2.0 ** -4 + 2.0 ** -16) * exact.abs() + 2.0 ** -10 * scale[-n:, None].double()
    assert bool(((y[-n:].double() * scale[-n:, None].double() - exact).abs() <= tol).all())
    assert torch.equal(rows[-n:], 2 * last)


def test_misaligned_tensors_are_refused(cuda_ok):
    def off(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        return torch.zeros(n + 8, device="cuda", dtype=dtype)[1:1 + n].view(shape)

    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    b = lambda *s: torch.zeros(*s, device="cuda", dtype=BF16)  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    tok = torch.zeros(2, 2, device="cuda", dtype=torch.int32)
    calls = [
        lambda: bn.token_logprobs(off((2, 2, 64), BF16), tok, None, f(2, 2), ws),
        lambda: bn.token_logprobs_grad(b(2, 2, 64), tok, None, f(2, 2), f(2, 2), off((2, 2, 64), BF16), ws),
        lambda: bn.residual_norm(off((4, 64), BF16), None, b(64), 1e-6, b(4, 64), ws),
        lambda: bn.residual_norm(b(4, 64), None, b(64), 1e-6, off((4, 64), BF16), ws),
        lambda: bn.residual_norm_grad(b(4, 64), b(64), f(4), off((4, 64), BF16), b(4, 64), ws),
        lambda: bn.linear(off((4, 64), BF16), b(8, 64), b(4, 8), ws),
        lambda: bn.linear(b(4, 64), off((8, 64), BF16), b(4, 8), ws),
        lambda: bn.linear_grad(b(4, 64), b(8, 64), off((4, 8), BF16), ws, dx=b(4, 64)),
        lambda: bn.linear_grad(b(4, 64), b(8, 64), b(4, 8), ws, dx=off((4, 64), BF16)),
        lambda: bn.linear(b(4, 64), b(8, 64), b(4, 8), off((256,), torch.uint8)),
    ]
    for call in calls:
        with pytest.raises(bn.DSparkError, match="invalid argument"):
            call()
    for call in (lambda: bn.residual_norm(b(4, 60), None, b(60), 1e-6, b(4, 60), ws),
                 lambda: bn.linear(b(4, 60), b(8, 60), b(4, 8), ws),
                 lambda: bn.linear(b(0, 64), b(8, 64), b(0, 8), ws),
                 lambda: bn.linear_grad(b(4, 64), b(12, 64), b(4, 12), ws, dx=b(4, 64)),
                 lambda: bn.token_logprobs(b(2, 2, 60), tok, None, f(2, 2), ws)):
        with pytest.raises(bn.DSparkError, match="invalid argument"):
            call()


def test_buffers_made_by_a_call_belong_to_its_stream(cuda_ok):
    """run() and score() make their logits and scores at first use; neither the memory's last
    user on the current stream nor its own clearing may come behind the call's work."""
    w, host, th, dh = round_inputs()
    dev = to_device(host)
    side = torch.cuda.Stream()
    plain = SpecRound(w.B, w.K, w.V, w.r)
    plain.run(dev, SEED, 3, target_head=th, draft_head=dh)
    bad = dev["temp"].clone()
    bad[1] = -1
    want = plain.score(bad, n_top=2)
    assert want.status()[0] == bn.STATUS_BAD_TEMP
    rnd = SpecRound(w.B, w.K, w.V, w.r)
    old = [torch.empty_like(plain.target), torch.empty_like(plain.base)]
    for t in old:
        t.fill_(0)  # (the kernel is loaded now, not behind the sleep)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda._sleep(500_000_000)  # a quarter of a second; the current stream is still busy with the memory it frees
    for t in old:
        t.fill_(7)
    del t, old
    rnd.run(dev, SEED, 3, stream=side, target_head=th, draft_head=dh)
    got = rnd.score(bad, n_top=2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(rnd.target, plain.target) and torch.equal(rnd.base, plain.base)
    assert torch.equal(got.logp, want.logp) and torch.equal(rnd.out, plain.out)
    assert got.status() == (bn.STATUS_BAD_TEMP, 1)


def test_captured_between_streams_and_other_nodes(cuda_ok):
    """Launches that may start early, where the node before them is a copy, a fill, another
    stream's kernel or nothing: each still sees all that it waits for."""
    V, M = 4096, 48
    norm_w, w, g = parts(V, seed=11)
    head, scores = LogitHead(norm_w, w, M), TokenScores(M, 1, V, 3)
    src = [hidden(g, M) for _ in range(2)]
    tok = torch.randint(0, V, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    x, delta, dx = (torch.empty_like(src[0]) for _ in range(3))
    logits, dlogits = (torch.empty(M, V, device="cuda", dtype=BF16) for _ in range(2))
    gl, late = torch.empty(M, 1, device="cuda"), torch.empty(M, V, device="cuda", dtype=BF16)
    dnorm = torch.empty(H, device="cuda")
    dw, db = torch.empty_like(w), torch.empty(V, device="cuda")
    side = torch.cuda.Stream()

    def step(sync=lambda: None):
        main = torch.cuda.current_stream()
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        with torch.cuda.stream(side):
            delta.copy_(src[1])
            for _ in range(4):
                delta.mul_(1)
            join.record(side)
        sync()
        x.copy_(src[0])
        main.wait_event(join)  # a copy and another stream's kernel before the first launch
        sync()
        head.run(x, logits, delta=delta)
        sync()
        fork.record(main)
        side.wait_event(fork)  # a launch whose stream holds nothing but another's end
        scores.run(logits.view(M, 1, V), tok, None, stream=side)
        with torch.cuda.stream(side):
            gl.copy_(scores.logp)
            join.record(side)
        sync()
        main.wait_event(join)
        scores.gradient(logits.view(M, 1, V), tok, None, gl, dlogits.view(M, 1, V))
        sync()
        head.gradient(dlogits, dx, dweight=dw, dbias=db, dnorm_weight=dnorm)
        sync()
        fork.record(main)
        side.wait_event(fork)
        with torch.cuda.stream(side):
            late.copy_(dlogits)
            late.add_(dw.sum(1) + db)
            join.record(side)
        main.wait_event(join)
        sync()

    outs = (logits, scores.logp, scores.top_idx, dlogits, dx, dnorm, dw, db, late)
    step(torch.cuda.synchronize)
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    first = torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):  # the graph's first node
        head.run(x, logits, delta=delta)
    for run in (step, graph.replay, graph.replay, step):
        for t in outs + (x, delta, gl):
            t.fill_(3)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for _ in range(3):
        logits.fill_(3)
        first.replay()
        assert torch.equal(logits, want[0])
    assert head.status() == (0, -1) and scores.status() == (0, -1)
