"""What is measured of the operators around a speculative round: the logit head in front of it (residual norm,
linear product) and the scores of its tokens behind it (log probabilities), each direction and type.

listed() and draw() give cases, prepare() a case's inputs on the GPU, run() one pass in plain torch operations (own
False) or through the framework's calls (own True), work() what a pass cannot do without, exact() the definition in
64 bits. Weights are laid out [outputs, inputs]; a token of -1 is padding, as verification writes it behind the
emitted tokens.
"""
import math

import torch

own = False

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16}
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the smallest round's emitted tokens: latency alone
        dict(name="logprobs_b4_j5_v1024_f32_top5", op="logprobs", B=4, J=5, V=1024, dtype="f32", top=5, padded=True),
        # one request's block scored with the most alternatives that servers return
        dict(name="logprobs_b1_j6_v151936_top20", op="logprobs", B=1, J=6, V=151936, dtype="bf16", top=20, padded=False),
        # the emitted tokens of a full serving batch with five alternatives
        dict(name="logprobs_b256_j6_v129280_top5", op="logprobs", B=256, J=6, V=129280, dtype="bf16", top=5,
             padded=True),
        # the gradient of a drafter's or policy's loss over a batch of blocks, with an entropy bonus
        dict(name="logprobs_grad_b256_j5_v129280", op="logprobs_grad", B=256, J=5, V=129280, dtype="bf16", entropy=True,
             padded=False),
        # the same on a small vocabulary in 32 bits, sequences of uneven length
        dict(name="logprobs_grad_b37_j9_v32000_f32", op="logprobs_grad", B=37, J=9, V=32000, dtype="f32", entropy=False,
             padded=True),
        # final norm of a single token
        dict(name="norm_m1_h4096", op="norm", M=1, H=4096, dtype="bf16", out="bf16"),
        # final norm of a full verification batch, quantised for an 8-bit head
        dict(name="norm_m1536_h7168_e4m3", op="norm", M=1536, H=7168, dtype="bf16", out="e4m3"),
        # backward of the norm over a training batch
        dict(name="norm_grad_m8192_h4096", op="norm_grad", M=8192, H=4096, dtype="bf16"),
        # logits of a small decode batch: the weights' bytes
        dict(name="linear_m16_n129280_k4096", op="linear", M=16, N=129280, K=4096, type="bf16", act="none", bias=False,
             residual=False),
        # logits of a full verification batch (256 requests, 6 rows each) with an 8-bit head: the tensor cores' rate
        dict(name="linear_m1536_n129280_k4096_e4m3", op="linear", M=1536, N=129280, K=4096, type="e4m3", act="none",
             bias=False, residual=False),
        # a hidden layer of a drafter's head, odd sizes, everything in its epilogue
        dict(name="linear_m1283_n5003_k4096_silu", op="linear", M=1283, N=5003, K=4096, type="bf16", act="silu",
             bias=True, residual=True),
        # its backward pass
        dict(name="linear_grad_m2048_n5120_k4096_gelu", op="linear_grad", M=2048, N=5120, K=4096, act="gelu",
             bias=True),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, rounded to a multiple of step."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n // step * step))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "norm", "norm_grad", "linear", "linear", "linear_grad"])
    if op == "logprobs":
        dtype, V = rng.choice(["bf16", "bf16", "f32"]), _log(rng, 1000, 152000, 8)
        rows = _log(rng, 1, max(2, min(1536, 150_000_000 // V)))
        J = min(rows, rng.randint(1, 17))
        return dict(op=op, B=max(1, rows // J), J=J, V=V, dtype=dtype, top=rng.choice([0, 1, 5, 8, 20, 32]),
                    padded=rng.random() < 0.5)
    if op == "logprobs_grad":
        V = _log(rng, 1000, 152000, 8)
        rows = _log(rng, 1, max(2, min(4096, 120_000_000 // V)))
        J = min(rows, rng.randint(1, 17))
        return dict(op=op, B=max(1, rows // J), J=J, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    entropy=rng.random() < 0.5, padded=rng.random() < 0.5)
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, M=_log(rng, 1, 8192), H=_log(rng, 256, 8192, 8), dtype=dtype, out=rng.choice([dtype, "e4m3"]))
    if op == "norm_grad":
        return dict(op=op, M=_log(rng, 1, 8192), H=_log(rng, 256, 8192, 8), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "linear":
        M, K, kind = _log(rng, 1, 2048), _log(rng, 256, 8192, 16), rng.choice(["bf16", "e4m3"])
        N = _log(rng, 1, int(max(64, min(152000, 8e11 / (M * K)))))
        return dict(op=op, M=M, N=N, K=K, type=kind, act=rng.choice(["none", "none", "relu", "silu", "gelu"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    M, K = _log(rng, 1, 4096), _log(rng, 256, 8192, 8)
    N = _log(rng, 64, int(max(128, min(32000, 8e10 / (M * K)))), 8)
    return dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.5)


def _rows(case):
    """How many of a case's B x J rows hold a token: request b emits 1 + (b mod J) of them where rows are padded."""
    B, J = case["B"], case["J"]
    return sum(1 + b % J for b in range(B)) if case["padded"] else B * J


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"logprobs": _prepare_logprobs, "logprobs_grad": _prepare_logprobs, "norm": _prepare_norm,
            "norm_grad": _prepare_norm, "linear": _prepare_linear, "linear_grad": _prepare_linear}[case["op"]](case, g)


def _normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _prepare_logprobs(case, g):
    B, J, V, dtype = case["B"], case["J"], case["V"], TYPES[case["dtype"]]
    # Zipf log probabilities in a random order plus noise per row, as a language model's logits fall off
    zipf = -1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=F32))
    zipf = zipf[torch.randperm(V, generator=g, device="cuda")]
    logits = torch.empty(B, J, V, device="cuda", dtype=dtype)
    for b0 in range(0, B, 64):
        part = logits[b0:b0 + 64]
        part.copy_(zipf + torch.randn(part.shape, generator=g, device="cuda") * 0.7)
    # likely tokens, as sampling gives them: the largest of the row under Gumbel noise on a random subset
    subset = torch.randint(0, V, (256,), generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(B, J, 256, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    tok = subset[(logits[:, :, subset].float() + noise).argmax(-1)].to(torch.int32)
    if case["padded"]:
        count = (1 + torch.arange(B, device="cuda") % J)[torch.randperm(B, generator=g, device="cuda")]
        tok = torch.where(torch.arange(J, device="cuda") < count[:, None], tok, -1).to(torch.int32)
    temp = torch.tensor([0.6, 0.8, 1.0], device="cuda")[torch.randint(0, 3, (B,), generator=g, device="cuda")]
    f32 = dict(device="cuda", dtype=F32)
    s = dict(case=case, logits=logits, tok=tok, temp=temp, lse=torch.empty(B, J, **f32),
             entropy=torch.empty(B, J, **f32), ws=None)
    if case["op"] == "logprobs":
        n = case["top"]
        s.update(logp=torch.empty(B, J, **f32),
                 top_idx=torch.empty(B, J, n, device="cuda", dtype=torch.int32) if n else None,
                 top_logp=torch.empty(B, J, n, **f32) if n else None)
        return s
    s.update(g_logp=_normal(g, B, J) / _rows(case),
             g_entropy=torch.full((B, J), -0.01 / _rows(case), **f32) if case["entropy"] else None,
             dlogits=torch.empty_like(logits))
    for b0 in range(0, B, 16):  # what the forward call left for the backward one
        x = logits[b0:b0 + 16].double() / temp[b0:b0 + 16, None, None].double()
        lse = torch.logsumexp(x, -1)
        s["lse"][b0:b0 + 16] = lse.float()
        s["entropy"][b0:b0 + 16] = (lse - (torch.exp(x - lse[..., None]) * x).sum(-1)).float()
    return s


def _prepare_norm(case, g):
    M, H, dtype = case["M"], case["H"], TYPES[case["dtype"]]
    # a residual stream: a few channels carry far larger values than the others
    channel = torch.exp(_normal(g, H, std=0.5))
    channel[torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")] *= 20
    weight = (1 + _normal(g, H, std=0.1)).to(dtype)
    x = (_normal(g, M, H) * channel).to(dtype)
    s = dict(case=case, weight=weight, ws=None)
    if case["op"] == "norm":
        e4m3 = case["out"] == "e4m3"
        s.update(x=x, delta=(_normal(g, M, H, std=0.5) * channel).to(dtype), sum=torch.empty_like(x),
                 y=torch.empty(M, H, device="cuda", dtype=E4M3 if e4m3 else dtype),
                 y_scale=torch.empty(M, device="cuda", dtype=F32) if e4m3 else None,
                 rstd=torch.empty(M, device="cuda", dtype=F32))
        return s
    s.update(s=x, rstd=torch.rsqrt(x.double().square().mean(1) + EPS).float(), dy=_normal(g, M, H, std=0.01, dtype=dtype),
             dsum=_normal(g, M, H, std=0.01, dtype=dtype), dx=torch.empty_like(x),
             dweight=torch.empty(H, device="cuda", dtype=F32))
    return s


def _prepare_linear(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    e4m3 = case.get("type") == "e4m3"

    def factor(rows, std):
        v = torch.empty(rows, K, device="cuda", dtype=E4M3 if e4m3 else BF16)
        scale = torch.empty(rows, device="cuda", dtype=F32) if e4m3 else None
        for r0 in range(0, rows, 16384):
            part = _normal(g, min(16384, rows - r0), K, std=std)
            if e4m3:  # as a checkpoint holds them: each row over its largest value
                scale[r0:r0 + 16384] = part.abs().amax(1) / E4M3_MAX
                part = part / scale[r0:r0 + 16384, None]
            v[r0:r0 + 16384] = part.to(v.dtype)
        return v, scale

    x, x_scale = factor(M, 1.0)
    w, w_scale = factor(N, K ** -0.5)
    s = dict(case=case, x=x, w=w, x_scale=x_scale, w_scale=w_scale, ws=None)
    if case["op"] == "linear":
        s.update(bias=_normal(g, N, std=0.5) if case["bias"] else None,
                 residual=_normal(g, M, N, dtype=BF16) if case["residual"] else None,
                 y=torch.empty(M, N, device="cuda", dtype=BF16))
        return s
    s.update(dy=_normal(g, M, N, std=0.01, dtype=BF16),
             pre=_normal(g, M, N, dtype=BF16) if case["act"] != "none" else None,
             dx=torch.empty_like(x), dw=torch.empty_like(w),
             dbias=torch.empty(N, device="cuda", dtype=F32) if case["bias"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"logprobs": _run_logprobs, "logprobs_grad": _run_logprobs_grad, "norm": _run_norm,
            "norm_grad": _run_norm_grad, "linear": _run_linear, "linear_grad": _run_linear_grad}[s["case"]["op"]](s)


def _workspace(s, bn, op, rows, outputs, inputs, dtype):
    """The call's workspace, made once and kept with the state, as a program keeps it."""
    if s["ws"] is None:
        s["ws"] = torch.zeros(bn.workspace_bytes(op, rows, 1, outputs, inputs, dtype), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_logprobs(s):
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        B, J, V = s["logits"].shape
        ws = _workspace(s, bn, bn.OP_LOGPROBS, B * J, V, 0, bn.BF16 if s["logits"].dtype == BF16 else bn.F32)
        bn.token_logprobs(s["logits"], s["tok"], s["temp"], s["logp"], ws, entropy=s["entropy"], lse=s["lse"],
                          top_idx=s["top_idx"], top_logp=s["top_logp"])
        out = {k: s[k] for k in ("logp", "entropy", "lse")}
        if s["top_idx"] is not None:
            out.update(top_idx=s["top_idx"], top_logp=s["top_logp"])
        return out
    valid = s["tok"] >= 0
    x = s["logits"].float() / s["temp"][:, None, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1)
    lse = top[..., 0] + torch.log(total)
    entropy = torch.log(total) - (e * (x - top)).sum(-1) / total
    logp = x.gather(-1, s["tok"].clamp(min=0).long()[..., None])[..., 0] - lse
    zero = torch.zeros_like(lse)
    out = dict(logp=torch.where(valid, logp, zero), entropy=torch.where(valid, entropy, zero),
               lse=torch.where(valid, lse, zero))
    n = s["case"]["top"]
    if n:
        # whole keys in the values' order, the index behind them, so that ties go to the lowest index
        raw = s["logits"].float() + 0.0
        bits = raw.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        V = x.shape[-1]
        key = key * (1 << 24) - torch.arange(V, device=x.device)
        best = key.topk(n, -1).indices
        out["top_idx"] = torch.where(valid[..., None], best, -1).to(torch.int32)
        out["top_logp"] = torch.where(valid[..., None], x.gather(-1, best) - lse[..., None], -math.inf)
    return out


def _run_logprobs_grad(s):
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        B, J, V = s["logits"].shape
        ws = _workspace(s, bn, bn.OP_LOGPROBS, B * J, V, 0, bn.BF16 if s["logits"].dtype == BF16 else bn.F32)
        bn.token_logprobs_grad(s["logits"], s["tok"], s["temp"], s["lse"], s["g_logp"], s["dlogits"], ws,
                               entropy=s["entropy"] if s["g_entropy"] is not None else None, g_entropy=s["g_entropy"])
        return {"dlogits": s["dlogits"]}
    x = s["logits"].float() / s["temp"][:, None, None]
    logp = x - s["lse"][..., None]
    p = torch.exp(logp)
    g = s["g_logp"][..., None]
    d = -g * p
    if s["g_entropy"] is not None:
        d = d - s["g_entropy"][..., None] * p * (logp + s["entropy"][..., None])
    d.scatter_add_(-1, s["tok"].clamp(min=0).long()[..., None], g)
    d = d / s["temp"][:, None, None]
    return {"dlogits": torch.where(s["tok"][..., None] >= 0, d, 0.0).to(s["logits"].dtype)}


def _run_norm(s):
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        ws = _workspace(s, bn, bn.OP_NORM, s["x"].shape[0], s["x"].shape[1], 0, bn.F32)
        bn.residual_norm(s["x"], s["delta"], s["weight"], EPS, s["y"], ws, sum=s["sum"], y_scale=s["y_scale"],
                         rstd=s["rstd"])
        out = {k: s[k] for k in ("sum", "y", "rstd")}
        if s["y_scale"] is not None:
            out["y_scale"] = s["y_scale"]
        return out
    v = s["x"].float() + s["delta"].float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * rstd[:, None] * s["weight"].float()
    out = dict(sum=v.to(s["x"].dtype), rstd=rstd)
    if s["y_scale"] is None:
        out["y"] = y.to(s["y"].dtype)
    else:
        out["y_scale"] = y.abs().amax(1) / E4M3_MAX
        out["y"] = (y / out["y_scale"][:, None]).to(E4M3)
    return out


def _run_norm_grad(s):
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        ws = _workspace(s, bn, bn.OP_NORM, s["s"].shape[0], s["s"].shape[1], 0, bn.F32)
        bn.residual_norm_grad(s["s"], s["weight"], s["rstd"], s["dy"], s["dx"], ws, dsum=s["dsum"], dweight=s["dweight"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    v, r = s["s"].float(), s["rstd"][:, None]
    dy = s["dy"].float()
    wd = dy * s["weight"].float()
    dx = s["dsum"].float() + r * (wd - v * r * r * (wd * v).mean(1, keepdim=True))
    return {"dx": dx.to(s["dx"].dtype), "dweight": (dy * v * r).sum(0)}


def _run_linear(s):
    case = s["case"]
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        M, K = s["x"].shape
        ws = _workspace(s, bn, bn.OP_LINEAR, M, s["w"].shape[0], K, bn.BF16 if s["x_scale"] is None else bn.E4M3)
        bn.linear(s["x"], s["w"], s["y"], ws, x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"],
                  residual=s["residual"], act=case["act"])
        return {"y": s["y"]}
    y = s["x"].float() @ s["w"].float().t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] == "relu":
        y = y.clamp(min=0)
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(BF16)}


def _run_linear_grad(s):
    case = s["case"]
    if own:
        from speculative_decoding_draft_sample_b200 import binding as bn
        M, K = s["x"].shape
        ws = _workspace(s, bn, bn.OP_LINEAR, M, s["w"].shape[0], K, bn.BF16)
        bn.linear_grad(s["x"], s["w"], s["dy"], ws, dx=s["dx"], dw=s["dw"], dbias=s["dbias"], pre=s["pre"],
                       act=case["act"])
    else:
        d = s["dy"].float()
        if case["act"] == "relu":
            d = d * (s["pre"] > 0)
        elif case["act"] == "silu":
            z = s["pre"].float()
            sig = 1 / (1 + torch.exp(-z))
            d = d * sig * (1 + z * (1 - sig))
        elif case["act"] == "gelu":
            z = s["pre"].float()
            c = math.sqrt(2 / math.pi)
            t = torch.tanh(c * (z + 0.044715 * z * z * z))
            d = d * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
        dx, dw = d @ s["w"].float(), d.t() @ s["x"].float()
    out = dict(dx=s["dx"], dw=s["dw"]) if own else dict(dx=dx.to(BF16), dw=dw.to(BF16))
    if s["dbias"] is not None:
        out["dbias"] = s["dbias"] if own else d.sum(0)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("logprobs", "logprobs_grad"):
        es = 4 if case["dtype"] == "f32" else 2
        rows, every = _rows(case), case["B"] * case["J"]
        if op == "logprobs":  # a weight and two sums an entry
            return dict(bytes=rows * case["V"] * es + every * (16 + 8 * case["top"]), flops=6 * rows * case["V"])
        return dict(bytes=(rows + every) * case["V"] * es + every * 16, flops=6 * rows * case["V"])
    if op in ("norm", "norm_grad"):
        M, H, es = case["M"], case["H"], 4 if case["dtype"] == "f32" else 2
        if op == "norm":
            out = 1 if case["out"] == "e4m3" else es
            return dict(bytes=M * H * (3 * es + out) + H * es + M * 8, flops=6 * M * H)
        return dict(bytes=M * H * 4 * es + H * (es + 4) + M * 4, flops=10 * M * H)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear":
        es = 1 if case["type"] == "e4m3" else 2
        scales = 4 * (M + N) if es == 1 else 0
        return dict(bytes=(M + N) * K * es + scales + M * N * 2 * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
                    flops=2 * M * N * K)
    return dict(bytes=2 * (2 * M * K + 2 * N * K) + M * N * 2 * (1 if case["act"] == "none" else 2) +
                (4 * N if case["bias"] else 0), flops=4 * M * N * K)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "logprobs":
        got = {k: [] for k in ("logp", "entropy", "lse", "top_logp")}
        for b in range(case["B"]):
            keep = (s["tok"][b] >= 0)[:, None]
            d = torch.log_softmax(s["logits"][b].to(f64) / s["temp"][b].to(f64), -1)
            token = s["tok"][b].long().clamp(min=0)[:, None]
            got["logp"].append((d.gather(1, token) * keep)[:, 0])
            got["entropy"].append((torch.special.entr(d.exp()).sum(1, keepdim=True) * keep)[:, 0])
            scaled = s["logits"][b].to(f64) / s["temp"][b].to(f64)
            got["lse"].append((torch.logsumexp(scaled, 1, keepdim=True) * keep)[:, 0])
            if case["top"]:
                best = torch.sort(d, 1, descending=True).values[:, :case["top"]]
                got["top_logp"].append(best.masked_fill(~keep, -math.inf))
        out = {k: torch.stack(v) for k, v in got.items() if v}
        if case["top"]:
            out["top_idx"] = None
        return out
    if op == "logprobs_grad":
        d = torch.empty(s["logits"].shape, dtype=f64, device="cuda")
        for b in range(case["B"]):
            z = s["logits"][b].to(f64).requires_grad_()
            logp = torch.log_softmax(z / s["temp"][b].to(f64), -1)
            keep = s["tok"][b] >= 0
            loss = (logp.gather(1, s["tok"][b].long().clamp(min=0)[:, None])[:, 0] * s["g_logp"][b].to(f64))[keep].sum()
            if s["g_entropy"] is not None:
                entropy = -(logp.exp() * logp).sum(1)
                loss = loss + (entropy * s["g_entropy"][b].to(f64))[keep].sum()
            d[b] = torch.autograd.grad(loss, z)[0]
        return {"dlogits": d}
    if op == "norm":
        v = s["x"].to(f64) + s["delta"].to(f64)
        rms = torch.sqrt((v ** 2).sum(1) / case["H"] + EPS)
        y = v / rms[:, None] * s["weight"].to(f64)
        out = dict(sum=v, rstd=1 / rms, y=y)
        if case["out"] == "e4m3":
            out["y_scale"] = y.abs().max(1).values / E4M3_MAX
            out["y"] = (y / out["y_scale"][:, None]).float().to(E4M3).to(f64)
        return out
    if op == "norm_grad":
        v = s["s"].to(f64).requires_grad_()
        w = s["weight"].to(f64).requires_grad_()
        y = v / torch.sqrt((v ** 2).mean(1, keepdim=True) + EPS) * w
        dv, dw = torch.autograd.grad((y * s["dy"].to(f64)).sum() + (v * s["dsum"].to(f64)).sum(), (v, w))
        return {"dx": dv, "dweight": dw}
    act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
           "gelu": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
    if op == "linear":
        y = torch.empty(case["M"], case["N"], dtype=f64, device="cuda")
        x = s["x"].float().to(f64)
        for n0 in range(0, case["N"], 16384):
            z = x @ s["w"][n0:n0 + 16384].float().to(f64).t()
            if case["type"] == "e4m3":
                z = z * torch.outer(s["x_scale"].to(f64), s["w_scale"][n0:n0 + 16384].to(f64))
            z = act(z + s["bias"][n0:n0 + 16384].to(f64) if case["bias"] else z)
            y[:, n0:n0 + 16384] = z + s["residual"][:, n0:n0 + 16384].to(f64) if case["residual"] else z
        return {"y": y}
    pre = (torch.zeros_like(s["dy"]) if s["pre"] is None else s["pre"]).to(f64).requires_grad_()
    d = torch.autograd.grad((act(pre) * s["dy"].to(f64)).sum(), pre)[0]
    out = dict(dx=d @ s["w"].to(f64), dw=d.t() @ s["x"].to(f64))
    if case["bias"]:
        out["dbias"] = d.sum(0)
    return out
