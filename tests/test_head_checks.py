"""Refusals of the logit-head and token-score calls, before anything reaches a device: the
binding's shape, type and pairing checks, and the C entry points' argument errors."""
import ctypes

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn
from speculative_decoding_draft_sample_b200 import build

B, J, V = 3, 4, 64
bf, f32, i32, e4 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bn.lib()


def score_args(**over):
    a = dict(logits=torch.zeros(B, J, V, dtype=bf), tok=torch.zeros(B, J, dtype=i32), temp=torch.ones(B),
             logp=torch.zeros(B, J), ws=torch.zeros(256, dtype=torch.uint8))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(logits=torch.zeros(B, J, V, dtype=torch.float16)), "unsupported logit dtype"),
    (dict(logits=torch.zeros(B, V, J, dtype=bf).transpose(1, 2)), "logits must be contiguous"),
    (dict(tok=torch.zeros(B, J, dtype=torch.int64)), "tok must be"),
    (dict(tok=torch.zeros(B, J - 1, dtype=i32)), "tok must have shape"),
    (dict(temp=torch.ones(B, J)), "temp must have shape"),
    (dict(logp=torch.zeros(B, J, dtype=bf)), "logp must be"),
    (dict(entropy=torch.zeros(B)), "entropy must have shape"),
    (dict(lse=torch.zeros(B, J, device="meta")), "lse is on meta"),
    (dict(top_idx=torch.zeros(B, J, 5, dtype=i32)), "go together"),
    (dict(top_idx=torch.zeros(B, J, dtype=i32), top_logp=torch.zeros(B, J)), "top_idx must have shape"),
    (dict(top_idx=torch.zeros(B, J, 5, dtype=i32), top_logp=torch.zeros(B, J, 4)), "top_logp must have shape"),
    (dict(top_idx=torch.zeros(B, J, 5, dtype=torch.int64), top_logp=torch.zeros(B, J, 5)), "top_idx must be"),
    ({}, "must be CUDA tensors"),
])
def test_token_logprobs_checks(over, msg):
    with pytest.raises(bn.DSparkError, match=msg):
        bn.token_logprobs(**score_args(**over))


@pytest.mark.parametrize("over,msg", [
    (dict(lse=torch.zeros(B)), "lse must have shape"),
    (dict(g_logp=torch.zeros(B, J, dtype=bf)), "g_logp must be"),
    (dict(dlogits=torch.zeros(B, J, V)), "dlogits must be"),
    (dict(entropy=torch.zeros(B, J)), "go together"),
    (dict(g_entropy=torch.zeros(B, J)), "go together"),
    ({}, "must be CUDA tensors"),
])
def test_token_logprobs_grad_checks(over, msg):
    a = score_args(lse=torch.zeros(B, J), g_logp=torch.zeros(B, J), dlogits=torch.zeros(B, J, V, dtype=bf))
    del a["logp"]
    a.update(over)
    with pytest.raises(bn.DSparkError, match=msg):
        bn.token_logprobs_grad(**a)


M, H = 5, 64


@pytest.mark.parametrize("over,msg", [
    (dict(delta=torch.zeros(M, H)), "delta must be"),
    (dict(delta=torch.zeros(1, H, dtype=bf).expand(M, H)), "delta must be contiguous"),
    (dict(weight=torch.zeros(H)), "weight must be"),
    (dict(weight=torch.zeros(H - 8, dtype=bf)), "weight must have shape"),
    (dict(sum=torch.zeros(M, H)), "sum must be"),
    (dict(y=torch.zeros(M, H)), "y must be"),
    (dict(y=torch.zeros(M, H, dtype=e4)), "y_scale goes with"),
    (dict(y_scale=torch.zeros(M)), "y_scale goes with"),
    (dict(rstd=torch.zeros(M, 1)), "rstd must have shape"),
    (dict(x=torch.zeros(M, H, dtype=torch.float16), weight=torch.zeros(H, dtype=torch.float16), delta=None,
          y=torch.zeros(M, H, dtype=torch.float16)), "unsupported logit dtype"),
    ({}, "must be CUDA tensors"),
])
def test_residual_norm_checks(over, msg):
    a = dict(x=torch.zeros(M, H, dtype=bf), delta=torch.zeros(M, H, dtype=bf), weight=torch.zeros(H, dtype=bf), eps=1e-6,
             y=torch.zeros(M, H, dtype=bf), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    with pytest.raises(bn.DSparkError, match=msg):
        bn.residual_norm(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(dy=torch.zeros(M, H)), "dy must be"),
    (dict(rstd=torch.zeros(M + 1)), "rstd must have shape"),
    (dict(dsum=torch.zeros(M, H, 1, dtype=bf)), "dsum must have shape"),
    (dict(dweight=torch.zeros(H, dtype=bf)), "dweight must be"),
    ({}, "must be CUDA tensors"),
])
def test_residual_norm_grad_checks(over, msg):
    a = dict(s=torch.zeros(M, H, dtype=bf), weight=torch.zeros(H, dtype=bf), rstd=torch.zeros(M),
             dy=torch.zeros(M, H, dtype=bf), dx=torch.zeros(M, H, dtype=bf), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    with pytest.raises(bn.DSparkError, match=msg):
        bn.residual_norm_grad(**a)


N, K = 24, 32


@pytest.mark.parametrize("over,msg", [
    (dict(x=torch.zeros(M, K)), "x must be bfloat16"),
    (dict(w=torch.zeros(N, K + 8, dtype=bf)), "w must have shape"),
    (dict(w=torch.zeros(K, N, dtype=bf).t()), "w must be contiguous"),
    (dict(w=torch.zeros(N, K, dtype=e4)), "w must be"),
    (dict(x_scale=torch.zeros(M)), "go with float8"),
    (dict(x=torch.zeros(M, K, dtype=e4), w=torch.zeros(N, K, dtype=e4)), "go with float8"),
    (dict(x=torch.zeros(M, K, dtype=e4), w=torch.zeros(N, K, dtype=e4), x_scale=torch.zeros(M), w_scale=torch.zeros(1)),
     "w_scale must have shape"),
    (dict(bias=torch.zeros(N, dtype=bf)), "bias must be"),
    (dict(residual=torch.zeros(M, N)), "residual must be"),
    (dict(y=torch.zeros(M, N, dtype=torch.float16)), "unsupported logit dtype"),
    (dict(y=torch.zeros(M, N + 1, dtype=bf)), "y must have shape"),
    (dict(pre=torch.zeros(M, N)), "pre must be"),
    (dict(act="swish"), "unknown activation"),
    ({}, "must be CUDA tensors"),
])
def test_linear_checks(over, msg):
    a = dict(x=torch.zeros(M, K, dtype=bf), w=torch.zeros(N, K, dtype=bf), y=torch.zeros(M, N, dtype=bf),
             ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    with pytest.raises(bn.DSparkError, match=msg):
        bn.linear(**a)


@pytest.mark.parametrize("over,msg", [
    (dict(x=torch.zeros(M, K, dtype=e4)), "x must be"),
    (dict(dy=torch.zeros(M, N)), "dy must be"),
    (dict(dw=torch.zeros(N, K)), "dw must be"),
    (dict(dbias=torch.zeros(N, dtype=bf)), "dbias must be"),
    (dict(pre=torch.zeros(M, dtype=bf)), "pre must have shape"),
    ({}, "must be CUDA tensors"),
])
def test_linear_grad_checks(over, msg):
    a = dict(x=torch.zeros(M, K, dtype=bf), w=torch.zeros(N, K, dtype=bf), dy=torch.zeros(M, N, dtype=bf),
             dx=torch.zeros(M, K, dtype=bf), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    with pytest.raises(bn.DSparkError, match=msg):
        bn.linear_grad(**a)


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -4


def test_entry_points_refuse_before_any_device_call(lib):
    z = ctypes.c_void_p(0)
    a, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)  # never followed: each call below is refused
    score = lambda *o: lib.dspark_token_logprobs(*o)  # noqa: E731
    assert score(z, a, z, 2, 2, 64, 1, 0, a, z, z, z, z, a, 256, z) == INVALID
    assert score(odd, a, z, 2, 2, 64, 1, 0, a, z, z, z, z, a, 256, z) == INVALID
    assert score(a, a, z, 2, 2, 60, 1, 0, a, z, z, z, z, a, 256, z) == INVALID      # V % 8
    assert score(a, a, z, 2, 65, 64, 1, 0, a, z, z, z, z, a, 256, z) == INVALID     # J > 64
    assert score(a, a, z, 0, 2, 64, 1, 0, a, z, z, z, z, a, 256, z) == INVALID      # no rows
    assert score(a, a, z, 2, 2, 64, 2, 0, a, z, z, z, z, a, 256, z) == INVALID      # e4m3 logits
    assert score(a, a, z, 2, 2, 64, 1, 33, a, z, z, a, a, a, 256, z) == INVALID     # n_top > 32
    assert score(a, a, z, 2, 2, 8, 1, 9, a, z, z, a, a, a, 256, z) == INVALID       # n_top > V
    assert score(a, a, z, 2, 2, 64, 1, -1, a, z, z, a, a, a, 256, z) == INVALID
    assert score(a, a, z, 2, 2, 64, 1, 4, a, z, z, z, z, a, 256, z) == INVALID      # alternatives without outputs
    assert score(a, a, z, 2, 2, 64, 1, 0, a, z, z, z, z, a, 255, z) == WORKSPACE
    sgrad = lib.dspark_token_logprobs_grad
    assert sgrad(a, a, z, a, z, a, a, 2, 2, 64, 1, a, a, 256, z) == INVALID         # g_entropy without entropy
    assert sgrad(a, a, z, a, z, a, z, 2, 2, 64, 1, odd, a, 256, z) == INVALID
    assert sgrad(a, a, z, z, z, a, z, 2, 2, 64, 1, a, a, 256, z) == INVALID
    big = 1 << 40
    norm = lib.dspark_residual_norm
    assert norm(a, z, a, 2, 60, 1, 1e-6, z, a, 1, z, z, a, big, z) == INVALID       # H % 8
    assert norm(a, z, a, 2, 16392, 1, 1e-6, z, a, 1, z, z, a, big, z) == INVALID
    assert norm(a, z, a, 0, 64, 1, 1e-6, z, a, 1, z, z, a, big, z) == INVALID
    assert norm(a, z, a, 2, 64, 1, -1.0, z, a, 1, z, z, a, big, z) == INVALID       # eps < 0
    assert norm(a, z, a, 2, 64, 1, float("nan"), z, a, 1, z, z, a, big, z) == INVALID
    assert norm(a, z, a, 2, 64, 1, 1e-6, z, a, 0, z, z, a, big, z) == UNSUPPORTED   # f32 from bf16
    assert norm(a, z, a, 2, 64, 1, 1e-6, z, a, 2, z, z, a, big, z) == INVALID       # e4m3 without scales
    assert norm(a, odd, a, 2, 64, 1, 1e-6, z, a, 1, z, z, a, big, z) == INVALID
    assert norm(a, z, a, 2, 64, 1, 1e-6, z, a, 1, z, z, a, 256, z) == WORKSPACE
    ngrad = lib.dspark_residual_norm_grad
    assert ngrad(a, a, z, a, z, 2, 64, 1, a, z, a, big, z) == INVALID
    assert ngrad(a, a, a, a, z, 2, 64, 1, a, z, a, 256, z) == WORKSPACE
    lin = lib.dspark_linear
    assert lin(a, a, z, z, z, z, 2, 8, 60, 1, 1, 0, a, z, a, big, z) == INVALID     # K % 8
    assert lin(a, a, a, a, z, z, 2, 8, 72, 2, 1, 0, a, z, a, big, z) == INVALID     # e4m3 K % 16
    assert lin(a, a, a, z, z, z, 2, 8, 64, 2, 1, 0, a, z, a, big, z) == INVALID     # one scale of two
    assert lin(a, a, a, a, z, z, 2, 8, 64, 1, 1, 0, a, z, a, big, z) == INVALID     # scales with bf16
    assert lin(a, a, z, z, z, z, 2, 8, 64, 0, 1, 0, a, z, a, big, z) == UNSUPPORTED
    assert lin(a, a, z, z, z, z, 2, 8, 64, 1, 2, 0, a, z, a, big, z) == UNSUPPORTED
    assert lin(a, a, z, z, z, z, 2, 8, 64, 1, 1, 4, a, z, a, big, z) == INVALID     # activation
    assert lin(a, a, z, z, z, z, 0, 8, 64, 1, 1, 0, a, z, a, big, z) == INVALID
    assert lin(a, a, z, z, z, z, 2, 8, 64, 1, 0, 0, odd, z, a, big, z) == INVALID   # y not aligned to its type
    assert lin(odd, a, z, z, z, z, 2, 8, 64, 1, 1, 0, a, z, a, big, z) == INVALID
    assert lin(a, a, z, z, z, z, 2, 8, 64, 1, 1, 0, a, z, a, 16, z) == WORKSPACE
    lgrad = lib.dspark_linear_grad
    assert lgrad(a, a, a, z, 2, 12, 64, 0, a, a, a, a, big, z) == INVALID           # N % 8
    assert lgrad(a, a, a, z, 2, 8, 64, 1, a, a, a, a, big, z) == INVALID            # pre missing
    assert lgrad(a, a, a, z, 2, 8, 64, 0, z, z, z, a, big, z) == INVALID            # nothing asked
    assert lgrad(z, a, a, z, 2, 8, 64, 0, z, a, z, a, big, z) == INVALID            # dw without x
    assert lgrad(a, a, a, z, 2, 8, 64, 0, a, z, z, a, 256, z) == WORKSPACE


def test_workspace_sizes(lib):
    assert bn.workspace_bytes(bn.OP_LOGPROBS, 256, 6, 129280, 0, bn.BF16) == 256
    assert bn.workspace_bytes(bn.OP_LOGPROBS, 256, 65, 129280, 0, bn.BF16) == 0
    assert bn.workspace_bytes(bn.OP_NORM, 7, 0, 4096, 0, 0) == 256 + 296 * 4096 * 4
    assert bn.workspace_bytes(bn.OP_NORM, 7, 0, 4100, 0, 0) == 0
    assert bn.workspace_bytes(bn.OP_LINEAR, 7, 0, 100, 4100, bn.BF16) == 0
    assert bn.workspace_bytes(bn.OP_LINEAR, 7, 0, 100, 4096, bn.F32) == 0
    assert bn.workspace_bytes(bn.OP_LINEAR, 1, 0, 1, 16, bn.E4M3) == 256
    assert bn.workspace_bytes(bn.OP_LINEAR, 1536, 0, 129280, 4096, bn.BF16) == 256
    assert bn.workspace_bytes(bn.OP_LINEAR, 1, 1, 8, 16, bn.E4M3) == 256    # no backward call in 8 bits
    assert bn.workspace_bytes(bn.OP_LINEAR, 40, 3, 8, 16, bn.BF16) == 0
    # backward: dpre (with an activation) and column sums of up to ceil(M / 32) runs of rows
    assert bn.workspace_bytes(bn.OP_LINEAR, 40, 2, 256, 16, bn.BF16) == 256 + 2 * 256 * 4
    assert bn.workspace_bytes(bn.OP_LINEAR, 40, 1, 256, 16, bn.BF16) == 256 + 40 * 256 * 2 + 2 * 256 * 4


BIG = 2 ** 32 + 8   # rows that a C int would carry as 8


def test_sizes_past_a_c_int_are_refused():
    def meta(*shape, dtype=bf):
        return torch.empty(*shape, dtype=dtype, device="meta")

    ws = meta(1 << 16, dtype=torch.uint8)
    for call in (
            lambda: bn.residual_norm(meta(BIG, 8), None, meta(8), 1e-6, meta(BIG, 8), ws),
            lambda: bn.residual_norm_grad(meta(BIG, 8), meta(8), meta(BIG, dtype=f32), meta(BIG, 8), meta(BIG, 8), ws),
            lambda: bn.linear(meta(BIG, 8), meta(8, 8), meta(BIG, 8), ws),
            lambda: bn.linear(meta(8, 8), meta(BIG, 8), meta(8, BIG), ws),
            lambda: bn.linear(meta(8, BIG), meta(8, BIG), meta(8, 8), ws),
            lambda: bn.linear_grad(meta(BIG, 8), meta(8, 8), meta(BIG, 8), ws, dw=meta(8, 8)),
            lambda: bn.token_logprobs(meta(BIG, 1, 8), meta(BIG, 1, dtype=i32), None, meta(BIG, 1, dtype=f32), ws),
            lambda: bn.token_logprobs(meta(1, 1, BIG), meta(1, 1, dtype=i32), None, meta(1, 1, dtype=f32), ws),
            lambda: bn.token_logprobs(meta(1, 1, 16), meta(1, 1, dtype=i32), None, meta(1, 1, dtype=f32), ws,
                                      top_idx=meta(1, 1, BIG, dtype=i32), top_logp=meta(1, 1, BIG, dtype=f32)),
            lambda: bn.token_logprobs_grad(meta(BIG, 1, 8), meta(BIG, 1, dtype=i32), None, meta(BIG, 1, dtype=f32),
                                           meta(BIG, 1, dtype=f32), meta(BIG, 1, 8), ws)):
        with pytest.raises(bn.DSparkError, match="2\\*\\*31"):
            call()
    for sizes in ((BIG, 1, 8, 0), (1, BIG, 8, 0), (1, 1, BIG, 0)):
        assert bn.workspace_bytes(bn.OP_LOGPROBS, *sizes, bn.BF16) == 0
    assert bn.workspace_bytes(bn.OP_LINEAR, 8, 0, 8, BIG, bn.BF16) == 0
