"""What stands directly before and behind a round: the logit head and the token scores.

``LogitHead`` turns a model's last hidden states into the logits a round takes
(residual addition, root-mean-square norm, product with the output embedding), with
bfloat16 weights or with 8-bit ones; ``TokenScores`` returns the log probabilities of
the tokens a round emitted, their rows' entropies and most likely alternatives. Both
own their output buffers and workspaces and issue C-ABI calls on one stream, forward
and, for training against a target, backward.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as bn

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def quantize_rows(w: torch.Tensor, chunk: int = 8192) -> Tuple[torch.Tensor, torch.Tensor]:
    """A weight matrix [N, K] as float8_e4m3fn with one scale per row (its largest value
    over 448), the layout LogitHead takes; done once, when the weights are loaded."""
    q = torch.empty(w.shape, dtype=E4M3, device=w.device)
    scale = torch.empty((w.shape[0],), dtype=torch.float32, device=w.device)
    for r in range(0, w.shape[0], chunk):
        part = w[r:r + chunk].float()
        s = (part.abs().amax(1) / E4M3_MAX).clamp(min=MIN_SCALE)
        scale[r:r + chunk] = s
        q[r:r + chunk] = (part / s[:, None]).to(E4M3)
    return q, scale


def _width(t: torch.Tensor) -> int:
    """Entries of a row: the last dimension, which a head never spreads over rows."""
    return t.shape[-1] if t.dim() else -1


class LogitHead:
    """logits = norm(hidden + delta) @ weight^T (+ bias) for up to ``rows`` rows.

    norm_weight [H] bfloat16; weight [V, H] bfloat16, or float8_e4m3fn with w_scale [V]
    (the norm then writes e4m3 with a scale per row, and the product takes 8-bit operands);
    bias [V] float32 or None. ``run`` leaves what ``gradient`` needs (bfloat16 weights).
    """

    def __init__(self, norm_weight: torch.Tensor, weight: torch.Tensor, rows: int,
                 w_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 eps: float = 1e-6):
        V, H = weight.shape
        dev = weight.device
        if weight.dtype not in (torch.bfloat16, E4M3):
            raise bn.DSparkError(f"the head's weight must be bfloat16 or float8_e4m3fn, got {weight.dtype}")
        if (weight.dtype == E4M3) != (w_scale is not None):
            raise bn.DSparkError("w_scale goes with a float8_e4m3fn weight")
        if tuple(norm_weight.shape) != (H,):
            raise bn.DSparkError(f"norm_weight must have shape {(H,)}, got {tuple(norm_weight.shape)}")
        self.norm_weight, self.weight, self.w_scale, self.bias, self.eps = norm_weight, weight, w_scale, bias, eps
        self.rows, self.V, self.H = rows, V, H
        self.e4m3 = weight.dtype == E4M3
        code = bn.E4M3 if self.e4m3 else bn.BF16
        sizes = [bn.workspace_bytes(bn.OP_NORM, rows, 0, H, 0, 0), bn.workspace_bytes(bn.OP_LINEAR, rows, 0, V, H, code)]
        if 0 in sizes:
            raise bn.DSparkError(f"unsupported head: {rows} rows, H={H}, V={V}, {weight.dtype}")
        if not self.e4m3:  # the backward call without an activation (the head has none)
            sizes.append(bn.workspace_bytes(bn.OP_LINEAR, rows, 2, V, H, code))
        self.ws = torch.zeros((max(sizes),), dtype=torch.uint8, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self.sum = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((rows, H), dtype=weight.dtype, device=dev)
        self.y_scale = torch.empty((rows,), **f32) if self.e4m3 else None
        self.rstd = torch.empty((rows,), **f32)
        self._ran = 0  # rows of the run whose y, sum and rstd the buffers hold
        self._captured = False  # a run is in a graph: which one was the last, its replays decide

    def run(self, hidden: torch.Tensor, logits: torch.Tensor, delta: Optional[torch.Tensor] = None, stream=None) -> None:
        """hidden, delta [..., H] bfloat16 -> logits [..., V] (bfloat16 or float32); the summed
        residual stream stays in ``sum``."""
        rows_fit = _width(hidden) == self.H and _width(logits) == self.V and (delta is None or _width(delta) == self.H)
        x = hidden.reshape(-1, self.H) if rows_fit and hidden.is_contiguous() else hidden
        M = x.shape[0] if x.dim() == 2 else -1
        if not rows_fit or not 1 <= M <= self.rows or logits.numel() != M * self.V:
            shapes = f"hidden {tuple(hidden.shape)}" + (f", delta {tuple(delta.shape)}" if delta is not None else "")
            raise bn.DSparkError(f"{shapes} and logits {tuple(logits.shape)} do not fit a head of "
                                 f"{self.rows} rows, H={self.H}, V={self.V}")
        d = delta.reshape(-1, self.H) if delta is not None and delta.is_contiguous() else delta
        y, y_scale = self.y[:M], self.y_scale[:M] if self.e4m3 else None
        self._ran = 0
        self._captured = self._captured or (x.is_cuda and torch.cuda.is_current_stream_capturing())
        bn.residual_norm(x, d, self.norm_weight, self.eps, y, self.ws, sum=self.sum[:M], y_scale=y_scale,
                         rstd=self.rstd[:M], stream=stream)
        out = logits.view(M, self.V) if logits.is_contiguous() else logits
        bn.linear(y, self.weight, out, self.ws, x_scale=y_scale, w_scale=self.w_scale, bias=self.bias,
                  stream=stream)
        self._ran = M

    def gradient(self, dlogits: torch.Tensor, dhidden: torch.Tensor, dweight: Optional[torch.Tensor] = None,
                 dbias: Optional[torch.Tensor] = None, dnorm_weight: Optional[torch.Tensor] = None, stream=None) -> None:
        """The gradients of the last ``run``, whose rows these must be (a run of another batch in
        between replaces what they are made of; after a captured run, whose replays are not seen
        here, that is the caller's to keep): dlogits [..., V] bfloat16 -> dhidden [..., H]
        (hidden's and delta's alike), and where given dweight [V, H], dbias [V] and
        dnorm_weight [H] f32. Frozen weights are left out and cost nothing."""
        if self.e4m3:
            raise bn.DSparkError("an 8-bit head has no gradient")
        rows_fit = _width(dlogits) == self.V and _width(dhidden) == self.H
        dl = dlogits.reshape(-1, self.V) if rows_fit and dlogits.is_contiguous() else dlogits
        M = dl.shape[0] if dl.dim() else -1
        if not rows_fit or not 1 <= M <= self.rows or dhidden.numel() != M * self.H:
            raise bn.DSparkError(f"dlogits {tuple(dlogits.shape)} and dhidden {tuple(dhidden.shape)} do not fit the head")
        if M != self._ran and not self._captured:
            raise bn.DSparkError(f"gradient of {M} rows after a run of {self._ran}")
        dx = dhidden.view(M, self.H) if dhidden.is_contiguous() else dhidden
        # dx holds the gradient of the norm's output between the two calls
        bn.linear_grad(self.y[:M], self.weight, dl, self.ws, dx=dx, dw=dweight, dbias=dbias, stream=stream)
        bn.residual_norm_grad(self.sum[:M], self.norm_weight, self.rstd[:M], dx, dx, self.ws, dweight=dnorm_weight,
                              stream=stream)

    def status(self, stream=None) -> Tuple[int, int]:
        """(status bits, first offending row or -1) of the calls since the last status()."""
        return bn.read_status(self.ws, stream)


class TokenScores:
    """Log probabilities of given tokens, entropies and the n_top most likely alternatives
    of [B, J, V] logit rows; tokens of -1 are padding, as a round's ``out`` carries it."""

    def __init__(self, B: int, J: int, V: int, n_top: int = 0, dtype: torch.dtype = torch.bfloat16,
                 device: str = "cuda"):
        dev = torch.device(device)
        code = bn.F32 if dtype == torch.float32 else bn.BF16
        nbytes = bn.workspace_bytes(bn.OP_LOGPROBS, B, J, V, 0, code)
        if nbytes == 0 or not 0 <= n_top <= min(32, V):
            raise bn.DSparkError(f"unsupported scores: B={B} J={J} V={V} n_top={n_top}")
        f32 = dict(dtype=torch.float32, device=dev)
        self.logp = torch.empty((B, J), **f32)
        self.entropy = torch.empty((B, J), **f32)
        self.lse = torch.empty((B, J), **f32)
        self.top_idx = torch.empty((B, J, n_top), dtype=torch.int32, device=dev) if n_top else None
        self.top_logp = torch.empty((B, J, n_top), **f32) if n_top else None
        self.ws = torch.zeros((nbytes,), dtype=torch.uint8, device=dev)

    def run(self, logits: torch.Tensor, tok: torch.Tensor, temp: Optional[torch.Tensor], stream=None) -> None:
        bn.token_logprobs(logits, tok, temp, self.logp, self.ws, entropy=self.entropy, lse=self.lse,
                          top_idx=self.top_idx, top_logp=self.top_logp, stream=stream)

    def gradient(self, logits: torch.Tensor, tok: torch.Tensor, temp: Optional[torch.Tensor], g_logp: torch.Tensor,
                 dlogits: torch.Tensor, g_entropy: Optional[torch.Tensor] = None, stream=None) -> None:
        """dlogits (which may be logits) of sum g_logp logp + g_entropy entropy, after ``run`` on the same arguments."""
        bn.token_logprobs_grad(logits, tok, temp, self.lse, g_logp, dlogits, self.ws,
                               entropy=self.entropy if g_entropy is not None else None, g_entropy=g_entropy,
                               stream=stream)

    def status(self, stream=None) -> Tuple[int, int]:
        return bn.read_status(self.ws, stream)
