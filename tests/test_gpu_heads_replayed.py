"""A head whose runs are in graphs: the replays, not the order of capture, decide what a gradient
is made of."""
import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn
from speculative_decoding_draft_sample_b200.heads import LogitHead

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_gradient_after_a_replay_of_another_run(cuda_ok):
    V, H = 512, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    norm_w = torch.ones(H, device="cuda", dtype=BF16)
    w = (torch.randn(V, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    data = {m: (torch.randn(m, H, generator=g, device="cuda").to(BF16), torch.randn(m, V, generator=g, device="cuda").to(BF16))
            for m in (4, 8)}

    def gradient(head, m):
        dx = torch.empty(m, H, device="cuda", dtype=BF16)
        head.gradient(data[m][1], dx)
        return dx

    plain, want = LogitHead(norm_w, w, 8), {}
    for m, (x, _) in data.items():
        plain.run(x, torch.empty(m, V, device="cuda", dtype=BF16))
        want[m] = gradient(plain, m)
    with pytest.raises(bn.DSparkError, match="after a run of 8"):
        gradient(plain, 4)
    head, graphs = LogitHead(norm_w, w, 8), {}
    for m, (x, _) in data.items():
        logits = torch.empty(m, V, device="cuda", dtype=BF16)
        graphs[m] = (torch.cuda.CUDAGraph(), logits)
        with torch.cuda.graph(graphs[m][0]):
            head.run(x, logits)
    for m in (4, 8, 4):
        graphs[m][0].replay()
        assert torch.equal(gradient(head, m), want[m])
    assert head.status() == (0, -1)
