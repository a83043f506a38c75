"""The heads' launches overlap: what one writes (row scales, rstd, sums) the next one reads, in
buffers that every pass writes anew. Many passes with different rows, nothing between them, give
what each gives alone."""
import pytest
import torch

from speculative_decoding_draft_sample_b200.heads import LogitHead, quantize_rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("M,V,H", [(1, 264, 256), (6, 1000, 512), (300, 2048, 1536)])
def test_passes_in_a_row(cuda_ok, M, V, H, e4m3):
    g = torch.Generator(device="cuda").manual_seed(M)
    norm_w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    w = (torch.randn(V, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    bias = torch.zeros(V, device="cuda")
    q, scale = quantize_rows(w) if e4m3 else (w, None)
    head = LogitHead(norm_w, q, M, w_scale=scale, bias=bias)
    n = 12                                   # each pass's rows at another scale, its bias another value
    xs = [(torch.randn(M, H, generator=g, device="cuda") * 2.0 ** (i - n // 2)).to(BF16) for i in range(n)]
    dl = [torch.randn(M, V, generator=g, device="cuda").to(BF16) for _ in range(n)]

    def passes(sync):
        got = []
        for i in range(n):
            logits, dx = torch.empty(M, V, device="cuda", dtype=BF16), torch.empty(M, H, device="cuda", dtype=BF16)
            dw, dn = torch.empty_like(w), torch.empty(H, device="cuda")
            bias.fill_(float(i))
            sync()
            head.run(xs[i], logits)
            sync()
            got.append(logits)
            if not e4m3:
                head.gradient(dl[i], dx, dweight=dw, dnorm_weight=dn)
                sync()
                got += [dx, dw, dn]
        torch.cuda.synchronize()
        return got

    want = passes(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(passes(lambda: None), want):
            assert torch.equal(a, b)
    assert head.status() == (0, -1)
