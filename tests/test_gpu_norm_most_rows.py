"""The norm of as many rows as a C int counts: the first and the last ones against the same rows
alone (a row does not depend on the others)."""
import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("M", [2 ** 31 - 1])
def test_most_rows(cuda_ok, M):
    H, n = 8, 4099
    x_bytes = M * H * 2
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * x_bytes + M * 4 + (4 << 30):
        pytest.skip("needs 82 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    ends = [torch.randn(n, H, generator=g, device="cuda").to(BF16) for _ in range(2)]
    weight = torch.randn(H, generator=g, device="cuda").to(BF16)
    ws = torch.zeros(bn.workspace_bytes(bn.OP_NORM, M, 0, H, 0, 0), dtype=torch.uint8, device="cuda")
    x = torch.zeros(M, H, device="cuda", dtype=BF16)
    y, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    x[:n], x[-n:] = ends
    bn.residual_norm(x, None, weight, 1e-6, y, ws, rstd=rstd)
    assert bn.read_status(ws) == (0, -1)
    alone_y, alone_rstd = torch.empty(n, H, device="cuda", dtype=BF16), torch.empty(n, device="cuda")
    for part, rows in zip(ends, (slice(0, n), slice(M - n, M))):
        bn.residual_norm(part, None, weight, 1e-6, alone_y, ws, rstd=alone_rstd)
        assert torch.equal(y[rows], alone_y) and torch.equal(rstd[rows], alone_rstd)
    bn.residual_norm_grad(x, weight, rstd, y, y, ws)  # in dy's place
    alone_dx = torch.empty_like(alone_y)
    for part, rows in zip(ends, (slice(0, n), slice(M - n, M))):
        bn.residual_norm(part, None, weight, 1e-6, alone_y, ws, rstd=alone_rstd)
        bn.residual_norm_grad(part, weight, alone_rstd, alone_y, alone_dx, ws)
        assert torch.equal(y[rows], alone_dx)
    del x, y, rstd
    torch.cuda.empty_cache()
