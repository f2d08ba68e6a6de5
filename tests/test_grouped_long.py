"""A launch whose waits are longer than the limit of a single pipeline step (2 s)."""
import pytest
import torch

CUDA = "cuda"


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


@pytest.mark.gpu
def test_weight_gradient_whose_reduction_takes_seconds(B):
    """75 groups on 74 pairs, the first with 640 million rows (a multiple of 64), the last with 5: the
    same pair takes both, at about 0.24 us for 64 rows. The epilogue waits for the first tile's
    reduction and the warp that clears the lines behind a partial block for the second tile."""
    n = 640_000_000
    x = torch.zeros(n + 5, 8, dtype=torch.bfloat16, device=CUDA)
    some = torch.tensor([0, 1, 63, 64, 123_456_789, n - 64, n - 1], device=CUDA)
    x[some] = torch.arange(1, 57, dtype=torch.bfloat16, device=CUDA).view(7, 8)
    x[n:] = torch.arange(1, 41, dtype=torch.bfloat16, device=CUDA).view(5, 8)
    offs = torch.full((76,), n, dtype=torch.int32, device=CUDA)
    offs[0], offs[75] = 0, n + 5
    ws = B.workspace(256)
    dw = B.grouped_wgrad(x, x, offs, out="f32", ws=ws)
    B.check_device_status(ws)
    for e, rows in ((0, x[some]), (74, x[n:])):     # whole numbers below 2^24: exact in any order
        assert torch.equal(dw[e].double(), rows.double().t() @ rows.double())
    assert (dw[1:74] == 0).all()
