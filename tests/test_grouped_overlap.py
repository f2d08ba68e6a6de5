"""Offsets that go to and fro, an error of the caller's: groups overlap and have more
tiles together than the rows allow for, in the large cases more than 32 bits count.
Such a product writes nothing (and reads and writes nothing out of range)."""
import pytest
import torch

CUDA = "cuda"
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def _to_and_fro(E, rows):
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[1::2] = rows
    return offs.to(CUDA)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("E,rows", [(400, 200), (3, 400)])
def test_overlapping_groups(B, E, rows, dtype, transposed):
    a, w = torch.randn(rows, 64, device=CUDA).to(dtype), torch.randn(E, 64, 64, device=CUDA).to(dtype)
    y = torch.full((rows, 64), 7.5, dtype=dtype, device=CUDA)
    B.grouped_matmul(a, w, _to_and_fro(E, rows), transposed=transposed, y=y)
    assert (y == 7.5).all()
    dw = B.grouped_wgrad(a, a, _to_and_fro(E, rows), out="f32")   # every group by itself: whole or empty
    assert torch.equal(dw[0], dw[2]) and (dw[1] == 0).all()
    B.check_device_status()


@pytest.mark.parametrize("K", [64, 256])
def test_overlapping_groups_nvfp4(B, K):
    q, qw = B.quantize_nvfp4(torch.randn(200, K, device=CUDA)), B.quantize_nvfp4(torch.randn(400 * 64, K, device=CUDA))
    y = torch.full((200, 64), 7.5, dtype=torch.bfloat16, device=CUDA)
    B.grouped_matmul_nvfp4(q["codes"], q["scales"], qw["codes"].view(400, 64, -1), qw["scales"].view(400, 64, -1),
                           _to_and_fro(400, 200), y=y)
    assert (y == 7.5).all()
    B.check_device_status()


@pytest.mark.parametrize("dtype,rows", [(torch.bfloat16, 280_000_000), (torch.float32, 140_000_000)])
def test_overlapping_groups_whose_tiles_pass_32_bits(B, dtype, rows):
    a, y = torch.zeros(rows, 8, dtype=dtype, device=CUDA), torch.full((rows, 8), 7.5, dtype=dtype, device=CUDA)
    assert 512 * rows // (64 if dtype == torch.bfloat16 else 32) > 2 ** 31
    B.grouped_matmul(a, torch.ones(1024, 8, 8, dtype=dtype, device=CUDA), _to_and_fro(1024, rows), y=y)
    assert (y == 7.5).all()
    B.check_device_status()
