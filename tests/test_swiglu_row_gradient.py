"""The routing weights' gradient of bf16 rows is an fp32 result: each of its terms is good to fp32.

One term a row: drow_weight = d * h, h = (g * s) * u, s = 1 / (1 + e^-g). e^-g is off by at most two
steps (4 half steps of 2^-24), the sum by one half step, the hardware's reciprocal by one step (2), and
the three products by a half step each: 10 * 2^-24. Adding the row's other terms, all 0, is exact."""
import numpy as np
import pytest
import torch

CUDA = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("F", [8, 264, 2304])
def test_terms_of_the_row_sum(F, dtype):
    from mixture_experts_layer_sqrt_b200 import binding as B
    rng = np.random.default_rng(0)
    rows = 3000
    g = torch.from_numpy(np.concatenate([np.linspace(-80, 80, rows // 2), rng.standard_normal(rows // 2) * 4])).to(dtype)
    u, d = (torch.from_numpy(rng.standard_normal(rows)).to(dtype) for _ in range(2))
    at = torch.from_numpy(rng.integers(0, F, rows))
    gu, dh = torch.zeros(rows, 2 * F, dtype=dtype), torch.zeros(rows, F, dtype=dtype)
    r = torch.arange(rows)
    gu[r, at], gu[r, F + at], dh[r, at] = g, u, d
    got = B.swiglu_backward(gu.to(CUDA), dh.to(CUDA))["drow_weight"].double().cpu()
    want = d.double() * g.double() / (1 + torch.exp(-g.double())) * u.double()
    assert ((got - want).abs() <= 10 * 2.0 ** -24 * want.abs()).all()
