"""moe_grouped_workspace_size is 0 exactly for what the products refuse by its fields alone (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def _nvfp4(B, k):
    g = B.MoEGrouped(groups=2, rows=4, n=8, k=k, dtype=B.MOE_NVFP4, out_dtype=B.MOE_F32)
    return B.lib.moe_grouped_workspace_size(ctypes.byref(g)), g


def test_long_nvfp4_reductions(B):
    size, g = _nvfp4(B, 2 ** 26 + 32)
    assert size == 0
    # refused for its length before the workspace is looked at
    assert B.lib.moe_grouped_matmul_nvfp4(ctypes.byref(g), 16, 16, None, 16, 16, 16, None, None, 16, 16, 0,
                                          None) == B.MOE_ERR_UNSUPPORTED
    assert _nvfp4(B, 2 ** 26)[0] == _nvfp4(B, 2 ** 26 - 32)[0] == _nvfp4(B, 2 ** 26 + 256)[0] == 256


def test_wide_fp32_outputs(B):
    wide, ok = 4194240 + 8, 64
    g = lambda n, k: ctypes.byref(B.MoEGrouped(groups=2, rows=4, n=n, k=k, dtype=B.MOE_F32, out_dtype=B.MOE_F32))  # noqa: E731
    assert B.lib.moe_grouped_matmul(g(wide, ok), 16, 16, 16, 0, None, 16, 16, 256, None) == B.MOE_ERR_UNSUPPORTED
    assert B.lib.moe_grouped_wgrad(g(ok, wide), 16, 16, 16, 0, 16, 16, 256, None) == B.MOE_ERR_UNSUPPORTED
    assert B.lib.moe_grouped_workspace_size(g(wide, ok)) == B.lib.moe_grouped_workspace_size(g(ok, wide)) == 256
