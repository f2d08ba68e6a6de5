"""The scales of the NVFP4 product are magnitudes: the sign bit of an e4m3 scale is not read, whichever
way the scales get to the tensor cores and in every product of a token's and a weight's block."""
import numpy as np
import pytest
import torch

from tests import grouped_ref as R
from tests.test_grouped import CUDA, _nvfp4, _offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


@pytest.mark.parametrize("sizes,N,K", [([9, 0, 40], 72, 512), ([9, 0, 40], 136, 288), ([300, 77], 200, 768),
                                       ([300, 77], 72, 544), ([5], 128, 8192)])
def test_the_sign_of_a_scale_is_not_read(B, sizes, N, K):
    offs = torch.tensor(_offsets(sizes), dtype=torch.int32, device=CUDA)
    a, sa, ra = _nvfp4(1, (sum(sizes), K))
    w, sw, rw = _nvfp4(2, (len(sizes), N, K), K ** -0.5)
    rng = np.random.default_rng(3)
    signed = [s | (rng.integers(0, 2, s.shape) << 7).astype(np.uint8) for s in (sa, sw)]
    dev = lambda v: torch.from_numpy(v).to(CUDA)  # noqa: E731
    f = lambda sa, sw: B.grouped_matmul_nvfp4(dev(a), dev(sa), dev(w), dev(sw), offs, dev(ra), dev(rw), out="f32")  # noqa: E731
    assert torch.equal(f(*signed), f(sa, sw))


def test_every_scale_byte(B):
    # one term a row: every scale byte against a code of 1 and a scale of 1
    code, s8 = np.zeros((256, 256), np.uint8), np.zeros((256, 16), np.uint8)
    code[:, 16], s8[:, 1] = 2, np.arange(256)
    w, ws = np.zeros((1, 8, 256), np.uint8), np.full((1, 8, 16), 0x38, np.uint8)
    w[0, :, 16] = 2
    got = B.grouped_matmul_nvfp4(*(torch.from_numpy(v).to(CUDA) for v in (R.pack(code), s8, R.pack(w), ws)), None,
                                 out="f32").double().cpu().numpy()
    want = np.concatenate([R.E4M3, [np.nan]] * 2)
    np.testing.assert_array_equal(got, np.repeat(want[:, None], 8, 1))
