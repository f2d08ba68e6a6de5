"""The NaN scale (0x7f) that marks a block with an infinity or a NaN reaches the product:
its token's row, or its feature's column in the group, is NaN and nothing else is."""
import numpy as np
import pytest
import torch

from tests import grouped_ref as R
from tests.test_grouped import CUDA, _check, _np, _nvfp4, _offsets, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


# scales through TMA (K a multiple of 256) and copied by warps; few and many rows a group; a cut reduction
@pytest.mark.parametrize("sizes,N,K", [([9, 0, 40], 72, 512), ([9, 0, 40], 136, 288), ([300, 77], 200, 768),
                                       ([300, 77], 72, 544), ([5], 128, 8192)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nan_scale_through_the_product(B, sizes, N, K, out):
    offs = _offsets(sizes)
    E, rows, e = len(sizes), offs[-1], len(sizes) - 1
    a, sa, ra = _nvfp4(1, (rows, K))
    w, sw, rw = _nvfp4(2, (E, N, K), K ** -0.5)
    token, feature = offs[e] + 3, 37
    a[token, 8:16], sa[token, 1] = 0, 0x7F                              # block 1, codes 0
    last = K // 16 - 1
    w[e, feature, last * 8:], sw[e, feature, last] = 0, 0x7F
    t = [torch.from_numpy(v).to(CUDA) for v in (a, sa, w, sw)]
    got = _np(B.grouped_matmul_nvfp4(*t, torch.tensor(offs, dtype=torch.int32, device=CUDA),
                                     torch.from_numpy(ra).to(CUDA), torch.from_numpy(rw).to(CUDA), out=out))
    want = np.zeros(got.shape, bool)
    want[token] = True
    want[offs[e]:offs[e + 1], feature] = True
    assert np.array_equal(np.isnan(got), want)
    sa[token, 1], sw[e, feature, last] = 0, 0                           # the block without its mark
    ref, mag = R.matmul(R.decode(a, sa, ra), R.decode(w, sw, rw), offs)
    _check(got[~want], ref[~want], mag[~want], K, out, "y")


def test_an_infinity_stays_visible_from_the_quantisation_on(B):
    x, w = _rand(1, (40, 512), "bf16"), _rand(2, (72, 512), "bf16", 0.05)
    x[7, 100] = float("inf")
    q, qw = B.quantize_nvfp4(x.to(CUDA)), B.quantize_nvfp4(w.to(CUDA))
    y = B.grouped_matmul_nvfp4(q["codes"], q["scales"], qw["codes"].view(1, 72, -1), qw["scales"].view(1, 72, -1), None,
                               q["row_scale"], qw["row_scale"].view(1, 72))
    bad = torch.isnan(y)
    assert bad[7].all() and int(bad.sum()) == 72
