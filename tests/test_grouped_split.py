"""The grouped products where a tile's reduction is cut into parts, one a CTA (or
CTA pair) of a cluster, and the parts are summed through distributed shared memory.

With 74 pairs on the device the weight gradient is cut from 32 blocks of 64 rows a
group on average (2 parts from there while the tiles fill at most half of the
pairs, 4 while they fill a quarter), the bf16 product from K = 32 * 64 on.
Tolerances as in test_grouped.py: a sum of partial sums has no more additions than
terms.
"""
import numpy as np
import pytest
import torch

from tests import grouped_ref as R
from tests.test_grouped import CUDA, TORCH, _check, _np, _offsets, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([2100], 72, 72),              # 4 parts, the last block partial
                                       ([8200], 264, 136),            # 4 parts
                                       ([2112], 1000, 520),           # 2 parts, no partial block
                                       ([4500, 0, 40, 4000], 72, 136),  # 4: parts without rows, groups without any
                                       ([0, 8190, 1], 136, 264)])
def test_weight_gradient_in_parts(B, sizes, N, K, accumulate, out):
    offs = _offsets(sizes, first=3)
    rows = offs[-1] + 9
    dy, a, old = _rand(1, (rows, N), "bf16"), _rand(2, (rows, K), "bf16"), _rand(3, (len(sizes), N, K), out)
    for t in (dy, a):  # what lies outside the groups must not reach any sum
        t[:3], t[-9:] = float("nan"), float("inf")
    dw = old.to(CUDA).clone()
    B.grouped_wgrad(dy.to(CUDA), a.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA), dw=dw,
                    accumulate=accumulate)
    ref, mag = R.wgrad(_np(dy), _np(a), offs)
    if accumulate:
        ref, mag = ref + _np(old), mag + np.abs(_np(old))
    got = _np(dw)
    _check(got, ref, mag, max(sizes) + 1, out, "dw")
    for e, n in enumerate(sizes):
        if n == 0:
            assert (got[e] == (_np(old)[e] if accumulate else 0)).all(), "an empty group's gradient"


def test_weight_gradient_in_parts_keeps_nan_to_its_group(B):
    sizes = [2100, 2500]
    offs = _offsets(sizes)
    dy, a = _rand(1, (4600, 64), "bf16"), _rand(2, (4600, 72), "bf16")
    dy[2100], a[2100] = float("nan"), float("nan")  # the row behind the first group's last, partial block
    got = _np(B.grouped_wgrad(dy.to(CUDA), a.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA)))
    assert np.isnan(got[1]).all()
    dy[2100], a[2100] = 0, 0
    ref, mag = R.wgrad(_np(dy), _np(a), offs)
    _check(got[0], ref[0], mag[0], 2100, "bf16", "dw[0]")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,N,K", [([1501], 136, 2056), ([300], 136, 4104), ([0, 130, 1, 90], 72, 2048),
                                       ([3, 0, 20], 264, 4096)])
def test_product_in_parts(B, sizes, N, K, out, transposed):
    offs = _offsets(sizes, first=2)
    rows = offs[-1] + 5
    a, rw = _rand(1, (rows, K), "bf16"), _rand(3, (rows,), "f32")
    w = _rand(2, (len(sizes), K, N) if transposed else (len(sizes), N, K), "bf16", K ** -0.5)
    for t in (a, rw):  # rows of no group
        t[:2], t[-5:] = float("nan"), float("nan")
    y = torch.full((rows, N), 7.0, dtype=TORCH[out], device=CUDA)
    B.grouped_matmul(a.to(CUDA), w.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA), transposed=transposed,
                     row_weight=rw.to(CUDA), y=y)
    a[:2], a[-5:], rw[:2], rw[-5:] = 0, 0, 0, 0
    ref, mag = R.matmul(_np(a), _np(w), offs, transposed, _np(rw))
    got = _np(y)
    _check(got, ref, mag, K, out, "y")
    assert (got[:2] == 7.0).all() and (got[-5:] == 7.0).all(), "rows of no group were written"


@pytest.mark.parametrize("sizes,N,K", [([8200], 264, 136), ([4500, 0, 40, 4000], 72, 136)])
def test_parts_give_the_same_bits_every_time(B, sizes, N, K):
    rows = sum(sizes)
    dy, a = _rand(1, (rows, N), "bf16").to(CUDA), _rand(2, (rows, K), "bf16").to(CUDA)
    offs = torch.tensor(_offsets(sizes), dtype=torch.int32, device=CUDA)
    first, streams = B.grouped_wgrad(dy, a, offs, out="f32"), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [B.grouped_wgrad(dy, a, offs, out="f32", stream=s) for _ in range(5) for s in streams]  # side by side
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, first)
