"""The grouped products, quantisation and SwiGLU at the edges of what they accept:
the most groups, offsets out of range, sizes whose element offsets pass 32 bits,
base addresses aligned to 16 bytes only, inputs and offsets that change under a
captured graph, and the checked build's refusal of bad indices."""
import threading

import numpy as np
import pytest
import torch

from tests import grouped_ref as R
from tests.test_grouped import CUDA, _check, _np, _nvfp4, _offsets, _rand, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=CUDA)


# ------------------------------------------------------------------ groups and offsets

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_groups(B, dtype):
    rng = np.random.default_rng(0)
    sizes = rng.integers(0, 4, 1024)
    sizes[700] = 200
    offs = _offsets(sizes)
    rows, N, K = offs[-1], 40, 72
    a, w, dy = _rand(1, (rows, K), dtype), _rand(2, (1024, N, K), dtype, 0.1), _rand(3, (rows, N), dtype)
    y = B.grouped_matmul(a.to(CUDA), w.to(CUDA), _i32(offs))
    ref, mag = R.matmul(_np(a), _np(w), offs)
    _check(_np(y), ref, mag, K, dtype, "y")
    dw = B.grouped_wgrad(dy.to(CUDA), a.to(CUDA), _i32(offs))
    ref, mag = R.wgrad(_np(dy), _np(a), offs)
    _check(_np(dw), ref, mag, 200, dtype, "dw")


def test_most_groups_nvfp4(B):
    sizes = np.random.default_rng(0).integers(0, 4, 1024)
    offs = _offsets(sizes)
    a, sa, ra = _nvfp4(1, (offs[-1], 96))
    w, sw, rw = _nvfp4(2, (1024, 16, 96), 0.1)
    t = [torch.from_numpy(v).to(CUDA) for v in (a, sa, w, sw)]
    y = B.grouped_matmul_nvfp4(*t, _i32(offs), torch.from_numpy(ra).to(CUDA), torch.from_numpy(rw).to(CUDA))
    ref, mag = R.matmul(R.decode(a, sa, ra), R.decode(w, sw, rw), offs)
    _check(_np(y), ref, mag, 96, "bf16", "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [[0, 10, 4000], [-7, 10, 60], [-(2 ** 31), 10, 2 ** 31 - 1]])
def test_offsets_are_kept_within_the_rows(B, dtype, bad):
    a, w, dy = _rand(1, (60, 64), dtype), _rand(2, (2, 72, 64), dtype), _rand(3, (60, 72), dtype)
    a, w, dy = a.to(CUDA), w.to(CUDA), dy.to(CUDA)
    good = _i32([0, 10, 60])
    assert torch.equal(B.grouped_matmul(a, w, _i32(bad)), B.grouped_matmul(a, w, good))
    assert torch.equal(B.grouped_wgrad(dy, a, _i32(bad)), B.grouped_wgrad(dy, a, good))
    x = (_rand(4, (60, 64), dtype)).to(CUDA)
    if bad[-1] > 60:
        for k, v in B.quantize_nvfp4(x, offsets=_i32(bad)).items():
            assert v is None or torch.equal(v, B.quantize_nvfp4(x)[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decreasing_offsets_leave_the_group_empty(B, dtype):
    # group 1 ends before it starts: no rows; the others are whole
    a, w = _rand(1, (60, 64), dtype), _rand(2, (3, 72, 64), dtype)
    dy = _rand(3, (60, 72), dtype)
    offs = [0, 40, 40, 60]
    got = B.grouped_matmul(a.to(CUDA), w.to(CUDA), _i32(offs))
    ref, mag = R.matmul(_np(a), _np(w), offs)
    _check(_np(got), ref, mag, 64, dtype, "y")
    dw = _np(B.grouped_wgrad(dy.to(CUDA), a.to(CUDA), _i32([0, 40, 35, 60])))
    assert (dw[1] == 0).all()
    for e, (r0, r1) in ((0, (0, 40)), (2, (35, 60))):
        ref, mag = R.wgrad(_np(dy)[r0:r1], _np(a)[r0:r1], [0, r1 - r0])
        _check(dw[e], ref[0], mag[0], 40, dtype, f"dw[{e}]")


def test_graph_follows_its_inputs(B):
    """Offsets, rows and weights that change between replays."""
    a, w, dy = (torch.zeros(s, dtype=torch.bfloat16, device=CUDA) for s in ((500, 136), (5, 72, 136), (500, 72)))
    offs, ws = _i32([0] * 6), B.workspace(256)
    run = lambda: (B.grouped_matmul(a, w, offs, ws=ws), B.grouped_wgrad(dy, a, offs, ws=ws),  # noqa: E731
                   B.quantize_nvfp4(a[:, :128].contiguous(), values=True)["values"])
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed, sizes in enumerate([[100] * 5, [500, 0, 0, 0, 0], [1, 2, 3, 4, 5], [0, 0, 0, 0, 0], [7, 0, 433, 0, 60]]):
        a.copy_(_rand(seed, (500, 136), "bf16"))
        w.copy_(_rand(seed + 50, (5, 72, 136), "bf16"))
        dy.copy_(_rand(seed + 90, (500, 72), "bf16"))
        offs.copy_(_i32(_offsets(sizes)))
        for t in out:
            t.fill_(3.0)
        g.replay()
        want = run()
        n = sum(sizes)
        assert torch.equal(out[0][:n], want[0][:n]) and (out[0][n:] == 3).all()
        assert torch.equal(out[1], want[1]) and torch.equal(out[2], want[2])
        ref, mag = R.matmul(_np(a), _np(w), _offsets(sizes))
        _check(_np(out[0]), ref, mag, 136, "bf16", "y")
    B.check_device_status(ws)


# ------------------------------------------------------------------ large sizes, alignment

def test_product_rows_past_32_bit_offsets(B):
    rows, N, K = 1_100_000, 2048, 64
    a, w = torch.randn(rows, K, device=CUDA).bfloat16(), torch.randn(3, N, K, device=CUDA).bfloat16()
    offs = [0, 3, 1_050_001, rows]
    rw = torch.rand(rows, device=CUDA)
    y = B.grouped_matmul(a, w, _i32(offs), row_weight=rw)
    assert y.numel() > 2 ** 31
    for r, e in ((0, 0), (3, 1), (1_048_575, 1), (1_048_576, 1), (1_050_000, 1), (1_050_001, 2), (rows - 1, 2)):
        ref = (w[e].double() @ a[r].double()) * rw[r].double()
        mag = (w[e].double().abs() @ a[r].double().abs()) * rw[r].double()
        _check(_np(y[r]), _np(ref), _np(mag), K, "bf16", f"row {r}")
    x = B.grouped_matmul(y, w, _i32(offs), transposed=True, out="f32")   # back: reads past 2^31 elements
    for r, e in ((1_048_577, 1), (rows - 1, 2)):
        ref, mag = y[r].double() @ w[e].double(), y[r].double().abs() @ w[e].double().abs()
        _check(_np(x[r]), _np(ref), _np(mag), N, "f32", f"row {r}")


def test_weight_gradient_past_32_bit_offsets(B):
    E, N, K = 70, 8192, 4096
    sizes = [3] * E
    dy, a = torch.randn(3 * E, N, device=CUDA).bfloat16(), torch.randn(3 * E, K, device=CUDA).bfloat16()
    dw = B.grouped_wgrad(dy, a, _i32(_offsets(sizes)))
    assert dw.numel() > 2 ** 31
    for e in (0, 63, 64, 69):
        ref = dy[3 * e:3 * e + 3].double().t() @ a[3 * e:3 * e + 3].double()
        mag = dy[3 * e:3 * e + 3].double().abs().t() @ a[3 * e:3 * e + 3].double().abs()
        _check(_np(dw[e, ::97]), _np(ref[::97]), _np(mag[::97]), 3, "bf16", f"dw[{e}]")


def test_nvfp4_weights_past_32_bit_offsets(B):
    E, N, K, rows = 300, 4096, 4096, 600
    g = torch.Generator(device=CUDA).manual_seed(0)
    byte = lambda *s, hi=256: torch.randint(0, hi, s, generator=g, device=CUDA, dtype=torch.uint8)  # noqa: E731
    w, sw, a, sa = byte(E, N, K // 2), byte(E, N, K // 16, hi=100), byte(rows, K // 2), byte(rows, K // 16, hi=100)
    assert w.numel() > 2 ** 31
    y = B.grouped_matmul_nvfp4(a, sa, w, sw, _i32(_offsets([2] * E)), out="f32")
    for r in (0, 511, 513, 598, 599):
        A = R.decode(a[r:r + 1].cpu().numpy(), sa[r:r + 1].cpu().numpy())
        W = R.decode(w[r // 2].cpu().numpy(), sw[r // 2].cpu().numpy())
        _check(_np(y[r:r + 1]), A @ W.T, np.abs(A) @ np.abs(W).T, K, "f32", f"row {r}")


def test_rows_past_32_bit_offsets_quantize_and_swiglu(B):
    rows, F = 600_000, 2048
    gu = torch.randn(rows, 2 * F, device=CUDA, dtype=torch.bfloat16)
    assert gu.numel() > 2 ** 31
    at = torch.tensor([0, 1, 262_143, 262_144, 524_287, 524_288, rows - 1], device=CUDA)
    q = B.quantize_nvfp4(gu, values=True)
    _same({k: v[at] for k, v in q.items()}, R.quantize(_np(gu[at]), True))
    del q
    h = B.swiglu(gu)
    ref = R.swiglu(_np(gu[at]))
    assert (np.abs(_np(h[at]) - ref) <= (R.STEP["bf16"] + 24 * 2.0 ** -24) * np.abs(ref) + 1e-37).all()
    b = B.swiglu_backward(gu, h)
    small = B.swiglu_backward(gu[at].contiguous(), h[at].contiguous())
    for k in b:
        # the same rows by themselves; a row's sum may be shared by warps there
        if k == "drow_weight":
            torch.testing.assert_close(b[k][at], small[k], rtol=1e-4, atol=1e-4)
        else:
            assert torch.equal(b[k][at], small[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_addresses_aligned_to_16_bytes_only(B, dtype):
    skip = 8 if dtype == "bf16" else 4          # elements in 16 bytes
    def shifted(t):
        buf = torch.empty(t.numel() + skip, dtype=t.dtype, device=CUDA)
        v = buf[skip:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v
    x, w, dy = _rand(1, (70, 144), dtype), _rand(2, (2, 72, 144), dtype), _rand(3, (70, 72), dtype)
    offs, rw = _i32([0, 33, 70]), torch.rand(71, device=CUDA)[1:]
    q0, q1 = B.quantize_nvfp4(x.to(CUDA), values=True), B.quantize_nvfp4(shifted(x), values=True)
    out = {k: torch.empty(v.numel() + 16, dtype=v.dtype, device=CUDA)[16 // v.element_size():][:v.numel()].view(v.shape)
           for k, v in q0.items()}
    B.quantize_nvfp4(shifted(x), values=True, out=out)
    for k in q0:
        assert torch.equal(q0[k], q1[k]) and torch.equal(q0[k], out[k]), k
    for f in (lambda m: B.grouped_matmul(m(x), m(w), offs, row_weight=rw), lambda m: B.grouped_wgrad(m(dy), m(x), offs),
              lambda m: B.swiglu(m(x)), lambda m: B.swiglu_backward(m(x), m(dy), rw)["dgu"]):
        assert torch.equal(f(lambda t: t.to(CUDA)), f(shifted))


# ------------------------------------------------------------------ the checked build

@pytest.fixture(scope="module")
def BC(B):
    try:
        from mixture_experts_layer_sqrt_b200 import build
        build.build(checked=True)
    except (RuntimeError, OSError) as e:
        pytest.skip(f"cannot build the checked library here: {e}")
    normal = B.lib
    checked = B.load_library(B.LIB_CHECKED_PATH)
    B.lib = checked
    yield B, checked
    B.lib = normal


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_checked_build_refuses_bad_offsets(BC, dtype):
    B, lib = BC
    lib.moe_checked_violations()
    a, w, dy = _rand(1, (60, 64), dtype).to(CUDA), _rand(2, (3, 72, 64), dtype).to(CUDA), _rand(3, (60, 72), dtype).to(CUDA)
    for bad in ([0, 40, 20, 60], [-1, 20, 40, 60]):
        y = torch.full((60, 72), 7.5, dtype=a.dtype, device=CUDA)
        B.grouped_matmul(a, w, _i32(bad), y=y)
        assert lib.moe_checked_violations() >= 1 and (y == 7.5).all()
        dw = torch.full((3, 72, 64), 7.5, dtype=a.dtype, device=CUDA)
        B.grouped_wgrad(dy, a, _i32(bad), dw=dw)
        first = 0 if bad[0] < 0 else 1
        assert lib.moe_checked_violations() >= 1 and (dw[first] == 7.5).all()
    good = _i32([0, 20, 20, 60])
    B.grouped_matmul(a, w, good), B.grouped_wgrad(dy, a, good)
    assert lib.moe_checked_violations() == 0


def test_checked_build_refuses_bad_offsets_nvfp4_and_row_maps(BC):
    B, lib = BC
    lib.moe_checked_violations()
    a, sa, _ = _nvfp4(1, (60, 256))
    w, sw, _ = _nvfp4(2, (3, 72, 256), 0.1)
    t = [torch.from_numpy(v).to(CUDA) for v in (a, sa, w, sw)]
    y = torch.full((60, 72), 7.5, dtype=torch.bfloat16, device=CUDA)
    B.grouped_matmul_nvfp4(*t, _i32([0, 40, 20, 60]), y=y)
    assert lib.moe_checked_violations() >= 1 and (y == 7.5).all()
    x = _rand(3, (10, 32), "bf16").to(CUDA)
    q = B.quantize_nvfp4(x, row_token=_i32([0, 10, 3, -1]), values=True)
    assert lib.moe_checked_violations() == 2
    want = B.quantize_nvfp4(x, row_token=_i32([0, 3]), values=True)
    for k in q:
        assert torch.equal(q[k][[0, 2]], want[k]), k
    assert lib.moe_checked_violations() == 0


# ------------------------------------------------------------------ two host threads at once

@pytest.mark.gpu
def test_different_operators_from_two_threads_at_once(B):
    offs = torch.tensor([0, 40, 40, 130, 137], dtype=torch.int32, device=CUDA)
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(137, 256, generator=gen).to(CUDA, torch.bfloat16)
    w = torch.randn(4, 192, 256, generator=gen).to(CUDA, torch.bfloat16)
    dy = torch.randn(137, 192, generator=gen).to(CUDA, torch.bfloat16)
    q, qw = B.quantize_nvfp4(x), B.quantize_nvfp4(w.reshape(-1, 256))
    calls = [
        lambda s: B.grouped_matmul(x, w, offs, stream=s),
        lambda s: B.grouped_wgrad(dy, x, offs, stream=s),
        lambda s: B.grouped_matmul(dy, w, offs, transposed=True, stream=s),
        lambda s: B.grouped_matmul_nvfp4(q["codes"], q["scales"], qw["codes"].reshape(4, 192, 128),
                                         qw["scales"].reshape(4, 192, 16), offs, q["row_scale"],
                                         qw["row_scale"].reshape(4, 192), stream=s),
        lambda s: B.swiglu_quantize_nvfp4(x, values=True, stream=s)["values"],
    ]
    # rows outside the groups do not exist here (the offsets cover all), so whole outputs compare
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams, got, errors = [torch.cuda.Stream() for _ in range(2)], [[], []], []

    def run(i):
        try:
            for j in range(20):
                k = (j * (i + 1) + i) % len(calls)
                got[i].append((k, calls[k](streams[i])))
        except Exception as e:  # noqa: BLE001 - handed to the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for results in got:
        assert len(results) == 20
        for k, r in results:
            assert torch.equal(r, want[k]), k
