"""Products grouped by expert and their gradients, NVFP4 quantisation and product,
SwiGLU and its gradient, against float64 references (tests/grouped_ref.py).

Tolerances, derived from the arithmetic:
 - a product of K terms: the terms are exact in fp32 (bf16 or NVFP4 operands) or
   rounded within an FMA; every addition is off by at most one fp32 step, 2^-23
   of a partial sum that never exceeds the sum M of the terms' magnitudes, so
   |err| <= K 2^-23 M, plus a few 2^-24 for the row weights and scales, plus half
   a step of the output type.
 - codes, scales and row scales: equal bit by bit.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests import grouped_ref as R

CUDA = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def _np(t):
    t = t.detach().cpu()
    return (t.float() if t.dtype == torch.bfloat16 else t).numpy().astype(np.float64)


def _rand(seed, shape, dtype, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape) * scale
    return torch.from_numpy(x.astype(np.float32)).to(TORCH[dtype])


def _offsets(sizes, first=0):
    return [first] + [first + int(v) for v in np.cumsum(sizes)]


def _check(got, ref, mag, terms, out, what, extra=4):
    """|got - ref| within the bound above; ref NaN = a value that must not have been written."""
    keep = ~np.isnan(ref)
    lim = R.STEP[out] * np.abs(ref) + (terms * 2.0 ** -23 + extra * 2.0 ** -24) * mag
    err = np.abs(got - ref)
    bad = keep & ~(err <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, e.g. at {np.argwhere(bad)[0]}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}"


SIZES = {
    "one": [1],
    "edges": [0, 1, 15, 16, 17, 0, 63, 64, 65, 0],
    "wide": [255, 256, 257, 0, 300, 1],
    "few_of_many": [0] * 5 + [1, 0, 0, 2] + [0] * 30 + [1],
    "long": [1501],                  # one group: its few tiles' reductions are cut into parts
    "two_long": [300, 0, 419],
    "many": [900, 37, 1500, 64, 0, 1030],    # more tiles than the GPU runs at once
    "many_small": [(7 * i) % 23 for i in range(45)],
}


# ------------------------------------------------------------------ products

@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("sizes,N,K", [("one", 8, 8), ("one", 520, 4104), ("edges", 136, 72), ("edges", 384, 512),
                                       ("wide", 128, 64), ("wide", 264, 200), ("few_of_many", 72, 1032),
                                       ("two_long", 264, 2056), ("long", 136, 1096), ("many", 2048, 136),
                                       ("many_small", 640, 200)])
def test_matmul(B, sizes, N, K, dtype, out, transposed):
    sizes = SIZES[sizes]
    E, dead = len(sizes), 5
    offs = _offsets(sizes, first=2)  # two rows before the first group, five behind the last
    rows = offs[-1] + dead
    a = _rand(1, (rows, K), dtype)
    w = _rand(2, (E, K, N) if transposed else (E, N, K), dtype, K ** -0.5)
    rw = _rand(3, (rows,), "f32")
    y = torch.full((rows, N), 7.0, dtype=TORCH[out], device=CUDA)
    B.grouped_matmul(a.to(CUDA), w.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA), transposed=transposed,
                     row_weight=rw.to(CUDA), y=y)
    got = _np(y)
    ref, mag = R.matmul(_np(a), _np(w), offs, transposed, _np(rw))
    _check(got, ref, mag, K, out, "y")
    assert (got[:2] == 7.0).all() and (got[-dead:] == 7.0).all(), "rows of no group were written"


@pytest.mark.gpu
def test_matmul_one_group_without_offsets_and_weights(B):
    a, w = _rand(1, (70, 96), "bf16"), _rand(2, (1, 40, 96), "bf16", 0.1)
    y = B.grouped_matmul(a.to(CUDA), w.to(CUDA), None)
    ref, mag = R.matmul(_np(a), _np(w), [0, 70])
    _check(_np(y), ref, mag, 96, "bf16", "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matmul_keeps_nan_and_infinity_to_their_rows(B, dtype):
    sizes = [20, 30, 3]
    offs = _offsets(sizes)
    a, w = _rand(1, (53, 128), dtype), _rand(2, (3, 64, 128), dtype, 0.1)
    a[25], a[50, 3] = float("nan"), float("inf")
    got = _np(B.grouped_matmul(a.to(CUDA), w.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA)))
    assert np.isnan(got[25]).all() and not np.isfinite(got[50]).any()
    keep = np.ones(53, bool)
    keep[[25, 50]] = False
    a[25], a[50] = 0, 0
    ref, mag = R.matmul(_np(a), _np(w), offs)
    _check(got[keep], ref[keep], mag[keep], 128, dtype, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,N,K", [("one", 8, 8), ("edges", 136, 72), ("edges", 128, 520), ("wide", 264, 200),
                                       ("few_of_many", 72, 264), ("long", 136, 264), ("two_long", 72, 520),
                                       ("many", 1000, 1032), ("many_small", 264, 136)])
def test_wgrad(B, sizes, N, K, dtype, out, accumulate):
    sizes = SIZES[sizes]
    offs = _offsets(sizes, first=3)
    rows = offs[-1] + 9
    dy, a = _rand(1, (rows, N), dtype), _rand(2, (rows, K), dtype)
    old = _rand(3, (len(sizes), N, K), out)
    # what lies outside the groups must not reach any sum, whatever it holds
    for t in (dy, a):
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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wgrad_keeps_nan_to_its_group(B, dtype):
    sizes = [5, 70, 33]
    offs = _offsets(sizes)
    dy, a = _rand(1, (108, 64), dtype), _rand(2, (108, 72), dtype)
    dy[30], a[30] = float("nan"), float("nan")
    got = _np(B.grouped_wgrad(dy.to(CUDA), a.to(CUDA), torch.tensor(offs, dtype=torch.int32, device=CUDA)))
    assert np.isnan(got[1]).all()
    dy[30], a[30] = 0, 0
    ref, mag = R.wgrad(_np(dy), _np(a), offs)
    for e in (0, 2):
        _check(got[e], ref[e], mag[e], 70, dtype, f"dw[{e}]")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wgrad_without_rows(B, dtype):
    dy, a = torch.empty((0, 64), dtype=TORCH[dtype], device=CUDA), torch.empty((0, 72), dtype=TORCH[dtype], device=CUDA)
    offs = torch.zeros(4, dtype=torch.int32, device=CUDA)
    dw = torch.full((3, 64, 72), 5.0, dtype=TORCH[dtype], device=CUDA)
    B.grouped_wgrad(dy, a, offs, dw=dw, accumulate=True)
    assert (dw == 5).all()
    B.grouped_wgrad(dy, a, offs, dw=dw)
    assert (dw == 0).all()
    assert B.grouped_matmul(a, torch.zeros((3, 64, 72), dtype=TORCH[dtype], device=CUDA), offs).shape == (0, 64)


# ------------------------------------------------------------------ NVFP4

def _nvfp4(seed, shape, scale=1.0):
    """Packed codes, scales and row scales (numpy, by the reference) of random rows."""
    x = _np(_rand(seed, shape, "bf16", scale)).reshape(-1, shape[-1])
    code, s8, rs, _ = R.quantize(x, True)
    lead = shape[:-1]
    return R.pack(code).reshape(*lead, -1), s8.reshape(*lead, -1), rs.reshape(lead).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,N,K", [("one", 8, 32), ("one", 520, 4096), ("edges", 136, 96), ("edges", 128, 256),
                                       ("edges", 264, 832), ("wide", 200, 512), ("wide", 72, 288), ("wide", 256, 320),
                                       ("few_of_many", 72, 1280), ("two_long", 136, 4064), ("long", 128, 8192),
                                       ("many", 1024, 512), ("many_small", 640, 544)])
def test_matmul_nvfp4(B, sizes, N, K, out):
    sizes = SIZES[sizes]
    E, dead = len(sizes), 4
    offs = _offsets(sizes, first=1)
    rows = offs[-1] + dead
    a, sa, ra = _nvfp4(1, (rows, K))
    w, sw, rw = _nvfp4(2, (E, N, K), K ** -0.5)
    wt = _rand(3, (rows,), "f32")
    y = torch.full((rows, N), 7.0, dtype=TORCH[out], device=CUDA)
    t = [torch.from_numpy(v).to(CUDA) for v in (a, sa, w, sw)]
    B.grouped_matmul_nvfp4(*t, torch.tensor(offs, dtype=torch.int32, device=CUDA),
                           a_row_scale=torch.from_numpy(ra).to(CUDA), w_row_scale=torch.from_numpy(rw).to(CUDA),
                           row_weight=wt.to(CUDA), y=y)
    got = _np(y)
    ref, mag = R.matmul(R.decode(a, sa, ra), R.decode(w, sw, rw), offs, row_weight=_np(wt))
    _check(got, ref, mag, K, out, "y")
    assert (got[:1] == 7.0).all() and (got[-dead:] == 7.0).all(), "rows of no group were written"


@pytest.mark.gpu
def test_matmul_nvfp4_every_scale_and_code(B):
    # one term a row: every finite scale byte against every code, no row scales
    K, N = 256, 128
    code = np.zeros((127, K), np.uint8)
    code[:, 16] = 2                                    # 1.0
    s8 = np.zeros((127, K // 16), np.uint8)
    s8[:, 1] = np.arange(127)
    w = np.zeros((1, N, K), np.uint8)
    w[0, :16, 16] = np.arange(16)
    ws = np.full((1, N, K // 16), 0x38, np.uint8)      # 1.0
    t = [torch.from_numpy(v).to(CUDA) for v in (R.pack(code), s8, R.pack(w), ws)]
    got = _np(B.grouped_matmul_nvfp4(*t, None, out="f32"))
    ref, _ = R.matmul(R.decode(R.pack(code), s8), R.decode(R.pack(w), ws), [0, 127])
    assert np.array_equal(got, ref)


def _source(kind, dtype, rows, cols):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((rows, cols))
    if kind == "wide":       # magnitudes over many binades, block by block
        x = x * 2.0 ** rng.integers(-30, 30, (rows, cols // 16)).repeat(16, 1)
    elif kind == "ties":     # exact ties of both formats: multiples of 1/4 times small integers
        x = rng.integers(-24, 25, (rows, cols)) * 0.25
        x[:, ::16] = 6.0 * rng.integers(16, 32, x[:, ::16].shape) / 16.0
    elif kind == "special":
        x[0] = 0.0
        x[1, :16] = 0.0
        x[2, 3], x[2, cols - 1] = np.inf, -np.inf
        x[3, 5] = np.nan
        x[4] = np.nan
        x[5] *= 1e-38        # below the smallest row scale's range
        x[6] *= 1e37
        x[7] = 2688.0 * 2.0 ** -20
        x[8] = -0.0
        x[9, 1:] *= 1e-8     # one large element
        x[10] = 2.0 ** -130  # subnormal
        x[11] = 3.3e38
    return torch.from_numpy(x.astype(np.float32)).to(TORCH[dtype])


def _same(q, ref, keep=None):
    code, s8, rs, values = ref
    keep = slice(None) if keep is None else keep
    np.testing.assert_array_equal(q["scales"].cpu().numpy()[keep], s8[keep])
    np.testing.assert_array_equal(R.unpack(q["codes"].cpu().numpy())[keep], code[keep])
    if q["row_scale"] is not None:
        np.testing.assert_array_equal(_np(q["row_scale"])[keep], rs[keep])
    if q["values"] is not None:
        np.testing.assert_array_equal(_np(q["values"])[keep], values[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("row_scaled", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,rows,cols", [("normal", 1, 16), ("normal", 37, 528), ("normal", 3, 4096),
                                            ("normal", 5, 8208), ("wide", 40, 1024), ("ties", 64, 256),
                                            ("special", 12, 4112), ("special", 12, 64)])
def test_quantize(B, kind, rows, cols, dtype, row_scaled):
    x = _source(kind, dtype, rows, cols)
    q = B.quantize_nvfp4(x.to(CUDA), row_scaled=row_scaled, values=True)
    # the values are bf16: those of a row scale of 1 may exceed its range downwards nowhere (min 2^-10)
    _same(q, R.quantize(_np(x), row_scaled))


@pytest.mark.gpu
def test_quantize_every_bf16_quotient(B):
    # every bf16 significand against every e4m3 significand, both signs: the quotient's
    # rounding must be that of the exact quotient
    rows = []
    for s in range(8, 16):
        top = 6.0 * s / 8.0                            # block maximum: scale s / 8 exactly
        mant = np.arange(128, 256) / 128.0
        for e in range(-4, 3):
            v = mant * 2.0 ** e
            v = v[v <= top]
            v = np.concatenate([v, np.zeros(-len(v) % 15)]).reshape(-1, 15)
            rows.append(np.concatenate([np.full((len(v), 1), top), v], 1))
    x = np.concatenate(rows)
    x = np.concatenate([x, -x])
    t = torch.from_numpy(x.astype(np.float32)).bfloat16()
    assert np.array_equal(_np(t), x)
    for dtype in ("bf16", "f32"):
        for scaled in (False, True):
            _same(B.quantize_nvfp4(t.to(TORCH[dtype]).to(CUDA), row_scaled=scaled, values=True), R.quantize(x, scaled))


@pytest.mark.gpu
def test_quantize_gathers_through_a_row_map(B):
    x = _source("normal", "bf16", 20, 512)
    rt = np.array([3, 3, 19, 0, -1, 7, 20, 1 << 30, 11, 5], np.int32)   # -1, 20 and 2^30 are no rows of x
    offs = torch.tensor([0, 4, 9], dtype=torch.int32, device=CUDA)      # the tenth row is behind the last group
    out = dict(codes=torch.full((10, 256), 9, dtype=torch.uint8, device=CUDA),
               scales=torch.full((10, 32), 9, dtype=torch.uint8, device=CUDA),
               row_scale=torch.full((10,), 9.0, device=CUDA),
               values=torch.full((10, 512), 9.0, dtype=torch.bfloat16, device=CUDA))
    q = B.quantize_nvfp4(x.to(CUDA), row_token=torch.from_numpy(rt).to(CUDA), offsets=offs, values=True, out=out)
    keep = np.array([0, 1, 2, 3, 5, 8])
    _same(q, R.quantize(_np(x)[np.clip(rt, 0, 19)], True), keep)
    rest = np.array([4, 6, 7, 9])
    for t in out.values():
        assert (_np(t)[rest] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("clamp,mode", [(0.0, "preact"), (2.0, "preact"), (1.5, "output")])
@pytest.mark.parametrize("rows,F", [(1, 16), (70, 384), (9, 4112)])
def test_swiglu_quantize_is_the_two_calls(B, rows, F, clamp, mode, dtype):
    gu = (_rand(1, (rows, 2 * F), dtype) * 2).to(CUDA)
    if rows > 8:
        gu[3, 5], gu[4, F + 7], gu[5] = float("nan"), float("inf"), 0.0
    h = B.swiglu(gu, clamp, mode)
    one, two = B.swiglu_quantize_nvfp4(gu, clamp, mode, values=True), B.quantize_nvfp4(h, values=True)
    for k in ("codes", "scales", "row_scale"):
        assert torch.equal(one[k], two[k]), k
    assert torch.equal(one["values"].nan_to_num(-1.0), two["values"].nan_to_num(-1.0))
    _same(two, R.quantize(_np(h), True))


# ------------------------------------------------------------------ SwiGLU

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("clamp,mode", [(0.0, "preact"), (2.0, "preact"), (1.5, "output")])
@pytest.mark.parametrize("rows,F", [(1, 8), (33, 264), (1500, 72), (7, 2304)])
def test_swiglu_and_backward(B, rows, F, clamp, mode, dtype):
    gu, d, rw = _rand(1, (rows, 2 * F), dtype) * 3, _rand(2, (rows, F), dtype), _rand(3, (rows,), "f32")
    if rows > 8:
        gu[2], gu[3, 0], gu[3, 1] = 0.0, 200.0, -200.0   # the exponential overflows on one side
    live = rows - rows // 4
    offs = torch.tensor([0, live], dtype=torch.int32, device=CUDA)
    g64, d64, w64 = _np(gu), _np(d), _np(rw)
    # relative error of a chain of about a dozen fp32 operations and expf (2 steps), times the value,
    # plus the error of 1 - s where it cancels (2^-24 of the terms' magnitude)
    eps = 24 * 2.0 ** -24
    h = torch.full((rows, F), 7.0, dtype=TORCH[dtype], device=CUDA)
    B.swiglu(gu.to(CUDA), clamp, mode, offsets=offs, h=h)
    ref = R.swiglu(g64, clamp, mode)
    err = np.abs(_np(h) - ref)[:live]
    assert (err <= ((R.STEP[dtype] + eps) * np.abs(ref) + 1e-37)[:live]).all()
    assert (_np(h)[live:] == 7).all()
    out = dict(dgu=torch.full((rows, 2 * F), 7.0, dtype=TORCH[dtype], device=CUDA),
               hw=torch.full((rows, F), 7.0, dtype=TORCH[dtype], device=CUDA),
               drow_weight=torch.full((rows,), 7.0, device=CUDA))
    B.swiglu_backward(gu.to(CUDA), d.to(CUDA), rw.to(CUDA), clamp, mode, offsets=offs, out=out)
    dgu, hw, drw = R.swiglu_backward(g64, d64, w64, clamp, mode)
    F64 = np.abs(d64 * w64[:, None])
    cl = clamp if clamp and mode == "preact" else np.inf
    g, u = np.clip(g64[:, :F], -cl, cl), np.clip(g64[:, F:], -cl, cl)
    s = R.sigmoid(g)
    scale = np.concatenate([F64 * np.abs(u) * s * (1 + np.abs(g)), F64 * np.abs(g) * s], 1)
    assert (np.abs(_np(out["dgu"]) - dgu) <= R.STEP[dtype] * np.abs(dgu) + eps * scale + 1e-37)[:live].all()
    assert (np.abs(_np(out["hw"]) - hw) <= (R.STEP[dtype] + eps) * np.abs(hw) + 1e-37)[:live].all()
    hm = np.abs(d64 * R.swiglu(g64, clamp, mode)).sum(1)
    assert (np.abs(_np(out["drow_weight"]) - drw) <= (F * 2.0 ** -24 + eps) * hm + 1e-37)[:live].all()
    for t in out.values():
        assert (_np(t)[live:] == 7).all()
    # in place: the gradient over gate|up
    buf = gu.to(CUDA).clone()
    r = B.swiglu_backward(buf, d.to(CUDA), rw.to(CUDA), clamp, mode, offsets=offs, out=dict(dgu=buf), need_hw=False,
                          need_drow_weight=False)
    assert r["hw"] is None and r["drow_weight"] is None
    assert torch.equal(buf[:live], out["dgu"][:live])


@pytest.mark.parametrize("clamp,mode", [(0.0, "preact"), (1.0, "preact"), (0.7, "output")])
def test_reference_backward_against_differences(clamp, mode):
    rng = np.random.default_rng(0)
    gu, d, w = rng.standard_normal((5, 16)) * 1.5, rng.standard_normal((5, 8)), rng.standard_normal(5)
    loss = lambda gu, w: (w[:, None] * R.swiglu(gu, clamp, mode) * d).sum()  # noqa: E731
    dgu, hw, drw = R.swiglu_backward(gu, d, w, clamp, mode)
    h = 1e-6
    for i in np.ndindex(gu.shape):
        p, m = gu.copy(), gu.copy()
        p[i] += h
        m[i] -= h
        assert abs((loss(p, w) - loss(m, w)) / (2 * h) - dgu[i]) < 1e-7
    for i in range(5):
        p, m = w.copy(), w.copy()
        p[i] += h
        m[i] -= h
        assert abs((loss(gu, p) - loss(gu, m)) / (2 * h) - drw[i]) < 1e-7
    np.testing.assert_allclose(hw, w[:, None] * R.swiglu(gu, clamp, mode))


@pytest.mark.gpu
def test_swiglu_keeps_nan_through_the_clamp(B):
    gu = torch.zeros((2, 32), device=CUDA)
    gu[0, 3], gu[1, 16 + 4] = float("nan"), float("nan")
    gu[1, 4] = 1.0
    for clamp, mode in ((0.0, "preact"), (1.0, "preact"), (1.0, "output")):
        h = B.swiglu(gu, clamp, mode)
        assert torch.isnan(h[0, 3]) and torch.isnan(h[1, 4]) and int(torch.isnan(h).sum()) == 2


# ------------------------------------------------------------------ runs of them together

def _route(B, cfg, x, wr):
    idx, w = B.route_topk(cfg, x, B.make_weights(dict(w_router=wr)))
    return B.dispatch(cfg, x, idx, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_of_the_expert_ffn(B, dtype):
    """Forward and backward of the routed experts, every gradient against float64."""
    T, D, F, E, k = 150, 256, 128, 6, 2
    cfg = B.make_config(E, k, D, F, act=dtype, expert=dtype)
    x, wr = _rand(1, (T, D), dtype).to(CUDA), _rand(2, (E, D), dtype, D ** -0.5).to(CUDA)
    wgu, wd = _rand(3, (E, 2 * F, D), dtype, D ** -0.5).to(CUDA), _rand(4, (E, D, F), dtype, F ** -0.5).to(CUDA)
    dy = _rand(5, (T * k, D), dtype).to(CUDA)
    m = _route(B, cfg, x, wr)
    offs, rw, xp = m["expert_offsets"], m["row_weight"], m["x_perm"]
    # forward
    gu = B.grouped_matmul(xp, wgu, offs)
    h = B.swiglu(gu, offsets=offs)
    y = B.grouped_matmul(h, wd, offs, row_weight=rw, out="f32")
    out = B.combine(cfg, y, m["slot_row"], T)
    # backward
    dh = B.grouped_matmul(dy, wd, offs, transposed=True)
    b = B.swiglu_backward(gu, dh, rw, offsets=offs)
    dwd = B.grouped_wgrad(dy, b["hw"], offs)
    dxp = B.grouped_matmul(b["dgu"], wgu, offs, transposed=True)
    dwgu = B.grouped_wgrad(b["dgu"], xp, offs)
    # the same in float64 with autograd, from the stored gate|up values on (they are the layer's own rounding)
    o = offs.tolist()
    X, WGU, WD, W = [v.double().requires_grad_() for v in (xp, wgu, wd, rw)]
    GU = torch.cat([X[o[e]:o[e + 1]] @ WGU[e].t() for e in range(E)])
    H = torch.nn.functional.silu(GU[:, :F]) * GU[:, F:]
    Y = torch.cat([H[o[e]:o[e + 1]] @ WD[e].t() for e in range(E)]) * W[:, None]
    Y.backward(dy.double())
    # the layer's roundings in bf16: gu, h (or hw), dh, dgu, each half a step, and the output's
    tol = {"f32": 2e-6, "bf16": 6 * 2.0 ** -8}[dtype]
    for name, got, want in (("y", y, Y), ("dwd", dwd, WD.grad), ("dx", dxp, X.grad), ("dwgu", dwgu, WGU.grad),
                            ("drw", b["drow_weight"], W.grad)):
        got, want = got.double(), want.detach()
        rms = float(want.square().mean().sqrt())
        rel = float((got - want).square().mean().sqrt()) / rms
        assert rel <= tol, f"{name}: {rel:.3g}"
    ref = torch.zeros(T, D, dtype=torch.float64, device=CUDA).index_add_(0, m["row_token"].long(), Y.detach())
    assert float((out.double() - ref).square().mean().sqrt()) <= tol * float(ref.square().mean().sqrt())


@pytest.mark.gpu
def test_layer_in_four_bits(B):
    """Route, dispatch maps, quantising gather, products in 4 bits, SwiGLU into 4 bits, combine."""
    T, D, F, E, k = 130, 512, 256, 8, 2
    cfg = B.make_config(E, k, D, F, capacity=40)
    x, wr = _rand(1, (T, D), "bf16").to(CUDA), _rand(2, (E, D), "bf16", D ** -0.5).to(CUDA)
    wgu, wd = _rand(3, (E, 2 * F, D), "bf16", D ** -0.5).to(CUDA), _rand(4, (E, D, F), "bf16", F ** -0.5).to(CUDA)
    q1, q2 = B.quantize_nvfp4(wgu.view(-1, D)), B.quantize_nvfp4(wd.view(-1, F))
    idx, w = B.route_topk(cfg, x, B.make_weights(dict(w_router=wr)))
    m = B.dispatch(cfg, x, idx, w, gather=False)
    offs = m["expert_offsets"]
    a = B.quantize_nvfp4(x, row_token=m["row_token"], offsets=offs)
    gu = B.grouped_matmul_nvfp4(a["codes"], a["scales"], q1["codes"].view(E, 2 * F, -1),
                                q1["scales"].view(E, 2 * F, -1), offs, a["row_scale"], q1["row_scale"].view(E, 2 * F))
    h = B.swiglu_quantize_nvfp4(gu, offsets=offs)
    y = B.grouped_matmul_nvfp4(h["codes"], h["scales"], q2["codes"].view(E, D, -1), q2["scales"].view(E, D, -1), offs,
                               h["row_scale"], q2["row_scale"].view(E, D), row_weight=m["row_weight"], out="f32")
    out = B.combine(cfg, y, m["slot_row"], T)
    # float64, stage by stage on the GPU's own inputs of each
    o = offs.tolist()
    n = o[-1]
    assert n < T * k, "the capacity drops rows"
    rt = m["row_token"].cpu().numpy()[:n]
    _same(a, R.quantize(np.concatenate([_np(x)[rt], np.zeros((T * k - n, D))]), True), np.arange(n))
    dec = lambda q, lead: R.decode(q["codes"].cpu().numpy().reshape(*lead, -1),  # noqa: E731
                                   q["scales"].cpu().numpy().reshape(*lead, -1), _np(q["row_scale"]).reshape(lead))
    live = lambda q: {k: v[:n] for k, v in q.items() if v is not None}  # noqa: E731
    ref, mag = R.matmul(dec(live(a), (n,)), dec(q1, (E, 2 * F)), o)
    _check(_np(gu)[:n], ref, mag, D, "bf16", "gate|up")
    ref, mag = R.matmul(dec(live(h), (n,)), dec(q2, (E, D)), o, row_weight=_np(m["row_weight"])[:n])
    _check(_np(y)[:n], ref, mag, F, "f32", "y", extra=8)
    want = np.zeros((T, D))
    np.add.at(want, rt, _np(y)[:n])
    np.testing.assert_allclose(_np(out), want, rtol=1e-6, atol=1e-6)
    # 4 bits keep the layer's output near the bf16 layer's (two operands quantised twice, each by at
    # most 1/4 of a value in its widest code interval: well inside half the output's norm)
    full = B.combine(cfg, B.grouped_matmul(B.swiglu(B.grouped_matmul(x[m["row_token"].clamp(0, T - 1).long()], wgu, offs)),
                                           wd, offs, row_weight=m["row_weight"], out="f32"), m["slot_row"], T)
    assert float((out - full).norm()) < 0.5 * float(full.norm())


# ------------------------------------------------------------------ streams, graphs, workspaces

def _call(B, kind, seed, ws):
    sizes = [40, 0, 90, 7]
    offs = torch.tensor(_offsets(sizes), dtype=torch.int32, device=CUDA)
    if kind == "nvfp4":
        a, sa, ra = (torch.from_numpy(v).to(CUDA) for v in _nvfp4(seed, (137, 512)))
        w, sw, rw = (torch.from_numpy(v).to(CUDA) for v in _nvfp4(seed + 1, (4, 192, 512)))
        return lambda s=None: B.grouped_matmul_nvfp4(a, sa, w, sw, offs, ra, rw, ws=ws, stream=s)
    a, dy = _rand(seed, (137, 256), "bf16").to(CUDA), _rand(seed + 1, (137, 192), "bf16").to(CUDA)
    w = _rand(seed + 2, (4, 192, 256), "bf16").to(CUDA)
    if kind == "matmul":
        return lambda s=None: B.grouped_matmul(a, w, offs, ws=ws, stream=s)
    if kind == "wgrad":
        return lambda s=None: B.grouped_wgrad(dy, a, offs, ws=ws, stream=s)
    if kind == "quantize":
        return lambda s=None: B.swiglu_quantize_nvfp4(a, values=True, stream=s)["values"]
    return lambda s=None: B.swiglu_backward(a, a[:, :128].contiguous(), stream=s)["dgu"]


KINDS = ["matmul", "wgrad", "nvfp4", "quantize", "swiglu"]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_captured_replayed_and_on_other_streams(B, kind):
    ws = B.workspace(256)
    one, two = _call(B, kind, 10, ws), _call(B, kind, 20, ws)  # both share the workspace
    want = [one().clone(), two().clone()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [f(s) for _ in range(3) for f, s in zip((one, two), streams)]  # at the same time
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])
    graphs, outs = [], []
    for f in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for _ in range(2):
        for t in outs:
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
    B.check_device_status(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_every_time(B, kind):
    f = _call(B, kind, 30, B.workspace(256))
    first = f().clone()
    for _ in range(5):
        assert torch.equal(f(), first)


# ------------------------------------------------------------------ refusals (no GPU)

def _g(B, **kw):
    base = dict(groups=4, rows=10, n=64, k=64, dtype=B.MOE_BF16, out_dtype=B.MOE_BF16)
    base.update(kw)
    return B.MoEGrouped(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), 1), (dict(groups=1025), 2), (dict(rows=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(n=60), 2),
    (dict(k=60), 2), (dict(dtype=7), 1), (dict(dtype=-1), 1), (dict(out_dtype=2), 1), (dict(dtype=0, out_dtype=1), 2),
    (dict(dtype=2), 1), (dict(rows=2 ** 31 - 1), 2)])
def test_products_refuse_sizes_and_types(B, kw, status):
    g = _g(B, **kw)
    r = ctypes.byref(g)
    assert B.lib.moe_grouped_matmul(r, 16, 16, 16, 0, None, 16, 16, 256, None) == status
    assert B.lib.moe_grouped_wgrad(r, 16, 16, 16, 0, 16, 16, 256, None) == status
    if kw != dict(dtype=2):
        assert B.lib.moe_grouped_workspace_size(r) == 0


def test_products_refuse_pointers_and_workspaces(B):
    lib, r = B.lib, ctypes.byref(_g(B))
    ok = dict(a=16, offs=16, w=16, rw=None, y=16, ws=16, n=256)

    def mm(**kw):
        v = {**ok, **kw}
        return lib.moe_grouped_matmul(r, v["a"], v["offs"], v["w"], 0, v["rw"], v["y"], v["ws"], v["n"], None)

    def wg(**kw):
        v = {**ok, **kw}
        return lib.moe_grouped_wgrad(r, v["a"], v["w"], v["offs"], 0, v["y"], v["ws"], v["n"], None)

    for f in (mm, wg):
        for kw in (dict(a=None), dict(a=24), dict(w=None), dict(w=20), dict(y=None), dict(y=8), dict(ws=None),
                   dict(ws=18), dict(offs=None), dict(offs=18)):
            assert f(**kw) == B.MOE_ERR_INVALID_ARG, kw
        assert f(n=255) == B.MOE_ERR_WORKSPACE
    assert mm(rw=18) == B.MOE_ERR_INVALID_ARG
    assert lib.moe_grouped_matmul(None, 16, 16, 16, 0, None, 16, 16, 256, None) == B.MOE_ERR_INVALID_ARG
    # no rows: nothing to read
    r0 = ctypes.byref(_g(B, rows=0))
    assert lib.moe_grouped_matmul(r0, None, 16, None, 0, None, None, 16, 256, None) == B.MOE_OK
    assert lib.moe_grouped_wgrad(r0, None, None, 16, 1, 16, 16, 256, None) == B.MOE_OK


def test_nvfp4_product_refuses(B):
    def f(a=16, sa=16, ra=None, offs=16, w=16, sw=16, rw=None, wt=None, y=16, ws=16, n=256, **kw):
        g = _g(B, **{**dict(dtype=B.MOE_NVFP4), **kw})
        return B.lib.moe_grouped_matmul_nvfp4(ctypes.byref(g), a, sa, ra, offs, w, sw, rw, wt, y, ws, n, None)

    for kw in (dict(a=None), dict(a=24), dict(sa=None), dict(sa=8), dict(w=None), dict(w=24), dict(sw=None), dict(sw=4),
               dict(y=None), dict(y=24), dict(ra=2), dict(rw=2), dict(wt=1), dict(offs=None), dict(dtype=B.MOE_BF16)):
        assert f(**kw) == B.MOE_ERR_INVALID_ARG, kw
    assert f(k=48) == B.MOE_ERR_UNSUPPORTED
    assert f(n=12) == B.MOE_ERR_WORKSPACE
    assert f(rows=0, a=None, w=None, y=None) == B.MOE_OK


def test_quantize_and_swiglu_refuse(B):
    lib, bf = B.lib, B.MOE_BF16

    def q(rows=4, cols=64, dt=bf, x=16, xr=4, rt=None, live=None, c=16, s=16, rs=None, v=None):
        return lib.moe_quantize_nvfp4(rows, cols, dt, x, xr, rt, live, c, s, rs, v, None)

    for kw in (dict(rows=-1), dict(cols=0), dict(dt=2), dict(x=None), dict(x=8), dict(xr=0), dict(xr=3), dict(c=None),
               dict(c=8), dict(s=None), dict(v=8), dict(rs=2), dict(rt=2), dict(live=2)):
        assert q(**kw) == B.MOE_ERR_INVALID_ARG, kw
    assert q(cols=24) == B.MOE_ERR_UNSUPPORTED
    assert q(rows=0, x=None, xr=0) == B.MOE_OK

    def sq(rows=4, cols=64, gu=16, clamp=0.0, mode=0, c=16, s=16, v=None):
        return lib.moe_swiglu_quantize_nvfp4(rows, cols, bf, gu, clamp, mode, None, c, s, None, v, None)

    def sw(rows=4, F=64, dt=bf, gu=16, clamp=0.0, mode=0, h=16):
        return lib.moe_swiglu(rows, F, dt, gu, clamp, mode, None, h, None)

    def sb(rows=4, F=64, gu=16, dh=16, rw=None, clamp=0.0, mode=0, dgu=16, hw=None, drw=None):
        return lib.moe_swiglu_backward(rows, F, bf, gu, dh, rw, clamp, mode, None, dgu, hw, drw, None)

    for f in (sq, sw, sb):
        for kw in (dict(rows=-1), dict(gu=None), dict(gu=8), dict(clamp=-1.0), dict(clamp=float("nan")), dict(mode=2)):
            assert f(**kw) == B.MOE_ERR_INVALID_ARG, kw
        assert f(rows=0, gu=None) == B.MOE_OK
    assert sq(cols=40) == sw(F=12) == sb(F=12) == B.MOE_ERR_UNSUPPORTED
    for kw in (dict(dh=None), dict(dgu=None), dict(hw=8), dict(rw=2), dict(drw=2)):
        assert sb(**kw) == B.MOE_ERR_INVALID_ARG, kw


def test_binding_refuses_tensors(B):
    bf = torch.bfloat16
    a, w, offs = torch.zeros(10, 64, dtype=bf), torch.zeros(4, 32, 64, dtype=bf), torch.zeros(5, dtype=torch.int32)
    gu = torch.zeros(10, 64, dtype=bf)
    codes, scales = torch.zeros(10, 32, dtype=torch.uint8), torch.zeros(10, 4, dtype=torch.uint8)
    wc, wsc = torch.zeros(4, 8, 32, dtype=torch.uint8), torch.zeros(4, 8, 4, dtype=torch.uint8)
    bad = [
        lambda: B.grouped_matmul(a, w, offs),                                     # not on a GPU
        lambda: B.grouped_matmul(a.t(), w, offs),
        lambda: B.grouped_matmul(a, w[0], offs),
        lambda: B.grouped_matmul(a, w.float(), offs),
        lambda: B.grouped_matmul(a.half(), w.half(), offs),
        lambda: B.grouped_matmul(a, w, offs[:-1]),
        lambda: B.grouped_matmul(a, w, offs.long()),
        lambda: B.grouped_matmul(a, w, None),
        lambda: B.grouped_matmul(a, w, offs, transposed=True),
        lambda: B.grouped_matmul(a, w, offs, row_weight=torch.zeros(9)),
        lambda: B.grouped_matmul(a, w, offs, y=torch.zeros(10, 31, dtype=bf)),
        lambda: B.grouped_wgrad(a, a[:9], offs),
        lambda: B.grouped_wgrad(a, a, offs, accumulate=True),
        lambda: B.grouped_wgrad(a, a, offs, dw=torch.zeros(4, 64, 63, dtype=bf)),
        lambda: B.grouped_matmul_nvfp4(codes, scales, wc, wsc, offs),
        lambda: B.grouped_matmul_nvfp4(codes, scales[:, :3].contiguous(), wc, wsc, offs),
        lambda: B.grouped_matmul_nvfp4(codes, scales, wc, wsc.float(), offs),
        lambda: B.grouped_matmul_nvfp4(codes, scales, wc, wsc, offs, a_row_scale=torch.zeros(10, dtype=bf)),
        lambda: B.quantize_nvfp4(a),
        lambda: B.quantize_nvfp4(a.half()),
        lambda: B.quantize_nvfp4(a, row_token=offs.long()),
        lambda: B.quantize_nvfp4(a, offsets=offs.float()),
        lambda: B.swiglu(gu),
        lambda: B.swiglu(gu[:, :63].contiguous()),
        lambda: B.swiglu_backward(gu, gu),
        lambda: B.swiglu_backward(gu, gu[:, :32].contiguous(), need_hw=False, out=dict(hw=gu)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
