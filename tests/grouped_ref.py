"""Plain float64 references of the grouped products, NVFP4 and SwiGLU (not a test module).

Written from the definitions in include/moe.h with numpy; nothing of the
library is used.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite e4m3 magnitudes by code: subnormals m 2^-9, then (8 + m) 2^(e - 10)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])

STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative to the value


def nearest_even(v: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Codes of the nearest entries of an ascending table, ties to the even code, saturating."""
    hi = np.clip(np.searchsorted(table, v), 0, len(table) - 1)
    lo = np.clip(hi - 1, 0, None)
    up, down = table[hi] - v, v - table[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(v >= table[-1], len(table) - 1, np.where(take_hi, hi, lo))


def quantize(x: np.ndarray, row_scaled: bool):
    """x float64 [rows, cols] -> codes uint8 [rows, cols] (sign in bit 3), scale bytes, row scales, values."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 16, 16)
    amax = np.abs(b).max(axis=2)
    bad = ~np.isfinite(b).all(axis=2)
    good = np.where(bad, 0.0, amax)
    rs = np.ones(rows)
    if row_scaled:
        top = good.max(axis=1)
        m, e = np.frexp(top)                      # top = m 2^e, m in [1/2, 1); 2688 = 0.65625 * 2^12
        exp = np.maximum(e - 12 + (m > 0.65625), -110)
        rs = np.where(top > 0, np.ldexp(1.0, exp), 1.0)
    s8 = nearest_even(np.minimum(good / rs[:, None] / 6.0, 448.0), E4M3).astype(np.uint8)
    s = E4M3[s8]
    d = s * rs[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where((s > 0)[..., None] & ~bad[..., None], np.abs(b) / d[..., None], 0.0)
    code = nearest_even(np.minimum(t, 6.0), E2M1).astype(np.uint8)
    sign = np.signbit(b) & (s > 0)[..., None] & ~bad[..., None]   # codes are 0 where the scale is
    values = np.where(sign, -1.0, 1.0) * E2M1[code] * d[..., None]
    values[bad] = np.nan
    code = code | (sign.astype(np.uint8) << 3)
    s8[bad] = 0x7F
    return code.reshape(rows, cols), s8, rs, values.reshape(rows, cols)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def decode(packed: np.ndarray, s8: np.ndarray, rs=None) -> np.ndarray:
    code = unpack(packed)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    v = v * np.repeat(E4M3[s8], 16, axis=-1)
    return v if rs is None else v * np.asarray(rs, np.float64)[..., None]


def segments(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def matmul(a, w, offsets, transposed=False, row_weight=None):
    """(y, sum of the terms' magnitudes) float64; rows of no group are NaN."""
    N = w.shape[2] if transposed else w.shape[1]
    y, mag = np.full((a.shape[0], N), np.nan), np.zeros((a.shape[0], N))
    for e, r0, r1 in segments(offsets):
        we = w[e] if transposed else w[e].T
        y[r0:r1] = a[r0:r1] @ we
        mag[r0:r1] = np.abs(a[r0:r1]) @ np.abs(we)
    if row_weight is not None:
        y, mag = y * row_weight[:, None], mag * np.abs(row_weight)[:, None]
    return y, mag


def wgrad(dy, a, offsets):
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], a.shape[1]))
    mag = np.zeros_like(dw)
    for e, r0, r1 in segments(offsets):
        dw[e] = dy[r0:r1].T @ a[r0:r1]
        mag[e] = np.abs(dy[r0:r1]).T @ np.abs(a[r0:r1])
    return dw, mag


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(gu, clamp=0.0, mode="preact"):
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    if clamp and mode == "preact":
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    h = g * sigmoid(g) * u
    return np.clip(h, -clamp, clamp) if clamp and mode == "output" else h


def swiglu_backward(gu, d, row_weight, clamp=0.0, mode="preact"):
    """(dgu, hw, drow_weight) of sum(row_weight * h * d)."""
    F = gu.shape[1] // 2
    g0, u0 = gu[:, :F], gu[:, F:]
    g, u = g0, u0
    pre = clamp and mode == "preact"
    if pre:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    s = sigmoid(g)
    h = g * s * u
    w = row_weight[:, None]
    dg, du = d * w * u * s * (1 + g * (1 - s)), d * w * g * s
    if pre:
        dg, du = np.where(np.abs(g0) > clamp, 0, dg), np.where(np.abs(u0) > clamp, 0, du)
    elif clamp:
        out = np.abs(h) > clamp
        dg, du, h = np.where(out, 0, dg), np.where(out, 0, du), np.clip(h, -clamp, clamp)
    return np.concatenate([dg, du], 1), w * h, (d * h).sum(1)
