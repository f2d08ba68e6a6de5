"""README's training step of the experts, run as it stands there, against float64 autograd.

Tolerance, relative to the rms of each result: in bf16 five stored roundings lie on the longest way
(gate|up, h or hw, dh, dgu, the result), each half a step of 2^-8 of a value; the fp32 sums of up to
512 terms in a row of three products add less than 512 * 2^-23 of their terms' magnitude each, about
0.64 * sqrt(512) = 14 times the result's rms: 3 * 14 * 2^-14 = 2.6e-3."""
import os
import re

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "cuda"


def _block():
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md"), encoding="utf-8").read(), re.S)
    return next(b for b in blocks if "dw_gate_up" in b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("capacity", [0, 60, 40])
def test_training_step(dtype, capacity):
    from mixture_experts_layer_sqrt_b200 import binding as B
    T, D, F, E, k = 150, 256, 128, 6, 2
    td = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    cfg = B.make_config(E, k, D, F, capacity=capacity, act=dtype, expert=dtype)
    rng = np.random.default_rng(1)
    new = lambda s, scale=1.0: torch.from_numpy((rng.standard_normal(s) * scale).astype(np.float32)).to(td).to(CUDA)  # noqa: E731
    x, dout, w_router = new((T, D)), new((T, D)), new((E, D), D ** -0.5)
    w_gate_up, w_down = new((E, 2 * F, D), D ** -0.5), new((E, D, F), F ** -0.5)
    topk_idx, topk_w = B.route_topk(cfg, x, B.make_weights(dict(w_router=w_router)))
    r = dict(B=B, cfg=cfg, T=T, x=x, dout=dout, topk_idx=topk_idx, topk_w=topk_w, w_gate_up=w_gate_up, w_down=w_down)
    exec(_block(), r)
    kept = r["m"]["slot_row"] >= 0
    if capacity == 40:  # 240 places for 300 assignments
        assert int(kept.sum()) <= 240
    # float64, from the routing on, the kept assignments only
    X, WGU, WD, W = [v.double().requires_grad_() for v in (x, w_gate_up, w_down, topk_w)]
    out = torch.zeros(T, D, dtype=torch.float64, device=CUDA)
    for e in range(E):
        t, j = ((topk_idx == e) & kept).nonzero(as_tuple=True)
        gu = X[t] @ WGU[e].t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, (h @ WD[e].t()) * W[t, j][:, None])
    out.backward(dout.double())
    drw = torch.zeros(T, k, device=CUDA)
    drw[kept] = r["b"]["drow_weight"][r["m"]["slot_row"][kept].long()]
    tol = 2.6e-3 + (5 * 2.0 ** -8 if dtype == "bf16" else 0.0)
    for name, got, want in (("out", r["out"], out), ("dx", r["dx"], X.grad), ("dw_gate_up", r["dw_gate_up"], WGU.grad),
                            ("dw_down", r["dw_down"], WD.grad), ("drow_weight", drw, W.grad)):
        want = want.detach()
        err = float((got.double() - want).square().mean().sqrt()) / float(want.square().mean().sqrt())
        assert err <= tol, f"{name}: {err:.3g}"
