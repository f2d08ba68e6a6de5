"""A timeout that a grouped product records reaches a caller who passes no workspace."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "cuda"


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def test_status_workspace_refuses(B):
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert B.lib.moe_status_workspace(None, ctypes.byref(n)) == B.MOE_ERR_INVALID_ARG
    assert B.lib.moe_status_workspace(ctypes.byref(p), None) == B.MOE_ERR_INVALID_ARG


def _calls(B):
    a, w = torch.ones(5, 64, device=CUDA).bfloat16(), torch.ones(2, 64, 64, device=CUDA).bfloat16()
    offs = torch.tensor([0, 2, 5], dtype=torch.int32, device=CUDA)
    q, qw = B.quantize_nvfp4(a), B.quantize_nvfp4(w.view(-1, 64))
    return [lambda s=None: B.grouped_matmul(a, w, offs, stream=s), lambda s=None: B.grouped_wgrad(a, a, offs, stream=s),
            lambda s=None: B.grouped_matmul_nvfp4(q["codes"], q["scales"], qw["codes"].view(2, 64, 32),
                                                  qw["scales"].view(2, 64, 4), offs, stream=s)]


class _Recorded:
    """The library, with the workspace of every grouped product noted."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if not name.startswith("moe_grouped_"):
            return f
        return lambda *a: (self.seen.append(a[-3:-1]), f(*a))[1]   # (ws, ws_bytes), before the stream


@pytest.mark.gpu
def test_calls_without_a_workspace_share_one_that_can_be_read(B, monkeypatch):
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert B.lib.moe_status_workspace(ctypes.byref(p), ctypes.byref(n)) == B.MOE_OK and n.value == 256
    rec = _Recorded(B.lib)
    monkeypatch.setattr(B, "lib", rec)
    for s in (None, torch.cuda.Stream()):
        for f in _calls(B):
            f(s)
    torch.cuda.synchronize()
    assert rec.seen == [(p.value, 256)] * 6
    B.check_device_status()


@pytest.mark.gpu
def test_a_timeout_is_seen_without_a_workspace(B):
    B.check_device_status()
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    B.lib.moe_status_workspace(ctypes.byref(p), ctypes.byref(n))
    s = torch.cuda.Stream()
    assert B.lib.moe_selftest_wait_timeout(p, n, s.cuda_stream) == B.MOE_OK  # a bounded wait that runs out, 2 s
    with pytest.raises(B.MoEError) as e:
        B.check_device_status(stream=s)
    assert e.value.status == B.MOE_ERR_DEVICE_TIMEOUT
    B.check_device_status(stream=s)                                          # read and cleared
    for f in _calls(B):
        f()
    B.check_device_status()


@pytest.mark.gpu
def test_first_use_inside_a_capture():
    code = """
import torch
from mixture_experts_layer_sqrt_b200 import binding as B
a, w = torch.ones(5, 64, device="cuda").bfloat16(), torch.ones(2, 72, 64, device="cuda").bfloat16()
offs = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, dw = B.grouped_matmul(a, w, offs), B.grouped_wgrad(a, a, offs)
for _ in range(2):
    y.zero_(), dw.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert (y == 64).all() and (dw[0] == 2).all() and (dw[1] == 3).all()
B.check_device_status()
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
