"""Two host threads make the first calls of the grouped operators at the same time, in a fresh
process and with the library that users load: what is asked for once per device and kernel is then
asked for by both."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import threading
import torch
from mixture_experts_layer_sqrt_b200 import binding as B

assert B.lib.moe_checked_build() == 0
g = torch.Generator().manual_seed(3)
whole = lambda *s: torch.randint(-3, 4, s, generator=g).float().cuda()   # small whole numbers: exact sums
x, w, dy = whole(700, 256), whole(4, 192, 256), whole(700, 192)
offs = torch.tensor([0, 300, 300, 690, 700], dtype=torch.int32, device="cuda")
code = torch.randint(0, 256, (700, 128), generator=g, dtype=torch.uint8).cuda()
wcode = torch.randint(0, 256, (4, 192, 128), generator=g, dtype=torch.uint8).cuda()
one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")   # scale 1
few = torch.tensor([0, 5, 5, 9, 10], dtype=torch.int32, device="cuda")
sc, wsc = one(700, 16), one(4, 192, 16)
xb, wb, dyb = x.bfloat16(), w.bfloat16(), dy.bfloat16()
calls = [
    lambda: B.grouped_matmul(xb, wb, offs, out="f32"), lambda: B.grouped_matmul(xb[:10], wb, few, out="f32"),
    lambda: B.grouped_matmul(dyb, wb, offs, transposed=True, out="f32"), lambda: B.grouped_matmul(x, w, offs),
    lambda: B.grouped_wgrad(dyb, xb, offs, out="f32"),
    lambda: B.grouped_matmul_nvfp4(code, sc, wcode, wsc, offs, out="f32"),
    lambda: B.grouped_matmul_nvfp4(code[:10], sc[:10], wcode, wsc, few, out="f32"),
    lambda: B.quantize_nvfp4(xb, values=True)["values"].float(), lambda: B.swiglu(x), lambda: B.swiglu_backward(x, dy[:, :128].contiguous())["dgu"],
]
torch.cuda.synchronize()
got, errors, start = [[], []], [], threading.Barrier(2)

def run(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for f in calls:
                got[i].append(f())
                start.wait()
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append(e)
        start.abort()

threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
torch.cuda.synchronize()
B.check_device_status()
for a, b, f in zip(got[0], got[1], calls):
    assert torch.equal(a, b) and torch.equal(a, f())
groups = [(0, 0, 300), (2, 300, 690), (3, 690, 700)]
y = torch.cat([x[a:b].double() @ w[e].double().t() for e, a, b in groups])
assert torch.equal(got[0][0].double(), y) and torch.equal(got[0][3].double(), y)
assert torch.equal(got[0][2].double(), torch.cat([dy[a:b].double() @ w[e].double() for e, a, b in groups]))
dw = torch.zeros(4, 192, 256, dtype=torch.float64, device="cuda")
for e, a, b in groups:
    dw[e] = dy[a:b].double().t() @ x[a:b].double()
assert torch.equal(got[0][4].double(), dw)
print("same")
"""


@pytest.mark.gpu
def test_first_calls_from_two_threads_at_once():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
