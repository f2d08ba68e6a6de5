"""Operators given a stream that is still busy, and inputs that the caller drops right after the call:
their memory must not be handed out again before the stream has read them."""
import pytest
import torch

CUDA = "cuda"


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


ROWS = 512
CALLS = {
    "matmul": lambda B, x, s: B.grouped_matmul(x(ROWS, 256), x(1, 64, 256), None, stream=s),
    "wgrad": lambda B, x, s: B.grouped_wgrad(x(ROWS, 64), x(ROWS, 256), None, stream=s),
    "quantize": lambda B, x, s: B.quantize_nvfp4(x(ROWS, 256), values=True, stream=s)["values"],
    "swiglu_quantize": lambda B, x, s: B.swiglu_quantize_nvfp4(x(ROWS, 512), values=True, stream=s)["values"],
    "swiglu": lambda B, x, s: B.swiglu(x(ROWS, 512), stream=s),
    "swiglu_backward": lambda B, x, s: B.swiglu_backward(x(ROWS, 512), x(ROWS, 256), x(ROWS).float(), stream=s)["dgu"],
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", [*CALLS, "nvfp4"])
def test_inputs_dropped_before_the_stream_reads_them(B, name):
    one = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=CUDA)  # noqa: E731
    call = CALLS.get(name)
    if call is None:
        w = B.quantize_nvfp4(one(64, 256))

        def call(B, x, s):
            codes = x(ROWS, 128).byte() * 34           # two codes of 1.0
            return B.grouped_matmul_nvfp4(codes, x(ROWS, 16).byte() * 56, w["codes"].view(1, 64, -1),
                                          w["scales"].view(1, 64, -1), None, stream=s)
    want = call(B, one, None).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(600_000_000)                 # about 0.3 s; the inputs are written meanwhile
    before = torch.cuda.Event()
    got = call(B, one, s)                              # its inputs live no longer than the call
    others = [torch.full((n,), 5, dtype=torch.bfloat16, device=CUDA) for n in (ROWS, ROWS * 16, ROWS * 64, ROWS * 128,
                                                                               ROWS * 256, ROWS * 512, 64 * 256) for _ in range(4)]
    before.record(s)
    assert not before.query(), "the stream was meant to be busy still"
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del others
