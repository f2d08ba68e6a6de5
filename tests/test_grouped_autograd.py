"""The grouped operators take no part in autograd: where it would follow a tensor they refuse it
instead of returning a result without its gradient; inside an autograd function they work."""
import pytest
import torch

CUDA = "cuda"


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_sqrt_b200 import build
    build.build()
    from mixture_experts_layer_sqrt_b200 import binding
    return binding


def _calls(B, dev):
    bf = torch.bfloat16
    t = dict(a=torch.zeros(4, 64, dtype=bf), w=torch.zeros(1, 64, 64, dtype=bf), rw=torch.zeros(4), ra=torch.zeros(4),
             wr=torch.zeros(1, 64), y=torch.zeros(4, 64, dtype=bf), dw=torch.zeros(1, 64, 64, dtype=bf),
             dh=torch.zeros(4, 32, dtype=bf), q=torch.zeros(4, 32, dtype=torch.uint8),
             s=torch.zeros(4, 4, dtype=torch.uint8), qw=torch.zeros(1, 64, 32, dtype=torch.uint8),
             sw=torch.zeros(1, 64, 4, dtype=torch.uint8), h=torch.zeros(4, 32, dtype=bf))
    t = {k: v.to(dev) for k, v in t.items()}
    return t, [
        ("a w rw y", lambda: B.grouped_matmul(t["a"], t["w"], None, row_weight=t["rw"], y=t["y"])),
        ("a y dw", lambda: B.grouped_wgrad(t["y"], t["a"], None, dw=t["dw"])),
        ("ra wr rw y", lambda: B.grouped_matmul_nvfp4(t["q"], t["s"], t["qw"], t["sw"], None, t["ra"], t["wr"], t["rw"],
                                                      y=t["y"])),
        ("a", lambda: B.quantize_nvfp4(t["a"])),
        ("a", lambda: B.swiglu_quantize_nvfp4(t["a"])),
        ("a h", lambda: B.swiglu(t["a"], h=t["h"])),
        ("a dh rw", lambda: B.swiglu_backward(t["a"], t["dh"], t["rw"])),
    ]


def test_a_tensor_that_requires_grad_is_refused(B):
    t, calls = _calls(B, "cpu")
    for names, f in calls:
        for n in names.split():
            t[n].requires_grad_(True)
            with pytest.raises(ValueError, match="requires grad"):
                f()
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # only the missing GPU is left
                f()
            t[n].requires_grad_(False)
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.mark.gpu
def test_no_grad_and_autograd_functions(B):
    t, calls = _calls(B, CUDA)
    for names, f in calls:
        for n in names.split():
            t[n].requires_grad_(True)
            with pytest.raises(ValueError, match="requires grad"):
                f()
            with torch.no_grad():
                f()
            t[n].requires_grad_(False)
        f()

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, w, offs):
            ctx.save_for_backward(a, w, offs)
            return B.grouped_matmul(a, w, offs)

        @staticmethod
        def backward(ctx, dy):
            a, w, offs = ctx.saved_tensors
            return B.grouped_matmul(dy, w, offs, transposed=True), B.grouped_wgrad(dy, a, offs), None

    # small whole numbers: every sum is exact, and so are the gradients
    g = torch.Generator().manual_seed(0)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g).float()  # noqa: E731
    a, w, dy = (whole(*s).to(CUDA) for s in ((30, 64), (3, 72, 64), (30, 72)))
    offs = torch.tensor([0, 11, 11, 30], dtype=torch.int32, device=CUDA)
    a.requires_grad_(True), w.requires_grad_(True)
    Product.apply(a, w, offs).backward(dy)
    A, W = a.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    torch.cat([A[:11] @ W[0].t(), A[11:] @ W[2].t()]).backward(dy.double())
    assert torch.equal(a.grad.double(), A.grad) and torch.equal(w.grad.double(), W.grad)
