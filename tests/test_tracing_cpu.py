"""torch.jit.trace of the layer norm, the adapters and the MXFP4 linear outside autograd, with the kernels replaced by their formulas on the
CPU: the traced call computes, and does not hand out memory that nothing was written to."""
import pytest
import torch

from float8linear_tensorwise_amax_amd import f8lin
from float8linear_tensorwise_amax_amd import module as m


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    """(written through numpy: torch's tracer sees nothing of them, as of the library's calls)"""
    def layer_norm_forward(x, y, weight=None, bias=None, eps=1e-5, stats=None, y_amax=None, stream=None):
        y.detach().numpy()[...] = torch.nn.functional.layer_norm(x, x.shape[-1:], weight, bias, eps).numpy()

    def lora_forward(base, x, a, b, scales, plan, y, h=None, ws=None, stream=None):
        base, x, a, b = (t.detach().numpy() for t in (base, x, a, b))
        y.detach().numpy()[...] = base + x @ a[0].T @ b[0].T

    for f in (layer_norm_forward, lora_forward):
        monkeypatch.setattr(f8lin, f.__name__, f)
    monkeypatch.setattr(f8lin, "lora_plan", lambda index, plan, stream=None: plan.written())
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))


def traced(f, *args):
    with torch.no_grad():
        t = torch.jit.trace(f, args, check_trace=False)
        junk = [torch.full_like(f(*args), float("nan")) for _ in range(8)]  # (what an empty tensor would hold)
        del junk
        others = [a + torch.randn_like(a) for a in args]
        return t(*others), f(*others)


@pytest.mark.filterwarnings("ignore")
def test_layer_norm():
    norm = m.LayerNorm(24)
    got, want = traced(norm, torch.randn(5, 24))
    assert torch.equal(got, want)
    got, want = traced(lambda x: m.layer_norm(x), torch.randn(2, 5, 24))
    assert torch.equal(got, want)


@pytest.mark.filterwarnings("ignore")
def test_adapters():
    batch = m.LoraBatch(torch.zeros(5, dtype=torch.int64), 1)
    a, b = torch.randn(1, 3, 8), torch.randn(1, 12, 3)
    got, want = traced(lambda base, x: m.lora_add(base, x, a, b, batch), torch.randn(5, 12), torch.randn(5, 8))
    assert torch.equal(got, want)


@pytest.mark.filterwarnings("ignore")
def test_mxfp4_linear(monkeypatch):
    def mxfp4_forward(x, w, y, *args, **kw):
        y.detach().numpy()[...] = (x @ w.t()).numpy()

    monkeypatch.setattr(f8lin, "mxfp4_forward", mxfp4_forward)
    monkeypatch.setattr(f8lin, "new_mxfp4s", lambda shapes, dev, *args: (None, [None] * len(shapes)))
    w = torch.randn(12, 8)
    got, want = traced(lambda x: m.mxfp4_linear(x, w), torch.randn(5, 8))
    assert torch.equal(got, want)
    packed = f8lin.MXFP4Tensor(torch.zeros((12, 16), dtype=torch.uint8), torch.zeros((12, 16), dtype=torch.uint8), 12, 8)
    with pytest.raises(RuntimeError, match="traced"), torch.no_grad():
        torch.jit.trace(lambda x: m.mxfp4_linear(x, packed), (torch.randn(5, 8),), check_trace=False)
