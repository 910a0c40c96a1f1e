"""MXFP4 linears and gradient clipping next to autograd's own bookkeeping: tangents, version counters, shared layers."""
import pytest
import torch
import torch.nn as nn
from torch.autograd import forward_ad

from test_gpu_mxfp4 import draw, f8lin, mod  # noqa: F401

pytestmark = pytest.mark.gpu


def test_tangents_are_refused_in_every_mode(mod):
    layer = mod.MXFP4Linear(64, 48, device="cuda", dtype=torch.float32, bias=True)
    x = draw((5, 64), torch.float32, 1).cuda()
    want = layer(x).detach()
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for frozen in (False, True):
            for grad in (True, False):
                with torch.set_grad_enabled(grad):
                    assert torch.equal(layer(x), want)
                    with pytest.raises(NotImplementedError):
                        layer(dual)
            layer.freeze()
        with pytest.raises(NotImplementedError):
            mod.get_grad_norm([dual])
        with pytest.raises(NotImplementedError):
            mod.clip_grads([x, dual], 1.0)


def test_a_backward_through_a_clipped_gradient_is_refused(mod):
    """A double backward needs the gradient as it was; a clip in place may not go by unseen."""
    w = nn.Parameter(draw((30,), torch.float32, 2).cuda())
    w.grad, = torch.autograd.grad((w ** 3).sum(), w, create_graph=True)
    again = (w.grad ** 2).sum()  # saves w.grad
    mod.clip_grad_norm_([w], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        again.backward()
    g = draw((30,), torch.float32, 3).cuda().requires_grad_()
    out = (g ** 2).sum()
    mod.get_grad_norm([g]), mod.clip_grads([g], 0.1)  # only read
    out.backward()
    assert torch.equal(g.grad, 2 * g.detach())


def test_a_shared_linear_trains_and_serves_as_one(mod, f8lin):
    class Twice(nn.Module):
        def __init__(self, lin):
            super().__init__()
            self.a, self.b = nn.Sequential(lin), nn.Sequential(lin)

        def forward(self, x):
            return self.b(torch.relu(self.a(x)))

    torch.manual_seed(0)
    model = mod.convert_to_mxfp4_training(Twice(nn.Linear(64, 64)).cuda())
    x = draw((7, 64), torch.float32, 4).cuda()
    layer = model.a[0]
    assert model.b[0] is layer
    with torch.no_grad():
        want = mod.mxfp4_linear(torch.relu(mod.mxfp4_linear(x, layer.weight, layer.bias)), layer.weight, layer.bias)
    y = model(x)
    assert torch.equal(y, want)
    y.sum().backward()
    assert layer.weight.grad.any() and len(list(model.parameters())) == 2
    mod.freeze_mxfp4(model)
    assert model.b[0].frozen and [p.shape for p in model.parameters()] == [(64,)]
    q = f8lin.MXFP4Tensor(layer.weight_codes, layer.weight_scales, 64, 64)
    with torch.no_grad():
        want = mod.mxfp4_linear(torch.relu(mod.mxfp4_linear(x, q, layer.bias)), q, layer.bias)
        assert torch.equal(model(x), want)
