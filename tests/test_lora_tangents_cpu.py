"""Forward-mode tangents of the adapters' arguments are refused in every grad mode, each argument's."""
import pytest
import torch
from torch.autograd import forward_ad

from float8linear_tensorwise_amax_amd import f8lin
from float8linear_tensorwise_amax_amd import module as m

SHAPES = dict(base=(5, 6), x=(5, 4), a=(3, 2, 4), b=(3, 6, 2), scales=(3,))


@pytest.mark.parametrize("which", list(SHAPES))
@pytest.mark.parametrize("mode", [torch.no_grad, torch.enable_grad, "graph"])
def test_tangents(monkeypatch, which, mode):
    for name in ("lora_plan", "lora_forward"):
        monkeypatch.setattr(f8lin, name, lambda *args, **kw: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    batch = m.LoraBatch(torch.zeros(5, dtype=torch.int64), 3)
    t = {k: torch.randn(s) for k, s in SHAPES.items()}
    if mode == "graph":
        t["x"].requires_grad_()
    with (torch.enable_grad if mode == "graph" else mode)(), forward_ad.dual_level():
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        with pytest.raises(NotImplementedError):
            m.lora_add(t["base"], t["x"], t["a"], t["b"], batch, t["scales"])
