"""Adapters under activation checkpointing on the GPU: two micro-batches in flight at once."""
import pytest
import torch
import torch.nn as nn
from torch.utils.checkpoint import checkpoint

from block_helpers import draw

pytestmark = pytest.mark.gpu


class Block(nn.Module):
    def __init__(self, d):
        super().__init__()
        self.norm, self.fc1, self.fc2 = nn.LayerNorm(d), nn.Linear(d, 2 * d), nn.Linear(2 * d, d)

    def forward(self, x, *batch):
        return x + self.fc2(torch.relu(self.fc1(self.norm(x), *batch)), *batch)


@pytest.mark.parametrize("tokens", [60, 1100])
@pytest.mark.parametrize("kind", ["plain", "mxfp4"])
def test_micro_batches(kind, tokens):
    from float8linear_tensorwise_amax_amd import module as mod
    torch.manual_seed(0)
    d, L, R = 64, 3, 8
    model = Block(d).cuda().bfloat16()
    if kind == "mxfp4":
        mod.convert_to_mxfp4_training(model)
    mod.convert_to_lora(mod.convert_layer_norm(model), L, R)
    for layer in (model.fc1, model.fc2):
        nn.init.normal_(layer.lora_b, std=0.2)
    xs = [draw((tokens, d), torch.bfloat16, i).cuda().requires_grad_() for i in range(2)]
    batches = [mod.LoraBatch(torch.zeros(tokens, dtype=torch.int64, device="cuda"), L),
               mod.LoraBatch(torch.arange(tokens, device="cuda") % 2 + 1, L)]
    params = [p for p in model.parameters() if p.requires_grad]

    def grads():
        out = [t.grad.clone() for t in (*params, *xs)]
        for t in (*params, *xs):
            t.grad = None
        return out

    for x, batch in zip(xs, batches):
        model(x, batch).float().square().sum().backward()
    want = grads()
    run = lambda i, reentrant, *batch: checkpoint(model, xs[i], *batch, use_reentrant=reentrant).float().square().sum()  # noqa: E731
    for reentrant in (False, True):
        losses = [run(i, reentrant, batches[i]) for i in range(2)]
        for loss in losses:
            loss.backward()
        assert all(torch.equal(p, q) for p, q in zip(grads(), want))
    losses = []
    for i in range(2):
        mod.set_lora_batch(model, batches[i])
        losses.append(run(i, False))
    with pytest.raises(RuntimeError, match="another batch"):
        losses[0].backward()
    grads_left = [t for t in (*params, *xs) if t.grad is not None]
    for t in grads_left:
        t.grad = None
    # the saved tensors of a plain graph kept in host memory
    with torch.autograd.graph.save_on_cpu():
        for x, batch in zip(xs, batches):
            model(x, batch).float().square().sum().backward()
    assert all(torch.equal(p, q) for p, q in zip(grads(), want))
