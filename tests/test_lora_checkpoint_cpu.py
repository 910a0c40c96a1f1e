"""Adapters under activation checkpointing, with the kernels replaced by their formulas on the CPU: a forward that runs
again inside a backward uses the batch that the first one had, or is refused."""
import pytest
import torch
import torch.nn as nn
from torch.utils.checkpoint import checkpoint

from float8linear_tensorwise_amax_amd import f8lin
from float8linear_tensorwise_amax_amd import module as m

T, D, L, R = 12, 8, 3, 2


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    """lora_plan keeps the index itself in the plan's buffer; the products are torch's."""
    def lora_plan(index, plan, stream=None):
        plan.buffer[:plan.tokens] = index.to(torch.int32)
        plan.written()

    def parts(plan, scales):
        for i in range(plan.adapters):
            rows = torch.nonzero(plan.buffer[:plan.tokens] == i).flatten()
            yield i, rows, 1.0 if scales is None else scales[i]

    def lora_forward(base, x, a, b, scales, plan, y, h=None, ws=None, stream=None):
        y.copy_(base)
        for i, rows, s in parts(plan, scales):
            y[rows] += s * (x[rows] @ a[i].t()) @ b[i].t()

    def lora_backward(dy, x, a, b, scales, plan, h, dx=None, da=None, db=None, ws=None, stream=None):
        for t in (dx, da, db):
            if t is not None:
                t.zero_()
        for i, rows, s in parts(plan, scales):
            g = s * dy[rows] @ b[i]
            if dx is not None:
                dx[rows] = g @ a[i]
            if da is not None:
                da[i] = g.t() @ x[rows]
            if db is not None:
                db[i] = dy[rows].t() @ (s * x[rows] @ a[i].t())

    for f in (lora_plan, lora_forward, lora_backward):
        monkeypatch.setattr(f8lin, f.__name__, f)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))


class Block(nn.Module):
    def __init__(self):
        super().__init__()
        self.fc1, self.fc2 = nn.Linear(D, D), nn.Linear(D, D)

    def forward(self, x, *batch):
        return x + self.fc2(torch.relu(self.fc1(x, *batch)), *batch)


def model_and_batches():
    torch.manual_seed(0)
    model = m.convert_to_lora(Block(), L, R)
    for layer in model.modules():
        if isinstance(layer, m.LoraLinear):
            nn.init.normal_(layer.lora_b)
    index = [torch.zeros(T, dtype=torch.int64), torch.arange(T) % 2 + 1]
    return model, [m.LoraBatch(i, L) for i in index], [torch.randn(T, D) for _ in range(2)]


def grads_of(model):
    out = [p.grad.clone() for p in model.parameters() if p.requires_grad]
    model.zero_grad()
    return out


def same(p, q):
    return all(torch.allclose(a, b, rtol=1e-5, atol=1e-6) for a, b in zip(p, q))


def wanted(model, batches, xs):
    m.set_lora_batch(model, None)
    for x, batch in zip(xs, batches):
        model(x, batch).square().sum().backward()
    return grads_of(model)


def run(model, x, reentrant, *batch):
    return checkpoint(model, x.clone().requires_grad_(), *batch, use_reentrant=reentrant).square().sum()


def test_the_batch_in_the_call_is_the_layers(formulas):
    model, batches, xs = model_and_batches()
    m.set_lora_batch(model, batches[0])
    y = model(xs[0])
    assert torch.equal(model(xs[0], batches[0]), y) and not torch.equal(model(xs[0], batches[1]), y)
    plain = model(xs[0], None)  # (None in the call: the base alone, whatever is set)
    m.set_lora_batch(model, None)
    assert torch.equal(model(xs[0]), plain) and not torch.equal(plain, y)


@pytest.mark.parametrize("reentrant", [False, True])
def test_batches_in_the_call(reentrant):
    """Two forwards, then their backwards, in either order."""
    model, batches, xs = model_and_batches()
    want = wanted(model, batches, xs)
    for order in ((0, 1), (1, 0)):
        losses = [run(model, xs[i], reentrant, batches[i]) for i in range(2)]
        for i in order:
            losses[i].backward()
        assert same(grads_of(model), want)


def test_the_batch_that_is_set():
    model, batches, xs = model_and_batches()
    want = wanted(model, batches, xs)
    for i in range(2):  # one after the other
        m.set_lora_batch(model, batches[i])
        run(model, xs[i], False).backward()
    assert same(grads_of(model), want)
    losses = []
    for i in range(2):
        m.set_lora_batch(model, batches[i])
        losses.append(run(model, xs[i], False))
    with pytest.raises(RuntimeError, match="another batch"):
        losses[0].backward()
    model.zero_grad()
    losses = []
    for i in range(2):
        m.set_lora_batch(model, batches[i])
        losses.append(run(model, xs[i], False))
    for i in range(2):  # set again for its backward
        m.set_lora_batch(model, batches[i])
        losses[i].backward()
    assert same(grads_of(model), want)


@pytest.mark.parametrize("reentrant", [False, True])
def test_set_and_taken_away(reentrant):
    """A batch where the forward had none, none where it had one."""
    for before, after in ((True, False), (False, True)):
        model, batches, xs = model_and_batches()
        m.set_lora_batch(model, batches[0] if before else None)
        loss = run(model, xs[0], reentrant)
        m.set_lora_batch(model, None if before else batches[0])
        with pytest.raises(Exception):
            loss.backward()


def test_one_layer_and_what_follows_it():
    """The last tensor that a segment saves is of the layer's own input's shape."""
    torch.manual_seed(0)
    model = m.convert_to_lora(nn.Sequential(nn.Linear(D, D), nn.ReLU()), L, R)
    batch = m.LoraBatch(torch.zeros(T, dtype=torch.int64), L)
    loss = run(model, torch.randn(T, D), False)
    m.set_lora_batch(model, batch)
    with pytest.raises(Exception):
        loss.backward()


@pytest.mark.parametrize("reentrant", [False, True])
def test_updated_between(reentrant):
    for call in (True, False):
        model, batches, xs = model_and_batches()
        m.set_lora_batch(model, batches[0])
        loss = run(model, xs[0], reentrant, *([batches[0]] if call else []))
        batches[0].update(torch.ones(T, dtype=torch.int64))
        with pytest.raises(RuntimeError):
            loss.backward()
    # (updated before its forward: as good as new)
    model, batches, xs = model_and_batches()
    want = wanted(model, batches[1:], xs[1:])
    batches[0].update(torch.arange(T) % 2 + 1)
    loss = run(model, xs[1], False, batches[0])
    loss.backward()
    assert same(grads_of(model), want)


def test_reentrant_with_a_batch_that_is_set_is_refused():
    model, batches, xs = model_and_batches()
    m.set_lora_batch(model, batches[0])
    loss = run(model, xs[0], True)
    with pytest.raises(RuntimeError, match="in the call"):
        loss.backward()


@pytest.mark.parametrize("reentrant", [False, True])
def test_frozen_adapters(reentrant):
    """Nothing of the layer takes part in the graph, but what follows it does: no node is there to compare, so the call
    inside the backward is refused unless it brings its batch."""
    model, batches, xs = model_and_batches()
    model.requires_grad_(False)
    head = nn.Linear(D, D)
    m.set_lora_batch(model, batches[0])
    flag = torch.zeros(1, requires_grad=True)

    def segment(x, flag, *batch):
        return head(model(x, *batch)) + flag

    loss = checkpoint(segment, xs[0], flag, use_reentrant=reentrant).square().sum()
    with pytest.raises(RuntimeError, match="in the call"):
        loss.backward()
    head.zero_grad()
    m.set_lora_batch(model, batches[1])
    checkpoint(segment, xs[0], flag, batches[0], use_reentrant=reentrant).square().sum().backward()
    got = head.weight.grad.clone()
    head.zero_grad()
    (head(model(xs[0], batches[0])) + flag).square().sum().backward()
    assert torch.allclose(got, head.weight.grad, rtol=1e-5, atol=1e-6)


def test_layers_that_never_had_a_batch():
    for reentrant in (False, True):
        model, _, xs = model_and_batches()
        x = xs[0].clone().requires_grad_()
        checkpoint(model, x, use_reentrant=reentrant).square().sum().backward()
        want = xs[0].clone().requires_grad_()
        model(want).square().sum().backward()
        assert torch.allclose(x.grad, want.grad)


def test_saved_tensors_on_the_cpu():
    """Hooks that hand back copies of what was saved."""
    model, batches, xs = model_and_batches()
    want = wanted(model, batches, xs)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        for x, batch in zip(xs, batches):
            model(x, batch).square().sum().backward()
    assert same(grads_of(model), want)


def test_calls_without_a_graph_inside_a_backward():
    model, batches, xs = model_and_batches()
    batches[0].update(torch.zeros(T, dtype=torch.int64))
    m.set_lora_batch(model, batches[0])
    with torch.no_grad():
        want = model(xs[0])
    seen = []

    def hook(g):
        with torch.no_grad():
            seen.append(model(xs[0]))

    leaf = torch.ones(3, requires_grad=True)
    y = leaf * 2
    y.register_hook(hook)
    y.sum().backward()
    assert torch.equal(seen[0], want)
