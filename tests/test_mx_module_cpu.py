"""The MXFP4 and clipping module surface without a GPU: the library's calls are replaced by stubs that fill their
outputs, and tensors say that they are on a GPU."""
import pytest
import torch
import torch.nn as nn
from torch.autograd import forward_ad

from float8linear_tensorwise_amax_amd import f8lin
from float8linear_tensorwise_amax_amd import module as m


@pytest.fixture
def stubbed(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(f8lin, "mxfp4_forward", lambda x, w, y, *a, **k: y.fill_(3.0))


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("packed, dual", [(True, "x"), (True, "bias"), (False, "x"), (False, "weight"), (False, "bias")])
def test_a_forward_mode_tangent_is_refused(stubbed, packed, grad, dual):
    """A linear that takes no part in autograd would drop a tangent, which reads as a derivative of zero."""
    ts = {"x": torch.ones(2, 3, 64), "weight": torch.ones(5, 64), "bias": torch.ones(5)}
    packed_w = f8lin.new_mxfp4(5, 64, "cpu")
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        plain = packed_w if packed else ts["weight"]
        assert m.mxfp4_linear(ts["x"], plain, ts["bias"]).shape == (2, 3, 5)  # no tangent: as ever
        ts[dual] = forward_ad.make_dual(ts[dual], torch.ones_like(ts[dual]))
        with pytest.raises(NotImplementedError):
            m.mxfp4_linear(ts["x"], packed_w if packed else ts["weight"], ts["bias"])
    with torch.inference_mode():  # no derivative of any kind there
        assert m.mxfp4_linear(torch.ones(2, 64), packed_w if packed else torch.ones(5, 64)).shape == (2, 5)


def test_a_tangent_of_a_gradient_is_refused(monkeypatch):
    """The norm and the clipped gradients would come back without it; in place it would stay unscaled."""
    monkeypatch.setattr(f8lin, "grad_norm", lambda grads, out, *a, **k: out.fill_(1.0))
    monkeypatch.setattr(f8lin, "grad_clip", lambda grads, max_norm, norm, *a, **k: norm.fill_(1.0))
    plain, p = torch.ones(4), nn.Parameter(torch.ones(4))
    with forward_ad.dual_level():
        p.grad = plain.clone()
        assert m.get_grad_norm([plain]) == 1 and m.clip_grads([plain], 1.0)[0] == 1 and m.clip_grad_norm_([p], 1.0) == 1
        dual = forward_ad.make_dual(torch.ones(4), torch.ones(4))
        p.grad = dual
        for call in (lambda: m.get_grad_norm([plain, dual]), lambda: m.clip_grads([plain, dual], 1.0),
                     lambda: m.clip_grad_norm_([p], 1.0)):
            with pytest.raises(NotImplementedError):
                call()


def test_written_gradients_count_as_changed(monkeypatch):
    """The library writes through pointers: the version counters, by which autograd finds a saved tensor that was
    changed, are moved for every tensor that a call writes and for none that it reads."""
    monkeypatch.setattr(f8lin, "_ptr", lambda t, dtype=None: 0 if t is None else t.data_ptr())
    monkeypatch.setattr(f8lin, "_call", lambda *a: None)
    grads, outs = [torch.ones(4), torch.ones(3, 2).t()], [torch.ones(4), torch.ones(3, 2).t()]
    norm, ws = torch.zeros(1), torch.zeros(f8lin.grad_workspace_bytes(), dtype=torch.uint8)

    def moved(*args, call=f8lin.grad_clip, **kw):
        ts = (*grads, *outs, norm)
        before = [t._version for t in ts]
        call(*args, **kw)
        return [t._version > b for t, b in zip(ts, before)]

    assert moved(grads, 1.0, norm, ws) == [True, True, False, False, True]
    assert moved(grads, 1.0, norm, ws, outs=outs) == [False, False, True, True, True]
    assert moved(grads, 1.0, norm, None, outs=outs, norm_given=True) == [False, False, True, True, False]
    assert moved(grads, norm, ws, call=f8lin.grad_norm) == [False] * 4 + [True]
    p = nn.Parameter(torch.ones(4))
    p.grad = torch.ones(4)
    saved = (p.grad.requires_grad_() * torch.ones(4, requires_grad=True)).sum()  # keeps p.grad for its backward
    m.clip_grad_norm_([p], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.backward()
    with torch.inference_mode():  # (tensors that count no versions)
        f8lin.grad_clip([torch.ones(4)], 1.0, torch.zeros(1), ws)


class Holder(nn.Module):
    def __init__(self, **children):
        super().__init__()
        for name, child in children.items():
            self.add_module(name, child)


def test_a_shared_linear_is_converted_everywhere():
    """One linear under several parents, twice under one, and inside a shared parent: one layer in all the places."""
    lin, other = nn.Linear(8, 8), nn.Linear(8, 4)
    inner = Holder(c=other)
    model = Holder(a=Holder(l=lin), b=Holder(l=lin, again=lin), s=inner, t=inner)
    m.convert_to_mxfp4_training(model, "ceil")
    layers = [model.a.l, model.b.l, model.b.again]
    assert all(isinstance(l, m.MXFP4Linear) and l is layers[0] and l.rule == "ceil" for l in layers)
    assert layers[0].weight is lin.weight and isinstance(model.t.c, m.MXFP4Linear) and model.t.c is model.s.c
    assert not any(type(l) is nn.Linear for l in model.modules())
    assert len(list(model.parameters())) == 4

    # each place is asked for by name, a shared parent's places under its first name
    seen = []
    lin = nn.Linear(8, 8)
    inner = Holder(c=lin)
    model = Holder(a=Holder(l=lin), s=inner, t=inner)
    m.convert_to_mxfp4_training(model, module_filter_fn=lambda fqn, child: seen.append(fqn) or fqn != "a.l")
    assert seen == ["a.l", "s.c"] and model.a.l is lin and isinstance(model.t.c, m.MXFP4Linear)


def test_tensors_in_a_given_buffer():
    """They lie inside it, or it is refused: their addresses go to the kernels as they are."""
    shapes = ((3, 100), (100, 3))
    buffer, made = f8lin.new_mxfp4s(shapes, "cpu")
    again, same = f8lin.new_mxfp4s(shapes, "cpu", buffer)
    assert again is buffer and [t._c for t in same] == [t._c for t in made]
    assert [t.codes.shape for t in same] == [(3, 64), (100, 16)] and same[1].scales.data_ptr() + 1600 == \
        buffer.data_ptr() + buffer.numel()
    larger = torch.empty(buffer.numel() + 64, dtype=torch.uint8)
    assert len(f8lin.new_mxfp4s(shapes, "cpu", larger)[1]) == 2
    for bad in (buffer[:-1], larger[8:8 + buffer.numel()], larger.view(-1, 16), larger[::2].expand(buffer.numel() // 2 + 32),
                torch.empty(2 * buffer.numel(), dtype=torch.uint8)[::2], buffer.view(torch.int8), buffer[:0]):
        with pytest.raises(ValueError):
            f8lin.new_mxfp4s(shapes, "cpu", bad)
    assert f8lin.new_mxfp4s(((0, 5), (5, 0)), "cpu", buffer[:0])[1][1].codes.shape == (5, 0)
