"""Host-side validation of the layer norm's and the low-rank adapters' entry points (every call here is refused, or has
nothing to launch), the modules and their swaps, and the plain oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch
import torch.nn as nn

from float8linear_tensorwise_amax_amd import f8lin
from float8linear_tensorwise_amax_amd import module as m
from oracle import block

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 4
MB = 1 << 20
A = 0x100000000  # fake, never-dereferenced addresses
BF16, FP16, FP32 = 0, 1, 2
lib = f8lin._lib


def at(i):
    """Addresses 64 MiB apart."""
    return A + 64 * MB * i


def call(fn, cls, good, **kw):
    fields = dict(good)
    fields.update(kw)
    return fn(ctypes.byref(cls(**fields)), None)


# -------------------------------------------------------------- layer norm

NORM = dict(rows=40, cols=100, x=at(1), ldx=0, weight=at(2), bias=at(3), y=at(4), stats=at(5), y_amax=at(7),
            x_dtype=BF16, weight_dtype=FP32, bias_dtype=FP16, y_dtype=BF16, eps=1e-5)


def test_layer_norm_forward_rejections():
    def f(**kw):
        return call(lib.f8lin_layer_norm_forward, f8lin.LayerNormFwdArgs, NORM, **kw)

    assert lib.f8lin_layer_norm_forward(None, None) == EINVAL
    for name in ("x_dtype", "y_dtype", "weight_dtype", "bias_dtype"):
        assert f(**{name: 3}) == EINVAL and f(**{name: -1}) == EINVAL
    assert f(y_dtype=FP32) == EINVAL and f(y_dtype=FP16) == EINVAL and f(x_dtype=FP16) == EINVAL
    assert f(rows=-1) == ESHAPE and f(cols=(1 << 22) + 1) == ESHAPE and f(rows=1 << 21, cols=1 << 21) == ESHAPE
    assert f(ldx=99) == ESHAPE and f(ldx=-5) == ESHAPE and f(ldx=1 << 41) == ESHAPE
    assert f(rows=1 << 22, ldx=1 << 40) == ESHAPE
    assert f(x=None) == EINVAL and f(y=None) == EINVAL
    assert f(x=at(1) + 1) == EALIGN and f(y=at(4) + 1) == EALIGN and f(weight=at(2) + 2) == EALIGN
    assert f(bias=at(3) + 1) == EALIGN and f(stats=at(5) + 2) == EALIGN
    assert f(y_amax=at(7) + 2) == EALIGN
    assert f(eps=-1e-9) == EINVAL and f(eps=math.nan) == EINVAL
    # anything written that meets anything else
    assert f(y=at(1)) == EINVAL and f(y=at(1) + 7998) == EINVAL and f(weight=at(4) + 7996) == EINVAL
    assert f(stats=at(4)) == EINVAL and f(y_amax=at(5) + 316) == EINVAL and f(y_amax=at(3)) == EINVAL
    assert f(ldx=1 << 22) == EINVAL  # x's stride reaches y
    assert f(rows=0, x=None, y=None, stats=None, y_amax=None) == OK


BACK = dict(rows=40, cols=100, dy=at(1), x=at(2), lddy=0, ldx=0, weight=at(3), stats=at(4), dx=at(6),
            dweight=at(7), dbias=at(8), dy_dtype=BF16, x_dtype=BF16, weight_dtype=FP32, dweight_dtype=FP32,
            dbias_dtype=FP16, ws=at(9), ws_bytes=32 * MB)


def test_layer_norm_backward_rejections():
    def f(**kw):
        return call(lib.f8lin_layer_norm_backward, f8lin.LayerNormBwdArgs, BACK, **kw)

    assert lib.f8lin_layer_norm_backward(None, None) == EINVAL
    for name in ("x_dtype", "dy_dtype", "weight_dtype", "dweight_dtype", "dbias_dtype"):
        assert f(**{name: 3}) == EINVAL
    assert f(dy_dtype=FP32) == EINVAL and f(x_dtype=FP16) == EINVAL
    assert f(rows=-1) == ESHAPE and f(cols=1 << 23) == ESHAPE and f(lddy=99) == ESHAPE and f(ldx=50) == ESHAPE
    for name in ("dy", "x", "stats"):
        assert f(**{name: None}) == EINVAL, name
    for name in ("dy", "x", "dx", "dbias"):
        assert f(**{name: BACK[name] + 1}) == EALIGN, name
    assert f(weight=at(3) + 2) == EALIGN and f(dweight=at(7) + 2) == EALIGN and f(stats=at(4) + 2) == EALIGN
    need = lib.f8lin_layer_norm_workspace_bytes(40, 100)
    assert need > 0 and need % 4 == 0
    assert f(ws=None) == EWORKSPACE and f(ws_bytes=need - 1) == EWORKSPACE and f(ws=at(9) + 8) == EALIGN
    assert f(dx=at(1)) == EINVAL and f(dx=at(2)) == EINVAL and f(dweight=at(8)) == EINVAL and f(ws=at(6)) == EINVAL
    assert f(dbias=at(4) + 300) == EINVAL
    assert f(dx=None, dweight=None, dbias=None, ws=None) == OK  # nothing asked for
    assert f(cols=0, dy=None, x=None, weight=None, stats=None, dx=None, dweight=at(7), ws=None) == OK
    assert lib.f8lin_layer_norm_workspace_bytes(0, 100) == 0 and lib.f8lin_layer_norm_workspace_bytes(-1, 100) == 0


# ------------------------------------------------------- low-rank adapters

def test_plan_rejections():
    f = lib.f8lin_lora_plan
    need = lib.f8lin_lora_plan_bytes(1000, 20)
    assert need >= 4 * (2 * 1000 + 22)
    assert f(at(1), 4, 1000, 20, None, need, None) == EWORKSPACE and f(at(1), 4, 1000, 20, at(2), need - 1, None) == EWORKSPACE
    assert f(at(1), 2, 1000, 20, at(2), need, None) == EINVAL and f(None, 4, 1000, 20, at(2), need, None) == EINVAL
    assert f(at(1), 4, -1, 20, at(2), need, None) == ESHAPE and f(at(1), 4, (1 << 22) + 1, 20, at(2), 1 << 40, None) == ESHAPE
    for n in (0, -1, 2048):
        assert f(at(1), 4, 10, n, at(2), need, None) == ESHAPE and lib.f8lin_lora_plan_bytes(10, n) == 0
    assert lib.f8lin_lora_plan_bytes(-1, 3) == 0 and lib.f8lin_lora_plan_bytes((1 << 22) + 1, 3) == 0
    assert f(at(1) + 4, 8, 1000, 20, at(2), need, None) == EALIGN and f(at(1) + 2, 4, 1000, 20, at(2), need, None) == EALIGN
    assert f(at(1), 4, 1000, 20, at(2) + 8, need, None) == EALIGN
    assert f(at(2) + 64, 4, 1000, 20, at(2), need, None) == EINVAL


FWD = dict(tokens=300, K=100, N=70, x=at(1), a=at(2), b=at(3), base=at(4), ldx=0, ldbase=0, y=at(5), scales=at(6),
           plan=at(7), h=at(8), ws=at(9), ws_bytes=32 * MB, rank=20, adapters=5, dtype=BF16)


def test_lora_forward_rejections():
    def f(**kw):
        return call(lib.f8lin_lora_forward, f8lin.LoraFwdArgs, FWD, **kw)

    assert lib.f8lin_lora_forward(None, None) == EINVAL
    assert f(dtype=3) == EINVAL and f(dtype=-1) == EINVAL
    assert f(tokens=-1) == ESHAPE and f(K=1 << 23) == ESHAPE and f(N=-2) == ESHAPE and f(tokens=1 << 21, K=1 << 21) == ESHAPE
    assert f(rank=0) == ESHAPE and f(rank=257) == ESHAPE and f(adapters=0) == ESHAPE and f(adapters=2048) == ESHAPE
    assert f(adapters=2047, rank=256, K=1 << 22) == ESHAPE  # more than 2^40 elements
    assert f(ldx=99) == ESHAPE and f(ldbase=69) == ESHAPE
    for name in ("x", "a", "b", "y", "plan"):
        assert f(**{name: None}) == EINVAL, name
    for name in ("x", "a", "b", "y", "base"):
        assert f(**{name: FWD[name] + 1}) == EALIGN, name
    assert f(scales=at(6) + 2) == EALIGN and f(plan=at(7) + 8) == EALIGN and f(h=at(8) + 4) == EALIGN
    need = lib.f8lin_lora_forward_workspace_bytes(300, 100, 70, 20, 5)
    assert need >= 300 * 32 * 4
    # (one part: with h given nothing else is kept)
    assert f(h=None, ws=None) == EWORKSPACE and f(h=None, ws_bytes=need - 1) == EWORKSPACE and f(h=None, ws=at(9) + 8) == EALIGN
    assert f(y=at(1)) == EINVAL and f(y=at(2)) == EINVAL and f(y=at(3)) == EINVAL and f(y=at(6)) == EINVAL
    assert f(y=at(4) + 2) == EINVAL and f(y=at(4), ldbase=71) == EINVAL  # base, but not in its place
    assert f(h=at(7)) == EINVAL and f(h=at(5)) == EINVAL and f(h=None, ws=at(4)) == EINVAL
    assert f(tokens=0, x=None, base=None, y=None, h=None, ws=None) == OK
    assert f(N=0, b=None, base=None, y=None) == OK


LBACK = dict(tokens=300, K=100, N=70, dy=at(1), x=at(2), a=at(3), b=at(4), lddy=0, ldx=0, scales=at(5), h=at(6),
             plan=at(7), dx=at(8), da=at(9), db=at(10), ws=at(11), ws_bytes=60 * MB, rank=20, adapters=5, dtype=FP16)


def test_lora_backward_rejections():
    def f(**kw):
        return call(lib.f8lin_lora_backward, f8lin.LoraBwdArgs, LBACK, **kw)

    assert lib.f8lin_lora_backward(None, None) == EINVAL
    assert f(dtype=3) == EINVAL and f(tokens=-1) == ESHAPE and f(rank=300) == ESHAPE and f(adapters=-4) == ESHAPE
    assert f(lddy=69) == ESHAPE and f(ldx=99) == ESHAPE
    for name in ("dy", "x", "a", "b", "h", "plan"):
        assert f(**{name: None}) == EINVAL, name
    for name in ("dy", "x", "a", "b", "dx", "da", "db"):
        assert f(**{name: LBACK[name] + 1}) == EALIGN, name
    assert f(h=at(6) + 8) == EALIGN and f(scales=at(5) + 1) == EALIGN and f(plan=at(7) + 4) == EALIGN
    need = lib.f8lin_lora_backward_workspace_bytes(300, 100, 70, 20, 5)
    assert f(ws=None) == EWORKSPACE and f(ws_bytes=need - 1) == EWORKSPACE and f(ws=at(11) + 8) == EALIGN
    assert f(dx=at(1)) == EINVAL and f(da=at(2)) == EINVAL and f(db=at(9)) == EINVAL and f(ws=at(6)) == EINVAL
    assert f(dx=None, da=None, db=None, ws=None) == OK
    for name in ("f8lin_lora_forward_workspace_bytes", "f8lin_lora_backward_workspace_bytes"):
        g = getattr(lib, name)
        assert g(-1, 8, 8, 4, 2) == 0 and g(8, 8, 8, 0, 2) == 0 and g(8, 8, 8, 4, 2048) == 0
        assert g(1 << 22, 64, 64, 256, 2047) > 0 and g(0, 64, 64, 4, 2) >= 0 and g(64, 0, 0, 4, 2) >= 0


def test_empty_sizes_have_a_workspace():
    for T, K, N in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (0, 0, 0), (1, 1, 1)):
        assert lib.f8lin_lora_forward_workspace_bytes(T, K, N, 1, 1) == 4 * T * 16
        assert lib.f8lin_lora_backward_workspace_bytes(T, K, N, 1, 1) >= 4 * T * 16


# ----------------------------------------------------------------- modules

def test_cpu_tensors_are_refused():
    x = torch.ones(4, 8)
    with pytest.raises(RuntimeError):
        m.layer_norm(x)
    with pytest.raises(RuntimeError):
        m.LoraBatch(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(RuntimeError):
        m.lora_add(x, x, x, x, None)
    with pytest.raises(ValueError):
        f8lin.layer_norm_forward(x, x.clone())
    for tokens, adapters in ((4, 0), (4, 2048), (-1, 3), ((1 << 22) + 1, 3)):
        with pytest.raises(ValueError):
            f8lin.LoraPlan(tokens, adapters, "cpu")


def test_layer_norm_module():
    n = m.LayerNorm((3, 4))
    assert n.weight.shape == (3, 4) and bool((n.weight == 1).all()) and not n.bias.any()
    assert m.LayerNorm(5, weight=False, bias=False).weight is None and m.LayerNorm(5, bias=False).bias is None
    with pytest.raises(ValueError):
        m.LayerNorm(5, weight=torch.ones(4))
    with pytest.raises(ValueError):
        m.LayerNorm(())
    norm = nn.LayerNorm(6, eps=0.5)
    model = nn.ModuleDict({"a": norm, "b": nn.Sequential(norm, nn.LayerNorm(6, elementwise_affine=False)),
                           "c": nn.LayerNorm(7)})
    w = norm.weight
    asked = []
    assert m.convert_layer_norm(model, lambda fqn, mod: asked.append(fqn) or fqn != "c") is model
    assert model["a"] is model["b"][0] and model["a"].weight is w and model["a"].eps == 0.5
    assert type(model["b"][1]) is m.LayerNorm and model["b"][1].weight is None and type(model["c"]) is nn.LayerNorm
    assert sorted(asked) == ["a", "b.0", "b.1", "c"]
    with pytest.raises(ValueError):
        m.convert_layer_norm(nn.LayerNorm(4))


def test_lora_module():
    lin = nn.Linear(6, 10)
    model = nn.ModuleDict({"a": lin, "b": nn.Sequential(lin, nn.Linear(6, 4, bias=False))})
    m.convert_to_lora(model, 3, 2, scale=0.5, module_filter_fn=lambda fqn, mod: mod.bias is not None)
    lora = model["a"]
    assert model["b"][0] is lora and lora.base is lin and type(model["b"][1]) is nn.Linear
    assert lora.lora_a.shape == (3, 2, 6) and lora.lora_b.shape == (3, 10, 2) and not lora.lora_b.any()
    assert lora.lora_scales.tolist() == [0.5] * 3 and "lora_scales" in lora.state_dict()
    assert not lin.weight.requires_grad and not lin.bias.requires_grad and lora.lora_a.requires_grad
    assert model["b"][1].weight.requires_grad
    x = torch.ones(2, 6)
    assert torch.equal(lora(x), lin(x))  # without a batch the base alone
    m.convert_to_lora(model, 3, 2)
    assert model["a"] is lora and lora.base is lin and type(model["b"][1]) is m.LoraLinear
    marker = object()
    m.set_lora_batch(model, marker)
    assert lora.batch is marker and model["b"][1].batch is marker
    with pytest.raises(ValueError):
        m.convert_to_lora(nn.Linear(3, 3), 1, 1)
    for adapters, rank in ((0, 1), (2048, 1), (1, 0), (1, 257)):
        with pytest.raises(ValueError):
            m.LoraLinear(lin, adapters, rank)


# ------------------------------------------------------------- the oracle

def test_oracle_layer_norm():
    x = np.array([[1.0, 3.0], [5.0, 5.0]])
    y, mean, rstd, xhat = block.layer_norm(x, np.array([2.0, 4.0]), np.array([10.0, 20.0]), 0.25)
    r = 1 / math.sqrt(1.25)
    assert np.allclose(mean[:, 0], [2, 5]) and np.allclose(rstd[:, 0], [r, 2])
    assert np.allclose(y, [[10 - 2 * r, 20 + 4 * r], [10, 20]])
    rng = np.random.default_rng(0)
    t = [torch.tensor(rng.standard_normal(s), requires_grad=True) for s in ((5, 9), (9,), (9,))]
    out = torch.nn.functional.layer_norm(t[0], (9,), t[1], t[2], 1e-3)
    dy = rng.standard_normal((5, 9))
    want = torch.autograd.grad(out, t, torch.from_numpy(dy))
    n = [q.detach().numpy() for q in t]
    y, mean, rstd, xhat = block.layer_norm(*n, 1e-3)
    assert np.allclose(y, out.detach())
    for got, ref in zip(block.layer_norm_grads(dy, xhat, rstd, n[1]), want):
        assert np.allclose(got, ref)


def test_oracle_lora():
    rng = np.random.default_rng(1)
    T, K, N, R, L = 12, 5, 7, 2, 3
    base, x, a, b = (torch.tensor(rng.standard_normal(s), requires_grad=True)
                     for s in ((T, N), (T, K), (L, R, K), (L, N, R)))
    index, scales = rng.integers(-1, L, T), np.array([0.5, 2.0, 3.0])
    rows = []
    for t in range(T):
        i = index[t]
        rows.append(base[t] if i < 0 else base[t] + scales[i] * (b[i] @ (a[i] @ x[t])))
    y = torch.stack(rows)
    dy = rng.standard_normal((T, N))
    want = torch.autograd.grad(y, (x, a, b), torch.from_numpy(dy), allow_unused=True)
    n = [q.detach().numpy() for q in (base, x, a, b)]
    got, h = block.lora(*n, index, scales)
    assert np.allclose(got, y.detach())
    dx, da, db, g = block.lora_grads(dy, *n[1:], index, scales, h)
    for p, q in zip((dx, da, db), want):
        assert np.allclose(p, q)
