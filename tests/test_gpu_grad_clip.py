"""Gradient norm and clipping against numpy in binary64.

The norm is summed in binary64 (n additions, each off by 2^-53 of a sum of positive terms) and rounded once to fp32:
|error| <= norm * (2^-24 + n * 2^-53).  The factor max_norm / (norm + 1e-6) takes two more fp32 roundings and the
product one: a result is off by at most 5 fp32 half steps (2^-24 each), plus half a step of its own type.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LISTS = {"one": [1], "odd": [7, 1, 4096, 33, 0, 16385], "single_large": [3_000_001], "many": list(range(1, 230)),
         "pieces": [16384, 16383, 16385, 32768, 5], "empty_tensors": [0, 0, 3]}


@pytest.fixture(scope="module")
def f8lin():
    from float8linear_tensorwise_amax_amd import f8lin
    return f8lin


@pytest.fixture(scope="module")
def mod():
    from float8linear_tensorwise_amax_amd import module
    return module


@pytest.fixture(scope="module")
def mx():
    from oracle import mxfp4
    return mxfp4


def draw(sizes, dtype, seed, std=0.02):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * std).to(dtype) for n in sizes]


def np64(t):
    return t.detach().cpu().double().numpy()


def near(got, want, n):
    return abs(got - want) <= want * (2.0 ** -24 + (n + 2) * 2.0 ** -53) * (1 + 2.0 ** -20)


def check_clipped(outs, grads, norm, max_norm):
    c = min(1.0, max_norm / (norm + 1e-6))
    for o, g in zip(outs, grads):
        want = np64(g) * c
        fi = torch.finfo(o.dtype)
        tol = np.abs(want) * (5 * 2.0 ** -24 * 1.01 + fi.eps / 2 * 1.01) + fi.smallest_normal * fi.eps
        assert o.shape == g.shape and np.all(np.abs(np64(o) - want) <= tol)


@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clip(mod, mx, name, dtype, p):
    grads = draw(LISTS[name], DTYPES[dtype], len(name))
    dev = [g.cuda() for g in grads]
    want = mx.norm([np64(g) for g in grads], p)
    n = sum(LISTS[name])
    norm = mod.get_grad_norm(dev, p)
    assert norm.dtype == torch.float32 and near(float(norm), want, n)
    for share in (0.3, 2.0):
        for out in (None, torch.float32, torch.bfloat16):
            got, outs = mod.clip_grads(dev, share * want, p, out)
            assert torch.equal(got, norm)
            assert all(o.dtype == (out or DTYPES[dtype]) for o in outs)
            check_clipped(outs, grads, want, share * want)
        params = [torch.nn.Parameter(torch.zeros_like(g)) for g in dev]
        for q, g in zip(params, dev):
            q.grad = g.clone()
        params.append(torch.nn.Parameter(torch.zeros(3, device="cuda")))  # without a gradient
        assert torch.equal(mod.clip_grad_norm_(params, share * want, p), norm)
        check_clipped([q.grad for q in params[:-1]], grads, want, share * want)
        if share > 1:
            assert all(torch.equal(q.grad, g) for q, g in zip(params, dev))
    assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))  # clip_grads leaves its inputs


def test_mixed_types_devices_views(f8lin, mod, mx):
    """Types mixed in one list; views that start at odd elements; permuted and strided gradients."""
    base = draw([5000], torch.bfloat16, 1)[0].cuda()
    half = draw([4000], torch.float16, 2)[0].cuda()
    full = draw([6000], torch.float32, 3)[0].cuda()
    grads = [base[1:1000], base[1001:2004], half[3:1234], full[5:3000], half[2000:2001], full[4001:],
             base[2004:4404].view(40, 60).t(), full[3000:3600].view(5, 10, 12).permute(2, 0, 1)]
    want = mx.norm([np64(g) for g in grads], 2.0)
    before = [g.clone() for g in grads]
    norm, outs = mod.clip_grads(grads, 0.1 * want)
    assert near(float(norm), want, 20000)
    check_clipped(outs, before, want, 0.1 * want)
    params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
    strided = torch.zeros((60, 80), device="cuda")
    params.append(torch.nn.Parameter(torch.zeros((60, 40), device="cuda")))
    for p, g in zip(params, grads):
        p.grad = g
    params[-1].grad = strided[:, ::2]
    params[-1].grad.copy_(draw([2400], torch.float32, 9)[0].view(60, 40))
    before.append(params[-1].grad.clone())
    want = mx.norm([np64(g) for g in before], 2.0)
    assert near(float(mod.clip_grad_norm_(params, 0.5 * want)), want, 30000)
    check_clipped([p.grad for p in params], before, want, 0.5 * want)
    assert not strided[:, 1::2].any()


def test_range_of_the_sum(mod):
    """Squares beyond fp32 in both directions, and one large value among many small ones."""
    for v in (1e-30, 1e30, 3e38):
        g = torch.full((1000,), v, device="cuda")
        want = math.sqrt(1000.0) * float(g[0])
        assert near(float(mod.get_grad_norm([g])), want, 1000) or (want > 3.4e38 and math.isinf(float(mod.get_grad_norm([g]))))
    tiny = torch.full((100,), 2.0 ** -149, device="cuda")
    assert float(mod.get_grad_norm([tiny])) == 10 * 2.0 ** -149
    g = torch.full((1 << 22,), 1e-4, device="cuda")
    g[12345] = 1.0
    want = math.sqrt(((1 << 22) - 1) * float(g[0]) ** 2 + 1.0)
    assert near(float(mod.get_grad_norm([g])), want, 1 << 22)


@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_nonfinite(mod, dtype, p):
    for place in (0, 20000, 39999):
        for bad in (math.nan, math.inf, -math.inf):
            grads = [g.cuda() for g in draw([100, 40000, 7], DTYPES[dtype], 1)]
            grads[1][place] = bad
            norm, outs = mod.clip_grads(grads, 1.0, p)
            if math.isnan(bad):
                assert torch.isnan(norm) and all(torch.isnan(o).all() for o in outs)
            else:
                assert float(norm) == math.inf and torch.isnan(outs[1][place])
                outs[1][place] = 0
                assert not any(o.any() for o in outs)
            params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
            for q, g in zip(params, grads):
                q.grad = g.clone()
            with pytest.raises(RuntimeError):
                mod.clip_grad_norm_(params, 1.0, p, error_if_nonfinite=True)
            assert all(torch.equal(q.grad.view(torch.uint8), g.view(torch.uint8)) for q, g in zip(params, grads))


def test_zero_norm_zero_max_and_no_gradients(mod):
    zeros = [torch.zeros(10, device="cuda"), torch.zeros(0, device="cuda")]
    norm, outs = mod.clip_grads(zeros, 1.0)
    assert float(norm) == 0.0 and not outs[0].any()
    grads = [g.cuda() for g in draw([100], torch.float32, 1)]
    assert not mod.clip_grads(grads, 0.0)[1][0].any()
    assert float(mod.clip_grad_norm_([torch.nn.Parameter(torch.zeros(3, device="cuda"))], 1.0)) == 0.0
    assert mod.clip_grads([], 1.0)[1] == []
    q = torch.nn.Parameter(torch.zeros(100, device="cuda"))
    q.grad = grads[0].clone()
    mod.clip_grad_norm_(q, 1e-3)
    assert float(q.grad.norm()) <= 1.001e-3


def test_given_norm(f8lin, mod):
    """The two halves apart: a norm taken over several ranks' shards, then the scaling with it."""
    shards = [[g.cuda() for g in draw([1000, 77], torch.bfloat16, s)] for s in (1, 2)]
    norms = [mod.get_grad_norm(s) for s in shards]
    total = torch.stack(norms).double().square().sum().sqrt().float().view(1)
    whole, want = mod.clip_grads(shards[0] + shards[1], 0.1)
    assert abs(float(total) - float(whole)) <= 2e-7 * float(whole)
    total.copy_(whole)
    got = [torch.empty_like(g) for g in shards[0] + shards[1]]
    f8lin.grad_clip(shards[0] + shards[1], 0.1, total, None, outs=got, norm_given=True)
    assert torch.equal(total, whole.view(1)) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_bits_every_time(mod):
    grads = [g.cuda() for g in draw([1_000_000, 3, 77777], torch.bfloat16, 1)]
    first = mod.clip_grads(grads, 0.1)
    for _ in range(3):
        again = mod.clip_grads(grads, 0.1)
        assert torch.equal(first[0], again[0]) and all(torch.equal(a, b) for a, b in zip(first[1], again[1]))


def test_refusals(f8lin, mod):
    g = torch.zeros(100, device="cuda")
    norm, ws = torch.zeros(1, device="cuda"), f8lin.new_grad_workspace()
    for p in (3.0, 0.0, -1.0, math.nan):
        with pytest.raises(ValueError):
            f8lin.grad_norm([g], norm, ws, p)
    for bad in (-1.0, math.nan):
        with pytest.raises(f8lin.F8linError):
            f8lin.grad_clip([g], bad, norm, ws)
    with pytest.raises(f8lin.F8linError):
        f8lin.grad_clip([g, g], 1.0, norm, ws)          # scaled twice
    with pytest.raises(f8lin.F8linError):
        f8lin.grad_clip([g[:60], g[50:]], 1.0, norm, ws)
    with pytest.raises(f8lin.F8linError):
        f8lin.grad_clip([g[:50]], 1.0, norm, ws, outs=[g[20:70]])
    with pytest.raises(f8lin.F8linError):
        f8lin.grad_norm([g], g[3:4], ws)                # the norm inside a gradient
    with pytest.raises(f8lin.F8linError):
        f8lin.grad_norm([g], norm, ws[:100])
    f8lin.grad_norm([g, g], norm, ws)                   # reading twice is fine
    with pytest.raises(TypeError):
        f8lin.grad_norm([g.double()], norm, ws)
    with pytest.raises(ValueError):
        f8lin.grad_norm([g.cpu()], norm, ws)
    with pytest.raises(ValueError):
        f8lin.grad_norm([g[::2]], norm, ws)
    with pytest.raises(ValueError):
        f8lin.grad_clip([g], 1.0, norm, ws, outs=[g, g])
    with pytest.raises(ValueError):
        mod.clip_grads([torch.zeros(4), g], 1.0)


def test_expanded_gradient_is_refused_in_place(mod):
    """Nothing is scaled when one of the gradients shares its elements; out of place it counts each of them."""
    a = torch.nn.Parameter(torch.zeros(4, device="cuda"))
    b = torch.nn.Parameter(torch.zeros(3, 5, device="cuda"))
    a.grad, b.grad = torch.full((4,), 2.0, device="cuda"), torch.full((1, 5), 3.0, device="cuda").expand(3, 5)
    with pytest.raises(ValueError):
        mod.clip_grad_norm_([a, b], 1.0)
    assert torch.equal(a.grad, torch.full((4,), 2.0, device="cuda"))
    norm, out = mod.clip_grads([a.grad, b.grad], 1.0, norm_type=1.0)
    assert norm.item() == 4 * 2.0 + 15 * 3.0 and out[1].shape == (3, 5)


@pytest.mark.parametrize("sizes, dtype, out", [([100_000_003, 70_000_001, 5], torch.bfloat16, None),
                                               ([60_000_001, 7], torch.float16, torch.float32),
                                               ([90_000_001], torch.float32, torch.float32)])
def test_more_than_the_caches_hold(f8lin, mod, sizes, dtype, out):
    """Big lists, in place (out None) and out of it: the norm against binary64, the clipped gradients bit for bit."""
    gen = torch.Generator("cuda").manual_seed(len(sizes))
    grads = [torch.empty(n, dtype=dtype, device="cuda").normal_(0, 0.02, generator=gen) for n in sizes]
    before = [g.clone() for g in grads]
    ref = sum(sum((c.double() ** 2).sum().item() for c in g.split(1 << 24)) for g in grads) ** 0.5
    norm = torch.empty((), device="cuda")
    f8lin.grad_norm(grads, norm, f8lin.new_grad_workspace())
    assert abs(norm.item() - ref) <= ref * 2.0 ** -24 * 1.01
    assert abs(mod.get_grad_norm(grads, math.inf).item() - max(g.abs().max().item() for g in grads)) == 0
    outs = grads if out is None else [torch.empty_like(g, dtype=out) for g in grads]
    got = torch.empty((), device="cuda")
    f8lin.grad_clip(grads, 0.5, got, f8lin.new_grad_workspace(), 2.0, outs=None if out is None else outs)
    assert torch.equal(got, norm)
    c = torch.tensor(0.5, device="cuda") / (norm + 1e-6)
    for g, b, o in zip(grads, before, outs):
        assert torch.equal(o, (b.float() * c).to(o.dtype))
        assert out is None or torch.equal(g, b)
