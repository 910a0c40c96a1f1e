"""Layer norm on the GPU: forward, backward and the parameters' gradients against binary64 within counted roundings,
strides, the output's amax, rows that are not finite, graphs, streams, the module and its swap."""
import numpy as np
import pytest
import torch
import torch.nn as nn

from block_helpers import DTYPES, close, draw, norm_bounds, norm_grad_bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def f8lin():
    from float8linear_tensorwise_amax_amd import f8lin
    return f8lin


@pytest.fixture(scope="module")
def mod():
    from float8linear_tensorwise_amax_amd import module
    return module


def check(mod, x, w, b, dy, eps=1e-5, out=None):
    """Forward and backward of the tensors (CPU) against binary64."""
    rows, cols = x.shape
    leaves = [None if t is None else t.cuda().requires_grad_() for t in (x, w, b)]
    y = mod.layer_norm(*leaves, eps, out)
    assert y.shape == x.shape and y.dtype == (out or x.dtype)
    n = norm_bounds(np64(x), None if w is None else np64(w), None if b is None else np64(b), eps, rows, cols)
    close(y, n["y"], n["d_y"], "y")
    given = [t for t in leaves if t is not None]
    grads = dict(zip([i for i, t in enumerate(leaves) if t is not None], torch.autograd.grad(y, given, dy.cuda())))
    refs, errs = norm_grad_bounds(n, np64(dy), None if w is None else np64(w), rows, cols)
    for i, what in enumerate(("dx", "dw", "db")):
        if i in grads:
            assert grads[i].dtype == leaves[i].dtype
            close(grads[i], refs[i], errs[i], what)
    with torch.no_grad():
        assert torch.equal(mod.layer_norm(*leaves, eps, out), y)


# every width of the kernels' tables (waves a row, chunks a thread, rows read again), their borders, odd ones
SIZES = [(1, 1), (3, 2), (1, 7), (5, 8), (2, 31), (9, 64), (1, 511), (4, 512), (7, 513), (33, 1000), (5, 1024), (6, 1025),
         (3, 1601), (66, 2048), (2, 2049), (17, 2055), (1, 4096), (130, 4097), (5, 8192), (2, 8193), (3, 12289), (1, 16384),
         (4, 16385), (2, 20000), (3, 70001), (1500, 96)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_against_binary64(mod, dtype, rows, cols):
    dt = DTYPES[dtype]
    x = draw((rows, cols), dt, rows + cols, 1.5, 0.3)
    if rows > 2:
        x[rows // 2] = 0
    check(mod, x, draw((cols,), dt, 1, 0.2, 1.0), draw((cols,), dt, 2, 0.3), draw((rows, cols), dt, 3, 0.05))


@pytest.mark.parametrize("cols", [40, 1601, 3000, 5000, 9001, 17000])
def test_types_and_missing_parameters(mod, cols):
    rows = 6
    for i, (xt, wt, bt, out) in enumerate([("bf16", "fp32", "fp16", None), ("fp16", None, "fp32", None),
                                           ("fp32", "bf16", None, "bf16"), ("fp32", None, None, "fp16"),
                                           ("bf16", None, None, None), ("fp32", "fp32", "fp32", "bf16")]):
        xt, out = DTYPES[xt], None if out is None else DTYPES[out]
        w = None if wt is None else draw((cols,), DTYPES[wt], 10 + i, 0.2, 1.0)
        b = None if bt is None else draw((cols,), DTYPES[bt], 20 + i, 0.3)
        check(mod, draw((rows, cols), xt, 30 + i), w, b, draw((rows, cols), out or xt, 40 + i, 0.1), out=out)


def test_many_rows_and_large_mean(mod):
    check(mod, draw((5000, 70), torch.float32, 5, 1.0, 100.0), draw((70,), torch.float32, 6), None,
          draw((5000, 70), torch.float32, 7))
    check(mod, draw((3000, 300), torch.bfloat16, 8), draw((300,), torch.float32, 9), draw((300,), torch.float32, 10),
          draw((3000, 300), torch.bfloat16, 11), eps=0.0)


@pytest.mark.parametrize("cols", [100, 1000, 3000, 20000])
def test_differences(mod, cols):
    """The gradients against central differences of the binary64 formula, along random directions."""
    from oracle import block
    rows, eps = 4, 1e-5
    x, w, b = draw((rows, cols), torch.float32, 1), draw((cols,), torch.float32, 2, 0.3, 1.0), draw((cols,), torch.float32, 3)
    dy = draw((rows, cols), torch.float32, 4)
    leaves = [t.cuda().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(mod.layer_norm(*leaves, eps), leaves, dy.cuda())
    for i in range(3):
        v = np64(draw(leaves[i].shape, torch.float32, 50 + i))
        step = 1e-4

        def value(s):
            t = [np64(x), np64(w), np64(b)]
            t[i] = t[i] + s * v
            return (block.layer_norm(*t, eps)[0] * np64(dy)).sum()

        want = (value(step) - value(-step)) / (2 * step)
        got = (np64(grads[i]) * v).sum()
        # the differences' own error is step^2 (1e-8); each gradient element is off by some tens of u of its terms
        assert abs(got - want) <= 1e-5 * (np.abs(np64(grads[i])) * np.abs(v)).sum() + 1e-6 * abs(want)


def test_strides_shapes_and_empty(mod, f8lin):
    x = draw((12, 400), torch.bfloat16, 1).cuda()
    w = draw((256, 2), torch.bfloat16, 2, 0.2, 1.0).cuda()[:, 0]  # a strided parameter
    want = mod.layer_norm(x[:, 8:264].contiguous(), w.contiguous())
    assert torch.equal(mod.layer_norm(x[:, 8:264], w), want)
    assert torch.equal(mod.layer_norm(x[:, 8:264].t().contiguous().t(), w), want)
    assert torch.equal(mod.layer_norm(x[:, 8:264].reshape(3, 2, 2, 256), w), want.view(3, 2, 2, 256))
    one = mod.layer_norm(x[0, 8:264], w)
    assert one.shape == (256,) and torch.equal(one, want[0])
    # a row stride into the kernels themselves, at an address of one element
    y = torch.empty((12, 255), dtype=torch.bfloat16, device="cuda")
    f8lin.layer_norm_forward(x[:, 1:256], y)
    assert torch.equal(y, mod.layer_norm(x[:, 1:256].contiguous()))
    # expanded rows and expanded gradients
    e = x[:1, :256].expand(5, 256).detach().requires_grad_()
    out = mod.layer_norm(e, w)
    g, = torch.autograd.grad(out, e, torch.ones((1, 1), dtype=torch.bfloat16, device="cuda").expand(5, 256))
    assert g.shape == (5, 256)
    for shape in ((0, 64), (3, 0), (0, 0), (2, 0, 5)):
        t = torch.empty(shape, dtype=torch.float32, device="cuda", requires_grad=True)
        p = torch.ones(shape[-1], device="cuda", requires_grad=True)
        out = mod.layer_norm(t, p, p)
        assert out.shape == shape
        gt, gp = torch.autograd.grad(out, (t, p), torch.empty(shape, device="cuda"))
        assert gt.shape == shape and torch.equal(gp, torch.zeros_like(p))


@pytest.mark.parametrize("cols", [96, 1024, 4096, 16000, 30000])
def test_rows_that_are_not_finite(mod, cols):
    """A row with an Inf or NaN is NaN (and its dx), the others are untouched; the parameters' sums become NaN."""
    x, dy = draw((9, cols), torch.bfloat16, 1).cuda(), draw((9, cols), torch.bfloat16, 2).cuda()
    clean = mod.layer_norm(x)
    bad = x.clone()
    bad[2, cols // 2] = float("inf")
    bad[5, 0] = float("nan")
    bad[7, cols - 1] = float("-inf")
    leaf = bad.requires_grad_()
    y = mod.layer_norm(leaf)
    dx, = torch.autograd.grad(y, leaf, dy)
    ok = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y[ok], clean[ok]) and torch.isfinite(dx[ok].float()).all()
    assert torch.isnan(y[[2, 5, 7]].float()).all() and torch.isnan(dx[[2, 5, 7]].float()).all()


def test_amax_feeds_float8(f8lin):
    """y_amax is max |y| of the rounded output, whatever the word held, and what f8lin_forward's own pass finds."""
    for rows, cols in ((1, 160), (48, 160), (300, 4096), (40, 9008)):
        x = draw((rows, cols), torch.bfloat16, rows).cuda()
        y, amax = torch.empty_like(x), torch.full((1,), 3e38, device="cuda")
        f8lin.layer_norm_forward(x, y, y_amax=amax)
        assert amax.item() == y.float().abs().max().item()
    x = draw((64, 160), torch.float32, 5).cuda()
    y, amax = torch.empty((64, 160), dtype=torch.bfloat16, device="cuda"), torch.empty(1, device="cuda")
    f8lin.layer_norm_forward(x, y, y_amax=amax)
    w = draw((96, 160), torch.bfloat16, 6, 0.1).cuda()
    own, given = f8lin.LinearBuffers(64, 96, 160), f8lin.LinearBuffers(64, 96, 160)
    own.forward(y, w)
    g = given
    g.sx.amax.copy_(amax)
    f8lin.forward(y, w, g.y, g.x8, g.x8t, g.w8, g.w8t, g.sx, g.sw, g.ws, x_amax_given=True)
    assert torch.equal(own.y, given.y) and torch.equal(own.x8, given.x8) and torch.equal(own.sx.scale, given.sx.scale)
    x[3, 7] = float("nan")
    f8lin.layer_norm_forward(x, y, y_amax=amax)
    assert torch.isnan(amax).item()
    f8lin.layer_norm_forward(x[:0], y[:0], y_amax=amax)
    assert amax.item() == 0


def test_same_bits_every_run(mod):
    x, w, b = (draw(s, torch.bfloat16, i).cuda().requires_grad_() for i, s in enumerate(((3001, 1600), (1600,), (1600,))))
    dy = draw((3001, 1600), torch.bfloat16, 9).cuda()
    runs = []
    for _ in range(3):
        y = mod.layer_norm(x, w, b)
        runs.append((y, *torch.autograd.grad(y, (x, w, b), dy)))
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


def test_refusals(mod, f8lin):
    x = torch.ones((4, 8), device="cuda")
    with pytest.raises(ValueError):
        mod.layer_norm(x, torch.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        mod.layer_norm(x, bias=torch.ones((1, 8), device="cuda"))
    with pytest.raises(ValueError):
        mod.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        mod.layer_norm(torch.ones((), device="cuda"))
    with pytest.raises(TypeError):
        mod.layer_norm(x.bfloat16(), out_dtype=torch.float32)
    with pytest.raises(TypeError):
        mod.layer_norm(x.double())
    with pytest.raises((ValueError, RuntimeError)):
        mod.layer_norm(x, torch.ones(8))
    with pytest.raises(NotImplementedError), torch.no_grad(), torch.autograd.forward_ad.dual_level():
        mod.layer_norm(torch.autograd.forward_ad.make_dual(x, x))
    leaf = draw((4, 8), torch.float32, 1).cuda().requires_grad_()
    g, = torch.autograd.grad((mod.layer_norm(leaf) ** 3).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):  # once differentiable
        torch.autograd.grad(g.sum(), leaf)
    with pytest.raises(f8lin.F8linError):
        f8lin.layer_norm_forward(x, x)  # in place
    with pytest.raises(f8lin.F8linError):
        f8lin.layer_norm_backward(x, x.clone(), None, x[:, :2].contiguous(), dweight=x[0].clone())


def test_module_and_swap(mod):
    torch.manual_seed(0)
    shared = nn.LayerNorm(40)
    model = nn.Sequential(shared, nn.Linear(40, 40), shared, nn.LayerNorm(40, elementwise_affine=False),
                          nn.Sequential(nn.LayerNorm(40, bias=False, eps=0.1)), nn.Unflatten(1, (5, 8)), nn.LayerNorm((5, 8)))
    model = model.cuda()
    with torch.no_grad():
        for p in model.parameters():
            p.add_(0.1 * torch.randn_like(p))
    x = torch.randn((30, 40), device="cuda", requires_grad=True)
    want = model(x)
    dy = torch.randn_like(want)
    wants = torch.autograd.grad(want, [x, *model.parameters()], dy)
    state = {k: v.clone() for k, v in model.state_dict().items()}
    assert mod.convert_layer_norm(model) is model
    assert sum(type(m) is mod.LayerNorm for m in model.modules()) == 4 and model[0] is model[2]
    assert model.state_dict().keys() == state.keys()
    got = model(x)
    gots = torch.autograd.grad(got, [x, *model.parameters()], dy)
    # both in binary32: some hundreds of roundings apart at most
    for p, q in zip((got, *gots), (want, *wants)):
        assert p.shape == q.shape and (p - q).abs().max() <= 3e-5 * q.abs().max()
    assert "normalized_shape" not in repr(model[6]) and "(5, 8)" in repr(model[6])
    with pytest.raises(ValueError):
        model[0](torch.ones((2, 41), device="cuda"))
    assert model[6](torch.empty((0, 5, 8), device="cuda")).shape == (0, 5, 8)


def test_captured_and_streams(mod):
    """A step replayed in a graph with new inputs, and eager steps between the replays; two streams at once."""
    w = draw((1600,), torch.float32, 1, 0.1, 1.0).cuda().requires_grad_()
    b = draw((1600,), torch.float32, 2).cuda().requires_grad_()
    x = draw((700, 1600), torch.bfloat16, 3).cuda().requires_grad_()
    dy = draw((700, 1600), torch.bfloat16, 4).cuda()

    def step(x, dy):
        y = mod.layer_norm(x, w, b)
        return (y.detach(), *torch.autograd.grad(y, (x, w, b), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, dy)
    for seed in range(3):
        with torch.no_grad():
            x.copy_(draw((700, 1600), torch.bfloat16, 10 + seed))
            dy.copy_(draw((700, 1600), torch.bfloat16, 20 + seed))
        graph.replay()
        got = [t.clone() for t in out]
        want = step(x.detach().clone().requires_grad_(), dy.clone())
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        torch.cuda.synchronize()
    del graph, out
    streams = [torch.cuda.Stream() for _ in range(2)]
    ins = [(draw((700, 1600), torch.bfloat16, 30 + i).cuda().requires_grad_(), dy.clone()) for i in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(step(*ins[i]))
    torch.cuda.synchronize()
    for i in range(2):
        want = step(*ins[i])
        for got in outs[i]:
            assert all(torch.equal(p, q) for p, q in zip(got, want))
