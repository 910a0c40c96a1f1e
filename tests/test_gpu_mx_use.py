"""The MXFP4 layer and gradient clipping as they are used: a training step of a small model, serving from frozen
weights, captured graphs, other streams, calls that overlap in time, mixed types."""
import numpy as np
import pytest
import torch
import torch.nn as nn

from test_gpu_mxfp4 import DTYPES, check_product, draw, f8lin, mod, mx, np64, out_half_step, random_mx  # noqa: F401

pytestmark = pytest.mark.gpu


class Block(nn.Module):
    def __init__(self, d, hidden):
        super().__init__()
        self.norm = nn.LayerNorm(d)
        self.fc1 = nn.Linear(d, hidden)
        self.fc2 = nn.Linear(hidden, d, bias=False)

    def forward(self, x):
        return x + self.fc2(torch.relu(self.fc1(self.norm(x))))


def build(mod, d=70, hidden=130, dtype=torch.float32):
    torch.manual_seed(0)
    model = nn.Sequential(Block(d, hidden), Block(d, hidden), nn.Linear(d, 5)).to("cuda", dtype)
    return mod.convert_to_mxfp4_training(model, module_filter_fn=lambda fqn, m: m.out_features != 5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_training_steps(mod, mx, dtype):
    """Forward, backward, clipping and an optimiser step: every MXFP4 layer's output and gradients against the formulas
    on the input and output gradient it really saw, the norm and the clipped gradients against binary64."""
    dt = DTYPES[dtype]
    model = build(mod, dtype=dt)
    layers = [m for m in model.modules() if isinstance(m, mod.MXFP4Linear)]
    assert len(layers) == 4 and type(model[2]) is nn.Linear
    seen = {}
    for layer in layers:
        layer.register_forward_hook(lambda m, i, o: seen.__setitem__(m, [i[0].detach().clone(), o.detach().clone()]))
        layer.register_full_backward_hook(
            lambda m, gi, go: seen[m].extend([gi[0].detach().clone(), go[0].detach().clone()]))
    opt = torch.optim.SGD(model.parameters(), lr=0.1)
    for step in range(3):
        x = draw((3, 11, 70), dt, step).cuda()
        target = draw((3, 11, 5), dt, 100 + step).cuda()
        loss = ((model(x) - target).float() ** 2).mean()
        opt.zero_grad()
        loss.backward()
        for layer in layers:
            inp, out, gin, gout = (np64(t).reshape(-1, t.shape[-1]) for t in seen[layer])
            w = np64(layer.weight)
            b = None if layer.bias is None else np64(layer.bias)
            check_product(seen[layer][1].view(33, -1), mx.rounded(inp), mx.rounded(w), dt, b, "Y")
            check_product(seen[layer][2].view(33, -1), mx.rounded(gout), mx.rounded(w.T), dt, what="dX")
            check_product(layer.weight.grad, mx.rounded(gout.T), mx.rounded(inp.T), dt, what="dW")
            if b is not None:
                tol = 35 * 2.0 ** -23 * np.abs(gout).sum(0)
                ref = gout.sum(0)
                assert np.all(np.abs(np64(layer.bias.grad) - ref) <= tol + out_half_step(np.abs(ref) + tol, dt))
        before = [np64(p.grad) for p in model.parameters()]
        want = mx.norm(before, 2.0)
        norm = mod.clip_grad_norm_(model.parameters(), 0.5 * want)
        n = sum(g.size for g in before)
        assert abs(float(norm) - want) <= want * (2.0 ** -23 + n * 2.0 ** -52)
        c = 0.5 * want / (want + 1e-6)
        for p, g in zip(model.parameters(), before):
            tol = np.abs(g * c) * (8 * 2.0 ** -24 + torch.finfo(dt).eps / 2 * 1.01) + 2.0 ** -133
            assert np.all(np.abs(np64(p.grad) - g * c) <= tol)
        opt.step()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_serving_from_frozen_weights(f8lin, mod, mx, dtype):
    dt = DTYPES[dtype]
    model = build(mod, dtype=dt).eval()
    x = draw((2, 9, 70), dt, 3).cuda()
    with torch.no_grad():
        want = model(x)
        mod.freeze_mxfp4(model)
        layers = [m for m in model.modules() if isinstance(m, mod.MXFP4Linear)]
        assert all(m.frozen and m.weight is None for m in layers) and "frozen=True" in repr(model)
        assert torch.equal(model(x), want)  # the same codes, the same kernels
        one = model(x[:1, :1])              # X quantised inside the product: other order of the same sums
        assert one.shape == (1, 1, 5)
        state = model.state_dict()
        assert state["0.fc1.weight_codes"].dtype == torch.uint8 and "0.fc1.weight" not in state
        other = mod.freeze_mxfp4(build(mod, dtype=dt))
        for p in other.parameters():
            p.add_(1)
        for m in other.modules():
            if isinstance(m, mod.MXFP4Linear):
                m.weight_codes.zero_()
        other.load_state_dict(state)
        assert torch.equal(other(x), want)
        assert torch.equal(other.cpu().cuda()(x), want)
    assert not layers[0].bias.requires_grad
    assert layers[0](x).requires_grad is False
    with pytest.raises(RuntimeError):
        layers[0](x.clone().requires_grad_())
    assert layers[0].freeze() is layers[0]


def test_mixed_types(mod, mx):
    """Activations, weight and bias of three types: outputs and gradients take their own tensor's."""
    x, w, b = draw((50, 70), torch.bfloat16, 1), draw((90, 70), torch.float32, 2, 0.1), draw((90,), torch.float16, 3)
    leaves = [t.cuda().requires_grad_() for t in (x, w, b)]
    dy = draw((50, 90), torch.bfloat16, 4, 0.1)
    y = mod.mxfp4_linear(*leaves)
    assert y.dtype == torch.bfloat16
    dx, dw, db = torch.autograd.grad(y, leaves, dy.cuda())
    assert (dx.dtype, dw.dtype, db.dtype) == (torch.bfloat16, torch.float32, torch.float16)
    X, W, DY = np64(x), np64(w), np64(dy)
    check_product(y, mx.rounded(X), mx.rounded(W), torch.bfloat16, np64(b))
    check_product(dx, mx.rounded(DY), mx.rounded(W.T), torch.bfloat16)
    check_product(dw, mx.rounded(DY.T), mx.rounded(X.T), torch.float32)
    assert np.all(np.abs(np64(db) - DY.sum(0)) <= 52 * 2.0 ** -23 * np.abs(DY).sum(0) + out_half_step(DY.sum(0), torch.float16) * 1.01)


def test_strided_operands(mod):
    """Slices of wider buffers and transposed weights and gradients give what their copies give."""
    wide = draw((60, 200), torch.bfloat16, 1).cuda()
    wt = draw((70, 90), torch.bfloat16, 2, 0.1).cuda()
    dyw = draw((90, 60), torch.bfloat16, 3, 0.1).cuda()
    x, w, dy = wide[:, 13:83], wt.t(), dyw.t()
    got, want = [], []
    for out, a, b, g in ((got, x, w, dy), (want, x.contiguous(), w.contiguous(), dy.contiguous())):
        a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
        y = mod.mxfp4_linear(a, b)
        out += [y, *torch.autograd.grad(y, (a, b), g)]
    assert all(torch.equal(p, q) for p, q in zip(got, want))


SHAPES = [(1, 300, 260), (40, 300, 260), (200, 300, 260), (1100, 1300, 700), (4200, 4100, 300)]


def step_buffers(f8lin, M, N, K, seed):
    """Inputs, buffers and the calls of one layer's forward, backward and clipping at the binding."""
    dt = torch.bfloat16
    x, w, dy, b = (draw(s, dt, seed + i, v).cuda() for i, (s, v) in
                   enumerate((((M, K), 1.0), ((N, K), 0.1), ((M, N), 0.1), ((N,), 1.0))))
    out = {"y": torch.empty((M, N), dtype=dt, device="cuda"), "dx": torch.empty((M, K), dtype=dt, device="cuda"),
           "dw": torch.empty((N, K), device="cuda"), "db": torch.empty((N,), dtype=dt, device="cuda"),
           "serve": torch.empty((M, N), dtype=dt, device="cuda"), "norm": torch.zeros((), device="cuda"),
           "cdw": torch.empty((N, K), dtype=dt, device="cuda"), "cdb": torch.empty((N,), device="cuda")}
    q = {n: f8lin.new_mxfp4(r, c) for n, r, c in (("x", M, K), ("xt", K, M), ("w", N, K), ("wt", K, N), ("dy", M, N),
                                                  ("dyt", N, M), ("x2", M, K))}
    dbw = torch.empty(max(1, f8lin.mxfp4_dbias_workspace_bytes(M, N) // 4), device="cuda")
    ws = f8lin.new_grad_workspace()

    def run(stream=None):
        f8lin.mxfp4_forward(x, w, out["y"], q["x"], q["w"], q["xt"], q["wt"], b, stream=stream)
        f8lin.mxfp4_backward(dy, q["xt"], q["wt"], out["dx"], out["dw"], q["dy"], q["dyt"], out["db"], dbw, stream=stream)
        f8lin.mxfp4_forward(x, None, out["serve"], q["x2"], q["w"], bias=b, stream=stream)
        f8lin.grad_clip([out["dw"], out["db"]], 0.01, out["norm"], ws, outs=[out["cdw"], out["cdb"]], stream=stream)

    return (x, w, dy, b), out, run


def snapshot(out):
    return {k: v.clone() for k, v in out.items()}


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_captured_and_replayed(f8lin, M, N, K):
    """One graph of forward, backward, serving and clipping; new inputs before each replay, eager calls between."""
    inputs, out, run = step_buffers(f8lin, M, N, K, 1)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(3):
        for t in inputs:
            t.copy_(draw(t.shape, t.dtype, 50 + seed, float(t.float().std())))
        run()
        want = snapshot(out)
        for t in out.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in out.items():
            assert torch.equal(t, want[k]), k
    assert all(torch.isfinite(t).all() for t in out.values())


def test_streams(f8lin, mod):
    """An explicit stream, the current stream of a context, and two steps at once on two streams."""
    sets = [step_buffers(f8lin, 200 + 900 * i, 300, 260, 10 * i) for i in range(2)]
    want = []
    for _, out, run in sets:
        run()
        want.append(snapshot(out))
    streams = [torch.cuda.Stream() for _ in sets]
    for how in ("given", "current"):
        for _, out, _ in sets:
            for t in out.values():
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for (_, _, run), st in zip(sets, streams):
                if how == "given":
                    run(st)
                else:
                    with torch.cuda.stream(st):
                        run()
        torch.cuda.synchronize()
        for (_, out, _), w in zip(sets, want):
            for k, t in out.items():
                assert torch.equal(t, w[k]), (how, k)


def test_rows_behind_the_last_are_left(f8lin):
    """Outputs of a padded batch: the rows behind M, and the codes of rows that were not quantised, stay as they were."""
    x = draw((40, 96), torch.bfloat16, 1).cuda()
    w = draw((50, 96), torch.bfloat16, 2).cuda()
    qw = f8lin.new_mxfp4(50, 96)
    f8lin.mxfp4_quantize(w, qw)
    for M in (1, 5, 17, 33):
        q = f8lin.new_mxfp4(40, 96)
        q.codes.fill_(0x5A)
        q.scales.fill_(0xA5)
        part = f8lin.MXFP4Tensor(q.codes[:M], q.scales[:M], M, 96)
        f8lin.mxfp4_quantize(x[:M], part)
        assert (q.codes[M:] == 0x5A).all() and (q.scales[M:] == 0xA5).all()
        y = torch.full((40, 50), 7.0, device="cuda")
        f8lin.mxfp4_forward(x[:M], None, y[:M], part, qw)
        assert (y[M:] == 7).all() and not (y[:M] == 7).all()
        d = torch.full((40, 96), 7.0, device="cuda")
        f8lin.mxfp4_dequantize(part, d[:M])
        assert (d[M:] == 7).all()


def test_largest_strides(f8lin, mx):
    """Rows set 4 MiB apart in codes (the largest stride): offsets of a tile pass 2^30 bytes."""
    M, N, K = 300, 70, 200
    a, av = random_mx(f8lin, mx, M, K, 1)
    b, bv = random_mx(f8lin, mx, N, K, 2)
    ld = 1 << 22
    codes = torch.empty(M * ld, dtype=torch.uint8, device="cuda").view(M, ld)
    codes[:, :a.codes.shape[1]] = a.codes
    far = f8lin.MXFP4Tensor(codes, a.scales, M, K)
    for rows in (300, 60):
        part = f8lin.MXFP4Tensor(codes[:rows], a.scales[:rows], rows, K)
        c = torch.empty((rows, N), device="cuda")
        f8lin.mxfp4_gemm([(part, b, c)])
        check_product(c, av[:rows], bv, torch.float32)
    c = torch.empty((N, M), device="cuda")
    f8lin.mxfp4_gemm([(b, far, c)])
    check_product(c, bv, av, torch.float32)
    with pytest.raises(f8lin.F8linError):
        f8lin.mxfp4_dequantize(f8lin.MXFP4Tensor(codes.view(-1)[:3 * 2 * ld].view(3, 2 * ld), a.scales[:3], 3, K),
                               torch.empty((3, K), device="cuda"))


def test_wide_and_tall(f8lin, mx):
    """One very long row, one very long column, and a contraction over each."""
    for rows, cols in ((1, 300_001), (300_001, 1), (2, 100_003)):
        x = draw((rows, cols), torch.bfloat16, 5)
        q, qt = f8lin.new_mxfp4(rows, cols), f8lin.new_mxfp4(cols, rows)
        f8lin.mxfp4_quantize(x.cuda(), q, qt)
        assert np.array_equal(np64(q.dequantize(torch.float32)), mx.rounded(np64(x)))
        assert np.array_equal(np64(qt.dequantize(torch.float32)), mx.rounded(np64(x).T))
    x, w = draw((3, 100_003), torch.bfloat16, 6), draw((5, 100_003), torch.bfloat16, 7)
    qx, qw = f8lin.new_mxfp4(3, 100_003), f8lin.new_mxfp4(5, 100_003)
    f8lin.mxfp4_quantize(x.cuda(), qx)
    f8lin.mxfp4_quantize(w.cuda(), qw)
    c = torch.empty((3, 5), device="cuda")
    f8lin.mxfp4_gemm([(qx, qw, c)])
    check_product(c, mx.rounded(np64(x)), mx.rounded(np64(w)), torch.float32)


@pytest.mark.parametrize("m, n", [(1, 1), (129, 33), (4096, 31), (4097, 32), (33000, 65), (140001, 3)])
def test_bias_gradient_of_many_rows(f8lin, m, n):
    """The column sums alone, over fewer and more row tiles than the groups that add them up; the same bits twice."""
    dy = draw((m, n), torch.float32, m + n).cuda()
    ws = torch.empty(f8lin.mxfp4_dbias_workspace_bytes(m, n) // 4, device="cuda")
    got = []
    for _ in range(2):
        db = torch.full((n,), float("nan"), device="cuda")
        f8lin.mxfp4_backward(dy, None, None, None, None, None, f8lin.new_mxfp4(n, m), db, ws.fill_(float("nan")))
        got.append(np64(db))
    ref = np64(dy).sum(0)
    # an element passes 32 + 2 additions in its tile, tiles / 32 in its group and 31 joining them, each off by half a
    # step of at most the sum of magnitudes
    depth = 34 + -(-m // 128) // 32 + 1 + 31
    assert np.all(np.abs(got[0] - ref) <= depth * 2.0 ** -24 * 1.01 * np.abs(np64(dy)).sum(0))
    assert np.array_equal(got[0], got[1])


@pytest.mark.parametrize("m", [1, 2, 3])
def test_codes_of_x_are_left_where_asked_for(f8lin, mx, m):
    """A forward that is given x4 writes X's codes there, however few the rows; without it the result is the same."""
    n, k = 96, 333
    x, w = draw((m, k), torch.bfloat16, m).cuda(), draw((n, k), torch.bfloat16, 7).cuda()
    w4, x4 = f8lin.new_mxfp4(n, k), f8lin.new_mxfp4(m, k)
    f8lin.mxfp4_quantize(w, w4)
    x4.codes.fill_(0xA5), x4.scales.fill_(0xA5)
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    f8lin.mxfp4_forward(x, None, y, x4, w4)
    assert np.array_equal(np64(x4.dequantize(torch.float32)), mx.rounded(np64(x)))
    check_product(y, mx.rounded(np64(x)), mx.rounded(np64(w)), torch.bfloat16)
    if f8lin.mxfp4_forward_fused(m, n, k):
        y2 = torch.empty_like(y)
        f8lin.mxfp4_forward(x, None, y2, None, w4)
        check_product(y2, mx.rounded(np64(x)), mx.rounded(np64(w)), torch.bfloat16)


@pytest.mark.parametrize("m, n, k", [
    (16, 40, 200), (13, 33, 511), (12, 70, 1024), (6, 50, 1600), (4, 50, 4096), (2, 35, 14336), (3, 17, 9),  # X quantised inside
    (16, 4100, 96), (9, 8200, 96), (16, 12300, 100), (5, 20001, 64),                      # one to four blocks of columns
    (17, 4100, 96), (17, 8200, 300), (32, 12288, 40), (17, 12289, 36),
    (33, 4100, 70), (64, 8192, 36), (33, 8193, 36), (49, 600, 4100), (20, 600, 8200)])
def test_few_rows_against_quantised_weights(mod, f8lin, mx, m, n, k):
    """Each path that a few rows can take: X quantised inside the product or ahead of it, its splits, the tiled one."""
    x, w = draw((m, k), torch.bfloat16, m + k).cuda(), draw((n, k), torch.bfloat16, n).cuda()
    bias = draw((n,), torch.bfloat16, 3).cuda()
    w4 = f8lin.new_mxfp4(n, k)
    f8lin.mxfp4_quantize(w, w4)
    y = mod.mxfp4_linear(x, w4, bias)
    check_product(y, mx.rounded(np64(x)), mx.rounded(np64(w)), torch.bfloat16, np64(bias))


def test_where_x_is_quantised_inside(f8lin):
    """One row for every weight whose row a workgroup can take on itself; no batch beyond 16 rows, nothing empty."""
    assert all(f8lin.mxfp4_forward_fused(1, n, k) for n in (1, 4096, 28672) for k in (1, 4096))
    assert f8lin.mxfp4_forward_fused(16, 64, 256) and not f8lin.mxfp4_forward_fused(17, 64, 256)
    assert not any(f8lin.mxfp4_forward_fused(*s) for s in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (16, 4096, 4096)))


def test_layer_step_captured(mod, f8lin):
    """A whole step of layers under autograd -- forward, backward, clipping -- as one graph, replayed on new inputs with
    eager steps between; the eager graphs of the same leaves are gone before the capture."""
    model = build(mod, dtype=torch.bfloat16)
    params = list(model.parameters())
    x, target = (torch.empty((3, 11, n), dtype=torch.bfloat16, device="cuda") for n in (70, 5))

    def step():
        y = model(x)
        grads = torch.autograd.grad(y, params, (y - target).detach())
        norm, clipped = mod.clip_grads(grads, 0.5, out_dtype=torch.float32)
        return [y.detach(), norm, *clipped]

    def load(seed):
        x.copy_(draw(x.shape, x.dtype, seed))
        target.copy_(draw(target.shape, target.dtype, 100 + seed))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up; nothing of it is kept
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(1, 4):
        load(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.isfinite(t).all() for t in want)
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("rows, cols, pad", [(8192, 1024, 0), (8190, 1030, 0), (8192, 1024, 8), (8300, 960, 64), (65536, 128, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_many_tiles(f8lin, mx, rows, cols, pad, dtype):
    """Enough tiles for the big ones, X's rows aligned to 128 bytes and not: both layouts at once, and each alone, agree
    with the oracle bit for bit."""
    buf = draw((rows, cols + pad), DTYPES[dtype], rows + cols + pad).cuda()
    x = buf[:, :cols]
    ref = [mx.rounded(np64(x)), mx.rounded(np64(x).T)]
    q, qt = f8lin.new_mxfp4(rows, cols), f8lin.new_mxfp4(cols, rows)
    f8lin.mxfp4_quantize(x, q, qt)
    for t, want in zip((q, qt), ref):
        assert np.array_equal(np64(t.dequantize(torch.float32)), want)
    for i, t in enumerate((f8lin.new_mxfp4(rows, cols), f8lin.new_mxfp4(cols, rows))):
        f8lin.mxfp4_quantize(x, t if i == 0 else None, t if i == 1 else None)
        assert np.array_equal(np64(t.dequantize(torch.float32)), ref[i])


@pytest.mark.parametrize("rows, cols", [(163840, 1088), (163841, 1090)])
def test_more_than_the_caches_hold(f8lin, rows, cols):
    """A large tensor, its rows aligned to 128 bytes and not, against the same in pieces: codes, scales and values."""
    gen = torch.Generator("cuda").manual_seed(rows)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    q, qt, alone, back = (f8lin.new_mxfp4(*s) for s in ((rows, cols), (cols, rows), (rows, cols), (cols, rows)))
    f8lin.mxfp4_quantize(x, q, qt)
    f8lin.mxfp4_quantize(x, alone)
    f8lin.mxfp4_quantize(x, None, back)
    values = q.dequantize()
    cb, step = -(-cols // 32), 4096
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        p, pt = f8lin.new_mxfp4(n, cols), f8lin.new_mxfp4(cols, n)
        f8lin.mxfp4_quantize(x[r0:r0 + n], p, pt)
        nb = -(-n // 32)
        for t in (q, alone):
            assert torch.equal(t.codes[r0:r0 + n, :16 * cb], p.codes[:, :16 * cb])
            assert torch.equal(t.scales[r0:r0 + n, :cb], p.scales[:, :cb])
        for t in (qt, back):
            assert torch.equal(t.codes[:, r0 // 2:r0 // 2 + 16 * nb], pt.codes[:, :16 * nb])
            assert torch.equal(t.scales[:, r0 // 32:r0 // 32 + nb], pt.scales[:, :nb])
        assert torch.equal(values[r0:r0 + n], p.dequantize())


def test_no_transposed_copies_without_gradients(mod, f8lin, mx, monkeypatch):
    """Under no_grad a trainable layer quantises for its product alone; with gradients for one operand, only for that."""
    layer = mod.MXFP4Linear(70, 50, device="cuda", dtype=torch.float32, bias=True)
    x = draw((9, 70), torch.float32, 5).cuda()
    made, real = [], f8lin.new_mxfp4s
    monkeypatch.setattr(f8lin, "new_mxfp4s", lambda shapes, *a: made.extend(shapes) or real(shapes, *a))
    with torch.no_grad():
        y = layer(x)
    assert sorted(made) == [(9, 70), (50, 70)] and not y.requires_grad
    made.clear()
    z = layer(x)
    assert torch.equal(z, y) and sorted(made) == [(9, 70), (50, 70), (70, 9)]
    made.clear()
    layer.weight.requires_grad_(False)
    z = layer(x.clone().requires_grad_())
    assert torch.equal(z, y) and sorted(made) == [(9, 70), (50, 70), (70, 50)]
    check_product(y, mx.rounded(np64(x)), mx.rounded(np64(layer.weight)), torch.float32, np64(layer.bias))
