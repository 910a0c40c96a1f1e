"""Low-rank adapters on the GPU: plans, forward and backward against binary64 within counted roundings and, at large
sizes, exactly; masked tokens, ranks, strides, bad indices, graphs, streams, the module."""
import numpy as np
import pytest
import torch
import torch.nn as nn

from block_helpers import DTYPES, close, draw, lora_bounds, lora_grad_bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def f8lin():
    from float8linear_tensorwise_amax_amd import f8lin
    return f8lin


@pytest.fixture(scope="module")
def mod():
    from float8linear_tensorwise_amax_amd import module
    return module


def index_of(tokens, adapters, seed, kind="mixed"):
    """Each token's adapter: sequences of several lengths, some without an adapter, in no order."""
    rng = np.random.default_rng(seed)
    if kind == "single":
        return rng.integers(-1, adapters, tokens).astype(np.int32)
    if kind == "one":
        return np.full(tokens, adapters - 1, dtype=np.int32)
    out = []
    while len(out) < tokens:
        out += [int(rng.integers(-1, adapters))] * int(rng.choice([1, 1, 2, 5, 63, 64, 65, 200, 700]))
    return np.array(out[:tokens], dtype=np.int32)


# ---------------------------------------------------------------- the plan

def plan_reference(index, adapters):
    i = np.where((index >= 0) & (index < adapters), index, adapters)
    order = np.argsort(i, kind="stable")
    starts = np.searchsorted(i[order], np.arange(adapters + 2))
    tiles, rows = [], 16 if len(index) <= 1024 else 64
    for a in range(adapters + 1):
        tiles += [(a, p, min(rows, starts[a + 1] - p), order[p]) for p in range(starts[a], starts[a + 1], rows)]
    return order, starts, tiles, i[order]


@pytest.mark.parametrize("tokens,adapters", [(1, 1), (1, 2047), (2, 3), (63, 1), (64, 64), (65, 7), (1000, 255), (1023, 256),
                                             (4097, 2047), (70000, 5), (70001, 2000)])
@pytest.mark.parametrize("kind", ["mixed", "single"])
def test_plan(f8lin, tokens, adapters, kind):
    index = index_of(tokens, adapters, tokens, kind).astype(np.int64)
    if tokens > 3:
        index[0], index[-1], index[tokens // 2] = 1 << 40, adapters, -(1 << 33)
    plan = f8lin.LoraPlan(tokens, adapters)
    plan.buffer.fill_(-7)
    version = plan.buffer._version
    f8lin.lora_plan(torch.from_numpy(index).cuda(), plan)
    assert plan.buffer._version > version
    got = plan.buffer.cpu().numpy()
    order, starts, tiles, owner = plan_reference(index, adapters)
    assert got[1:4].tolist() == [tokens, adapters, len(tiles)]
    assert np.array_equal(got[4:4 + adapters + 2], starts)
    at = (4 + adapters + 2 + 3) // 4 * 4
    assert np.array_equal(got[at:at + 4 * len(tiles)].reshape(-1, 4), np.array(tiles))
    assert np.array_equal(got[len(got) - 2 * tokens:len(got) - tokens], order)
    assert np.array_equal(got[len(got) - tokens:], owner)
    if np.all(np.abs(index) < 1 << 31):
        again = f8lin.LoraPlan(tokens, adapters)
        again.buffer.fill_(-7)
        f8lin.lora_plan(torch.from_numpy(index.astype(np.int32)).cuda(), again)
        assert torch.equal(again.buffer, plan.buffer)


# ------------------------------------------------- forward and backward

def tensors(T, K, N, R, L, dt, seed, base_std=1.0):
    x = draw((T, K), dt, seed)
    base = draw((T, N), dt, seed + 1, base_std)
    a, b = draw((L, R, K), dt, seed + 2, K ** -0.5), draw((L, N, R), dt, seed + 3, 0.3)
    dy = draw((T, N), dt, seed + 4, 0.1)
    scales = torch.rand(L, generator=torch.Generator().manual_seed(seed)) + 0.5
    return base, x, a, b, dy, scales


def check(mod, T, K, N, R, L, dt, index, seed=0, use_scales=True):
    base, x, a, b, dy, scales = tensors(T, K, N, R, L, dt, seed)
    if not use_scales:
        scales = torch.ones(L)
    batch = mod.LoraBatch(torch.from_numpy(index).cuda(), L)
    leaves = [t.cuda().requires_grad_() for t in (base, x, a, b)]
    dyc = dy.cuda()
    y = mod.lora_add(*leaves, batch, scales.cuda() if use_scales else None)
    db_, dx, da, db = torch.autograd.grad(y, leaves, dyc)
    B, X, A, Bm, DY, S = (np64(t) for t in (base, x, a, b, dy, scales))
    ref, h, d_y, d_h = lora_bounds(B, X, A, Bm, index, S, dt)
    close(y, ref, d_y, "y")
    none = (index < 0) | (index >= L)
    assert torch.equal(y.detach().cpu()[none], base[none])  # to the bit
    assert torch.equal(db_, dyc)
    refs, errs = lora_grad_bounds(DY, X, A, Bm, index, S, h, d_h, dt)
    for got, r, e, what in zip((dx, da, db), refs, errs, ("dx", "dA", "dB")):
        assert got.dtype == dt and got.shape == r.shape
        close(got, r, e, what)
    assert not np64(dx)[none].any()
    with torch.no_grad():
        again = mod.lora_add(*leaves, batch, scales.cuda() if use_scales else None)
    assert torch.equal(again, y)


SIZES = [  # T, K, N, R, L
    (1, 1, 1, 1, 1), (1, 64, 64, 16, 1), (2, 33, 17, 3, 4), (5, 130, 70, 8, 2), (64, 100, 300, 16, 3), (65, 64, 256, 17, 2),
    (200, 257, 129, 32, 5), (300, 96, 515, 33, 3), (1000, 40, 48, 64, 7), (130, 70, 66, 65, 2), (90, 50, 90, 128, 2),
    (70, 60, 61, 256, 3), (700, 31, 1025, 12, 40), (33, 513, 1, 5, 9), (1500, 160, 96, 4, 2), (257, 1, 40, 2, 6)]


@pytest.mark.parametrize("T,K,N,R,L", SIZES)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_against_binary64(mod, dtype, T, K, N, R, L):
    check(mod, T, K, N, R, L, DTYPES[dtype], index_of(T, L, T + R), seed=T + K)


@pytest.mark.parametrize("kind", ["single", "one"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_mixes(mod, dtype, kind):
    check(mod, 300, 96, 136, 16, 20, DTYPES[dtype], index_of(300, 20, 3, kind), seed=1, use_scales=False)
    check(mod, 40, 1100, 72, 24, 50, DTYPES[dtype], index_of(40, 50, 4, kind), seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_chunks(mod, dtype):
    """An adapter's tokens over several workgroups' chunks, two adapters that end and begin in one, one that fills chunks
    exactly, one without a token."""
    index = np.concatenate([np.full(n, i) for i, n in ((0, 700), (2, 1), (3, 1348), (4, 3 * 128), (5, 1200), (6, 463))])
    check(mod, len(index), 48, 40, 8, 7, DTYPES[dtype], index.astype(np.int32), seed=5)
    perm = np.random.default_rng(0).permutation(len(index))
    check(mod, len(index), 48, 40, 8, 7, DTYPES[dtype], index[perm].astype(np.int32), seed=6)


@pytest.mark.parametrize("T,K,N,R,L,kind", [(1, 4096, 4096, 16, 8, "one"), (64, 4096, 14336, 16, 64, "single"),
                                            (3001, 4096, 1601, 64, 6, "mixed"), (517, 1601, 4803, 12, 5, "mixed"),
                                            (20000, 1600, 1024, 16, 3, "mixed"), (100, 9000, 300, 200, 3, "single")])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_exact_at_large_sizes(mod, dtype, T, K, N, R, L, kind):
    """Small whole numbers, few of them not zero: every product and sum is a whole number that binary32 holds (and h a sum
    of two bf16 values), so each output is the exact one rounded once."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(T + K)

    def sparse(shape, top, share):
        v = rng.integers(-top, top + 1, shape) * (rng.random(shape) < share)
        return torch.from_numpy(v.astype(np.float32)).to(dt)

    x, a, b = sparse((T, K), 2, 0.5), sparse((L, R, K), 1, 0.1), sparse((L, N, R), 2, 0.3)
    base, dy = sparse((T, N), 9, 1.0), sparse((T, N), 1, 0.02)
    index = index_of(T, L, 1, kind)
    scales = torch.tensor([1.0, 2.0, 0.5, 1.0, 4.0, 2.0, 1.0, 0.5] * L)[:L]
    batch = mod.LoraBatch(torch.from_numpy(index).cuda(), L)
    leaves = [t.cuda().requires_grad_() for t in (base, x, a, b)]
    y = mod.lora_add(*leaves, batch, scales.cuda())
    grads = torch.autograd.grad(y, leaves[1:], dy.cuda())
    # (references in float64 on the GPU, products that are exact there)
    D = lambda t: t.cuda().double()  # noqa: E731
    X, A, B, DY = D(x), D(a), D(b), D(dy)
    want, dx, da, db = D(base), torch.zeros_like(X), torch.zeros_like(A), torch.zeros_like(B)
    top = 0.0
    for i in range(L):
        rows = torch.from_numpy(np.flatnonzero(index == i)).cuda()
        if rows.numel() == 0:
            continue
        s = float(scales[i])
        h = s * torch.matmul(X[rows], A[i].t().contiguous())
        g = s * torch.matmul(DY[rows], B[i])
        want[rows] += torch.matmul(h, B[i].t().contiguous())
        dx[rows] = torch.matmul(g, A[i])
        da[i] = torch.matmul(g.t().contiguous(), X[rows])
        db[i] = torch.matmul(DY[rows].t().contiguous(), h)
        top = max(top, h.abs().max().item(), g.abs().max().item())
        # the condition itself: steps of a half, 2^16 of them in h and g, 2^23 in every sum of magnitudes
        sums = (torch.matmul(h.abs(), B[i].abs().t().contiguous()).max(), torch.matmul(g.abs(), A[i].abs()).max(),
                torch.matmul(g.abs().t().contiguous(), X[rows].abs()).max(),
                torch.matmul(DY[rows].abs().t().contiguous(), h.abs()).max())
        assert max(float(v) for v in sums) < 2.0 ** 22
    assert top < 2.0 ** 15
    for got, ref, what in zip((y, *grads), (want, dx, da, db), ("y", "dx", "dA", "dB")):
        assert torch.equal(got.detach(), ref.to(torch.float32).to(dt)), what


def test_differences(mod):
    """The gradients against differences of the binary64 formula (linear in each argument: exact but for rounding)."""
    from oracle import block
    T, K, N, R, L = 150, 40, 50, 6, 3
    base, x, a, b, dy, scales = tensors(T, K, N, R, L, torch.float32, 9)
    index = index_of(T, L, 2)
    leaves = [t.cuda().requires_grad_() for t in (base, x, a, b)]
    batch = mod.LoraBatch(torch.from_numpy(index).cuda(), L)
    grads = torch.autograd.grad(mod.lora_add(*leaves, batch, scales.cuda()), leaves, dy.cuda())
    for i in range(4):
        v = np64(draw(leaves[i].shape, torch.float32, 60 + i))

        def value(s):
            t = [np64(q) for q in (base, x, a, b)]
            t[i] = t[i] + s * v
            return (block.lora(*t, index, np64(scales))[0] * np64(dy)).sum()

        want = (value(0.5) - value(-0.5))
        got = (np64(grads[i]) * v).sum()
        # a gradient element sums at most T * R terms: (T + K + N + R + 100) 2^-23 of their magnitudes, 5e-5
        assert abs(got - want) <= 5e-5 * (np.abs(np64(grads[i])) * np.abs(v)).sum() + 1e-9 * abs(want)


# ---------------------------------------------------------------- masks and edges

@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masked_tokens_may_hold_anything(mod, dtype):
    """What a token without an adapter holds in x, and in dy, reaches nothing but its own place; NaN in one token stays
    there; unused adapters may hold anything."""
    dt, T, K, N, R, L = DTYPES[dtype], 400, 72, 90, 20, 5
    base, x, a, b, dy, scales = tensors(T, K, N, R, L, dt, 3)
    index = index_of(T, 4, 8)  # (adapter 4 is not used)
    index[::9] = -1
    none = torch.from_numpy(np.flatnonzero(index < 0))
    assert len(none) > 3

    def run(x, dy, a, b, base):
        batch = mod.LoraBatch(torch.from_numpy(index).cuda(), L)
        leaves = [t.cuda().requires_grad_() for t in (base, x, a, b)]
        y = mod.lora_add(*leaves, batch, scales.cuda())
        return (y.detach(), *torch.autograd.grad(y, leaves[1:], dy.cuda()))

    clean = run(x, dy, a, b, base)
    x2, dy2, a2, b2 = x.clone(), dy.clone(), a.clone(), b.clone()
    x2[none[0]], x2[none[1]], dy2[none[2]] = float("nan"), float("inf"), float("-inf")
    a2[4], b2[4] = float("nan"), float("inf")
    got = run(x2, dy2, a2, b2, base)
    assert all(torch.equal(p, q) for p, q in zip(got, clean))
    t = int(np.flatnonzero(index == 2)[0])
    x2[t, 5] = float("nan")
    base2 = base.clone()
    base2[none[0], 0] = float("nan")
    got = run(x2, dy2, a2, b2, base2)
    others = torch.tensor([i for i in range(T) if i not in (t, int(none[0]))]).cuda()
    assert torch.equal(got[0][others], clean[0][others]) and torch.isnan(got[0][t].float()).all()
    assert torch.isnan(got[0][none[0], 0]) and torch.equal(got[1], clean[1])
    for i in (0, 1, 3, 4):
        assert torch.equal(got[2][i], clean[2][i]) and torch.equal(got[3][i], clean[3][i])
    # (a rank that is not a multiple of 16: an infinite x may not meet the padding's zeros)
    x3, big = x.clone(), torch.zeros_like(a)
    x3[t], big[:, :, 0] = 0, 1
    x3[t, 0] = float("inf")
    one = torch.ones_like(b)
    y = run(x3, dy, big, one, base)[0]
    assert torch.equal(y[t], torch.full_like(y[t], float("inf")))


def test_nobody_and_nothing(mod):
    T, K, N, R, L = 70, 40, 50, 4, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 4))
    batch = mod.LoraBatch(torch.full((T,), -1, device="cuda"), L)
    leaves = [t.requires_grad_() for t in (base, x, a, b)]
    y = mod.lora_add(*leaves, batch, scales)
    assert torch.equal(y, base)
    grads = torch.autograd.grad(y, leaves, dy)
    assert torch.equal(grads[0], dy) and not any(g.any() for g in grads[1:])
    for T, K, N in ((0, 40, 50), (5, 0, 50), (5, 40, 0), (0, 0, 0)):
        base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, max(K, 0), N, R, L, torch.float32, 5) if t is not None) \
            if K else (torch.randn(s, device="cuda") for s in ((T, N), (T, K), (L, R, K), (L, N, R), (T, N), (L,)))
        leaves = [t.requires_grad_() for t in (base, x, a, b)]
        batch = mod.LoraBatch(torch.zeros(T, dtype=torch.int32, device="cuda"), L)
        y = mod.lora_add(*leaves, batch)
        assert torch.equal(y, base)
        grads = torch.autograd.grad(y, leaves, dy)
        assert all(g.shape == t.shape for g, t in zip(grads, leaves)) and not any(g.any() for g in grads[1:])


def test_strides_shapes_and_some_gradients(mod, f8lin):
    T, K, N, R, L = 60, 72, 88, 8, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.float16, 6))
    index = torch.from_numpy(index_of(T, L, 3)).cuda()
    batch = mod.LoraBatch(index, L)
    want = mod.lora_add(base, x, a, b, batch, scales)
    wide_x, wide_b = torch.zeros((T, K + 9), device="cuda").half(), torch.zeros((T, N + 3), device="cuda").half()
    wide_x[:, 1:K + 1], wide_b[:, 2:N + 2] = x, base
    sx, sb = wide_x[:, 1:K + 1], wide_b[:, 2:N + 2]
    assert torch.equal(mod.lora_add(sb, sx, a, b, batch, scales), want)
    assert torch.equal(mod.lora_add(base.t().contiguous().t(), x.t().contiguous().t(), a.transpose(1, 2).contiguous()
                                    .transpose(1, 2), b.transpose(1, 2).contiguous().transpose(1, 2), batch, scales), want)
    assert torch.equal(mod.lora_add(base.view(3, 20, N), x.view(3, 20, K), a, b, mod.LoraBatch(index.view(3, 20), L), scales),
                       want.view(3, 20, N))
    # a strided index
    two = torch.stack([index, index + 1], dim=1)[:, 0]
    assert torch.equal(mod.lora_add(base, x, a, b, mod.LoraBatch(two, L), scales), want)
    leaves = [t.clone().requires_grad_() for t in (base, x, a, b)]
    full = torch.autograd.grad(mod.lora_add(*leaves, batch, scales), leaves, dy)
    for keep in ((0,), (1,), (2,), (3,), (1, 3), (2, 3), (0, 1)):
        part = [t.clone().requires_grad_(i in keep) for i, t in enumerate((base, x, a, b))]
        grads = torch.autograd.grad(mod.lora_add(*part, batch, scales), [part[i] for i in keep], dy)
        assert all(torch.equal(g, full[i]) for g, i in zip(grads, keep))
    # strided and expanded gradients; an expanded base and x
    sdy = torch.zeros((T, N + 5), device="cuda").half()
    sdy[:, 3:N + 3] = dy
    again = torch.autograd.grad(mod.lora_add(*leaves, batch, scales), leaves, sdy[:, 3:N + 3])
    assert all(torch.equal(p, q) for p, q in zip(again, full))
    ex = x[:1].detach().clone().requires_grad_()
    y = mod.lora_add(base[:1].expand(T, N), ex.expand(T, K), a, b, batch, scales)
    g, = torch.autograd.grad(y, ex, dy[:1].expand(T, N))
    assert g.shape == (1, K)
    # in place, without a base, and the kept inner products
    plan = batch.plan
    ws = torch.empty(f8lin.lora_forward_workspace_bytes(T, K, N, R, L), dtype=torch.uint8, device="cuda")
    h = torch.full((f8lin.lora_h_elements(T, R),), 7.0, device="cuda")
    y = base.clone()
    f8lin.lora_forward(y, x, a, b, scales, plan, y, h, ws)
    assert torch.equal(y, want)
    zero = torch.empty_like(base)
    f8lin.lora_forward(None, x, a, b, scales, plan, zero, None, ws)
    assert torch.equal(zero, mod.lora_add(torch.zeros_like(base), x, a, b, batch, scales))


def test_a_plan_of_another_batch_writes_nothing(f8lin):
    T, K, N, R, L = 30, 40, 50, 4, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 7))
    for buffer in (torch.zeros(4096, dtype=torch.int32, device="cuda"), None):
        plan = f8lin.LoraPlan(T, L, buffer=buffer)
        if buffer is None:  # a plan of fewer tokens in its place
            small = f8lin.LoraPlan(T - 1, L, buffer=plan.buffer)
            f8lin.lora_plan(torch.zeros(T - 1, dtype=torch.int32, device="cuda"), small)
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        y, dx, da, db = (torch.full_like(t, 5.0) for t in (base, x, a, b))
        h = torch.zeros(f8lin.lora_h_elements(T, R), device="cuda")
        f8lin.lora_forward(base, x, a, b, scales, plan, y, h, ws)
        f8lin.lora_backward(dy, x, a, b, scales, plan, h, dx, da, db, ws)
        assert all(bool((t == 5).all()) for t in (y, dx, da, db))


def test_same_bits_every_run_and_in_any_batch(mod):
    """The same bits on every run; a token's y and dx are those it has alone with its adapter's other tokens."""
    T, K, N, R, L = 3000, 320, 256, 16, 4
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 8))
    index = torch.from_numpy(index_of(T, L, 5)).cuda()
    leaves = [t.requires_grad_() for t in (base, x, a, b)]
    runs = []
    for _ in range(3):
        y = mod.lora_add(*leaves, mod.LoraBatch(index, L), scales)
        runs.append((y, *torch.autograd.grad(y, leaves, dy)))
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


# ---------------------------------------------------------------- refusals

def test_refusals(mod, f8lin):
    T, K, N, R, L = 6, 16, 24, 4, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.float32, 1))
    batch = mod.LoraBatch(torch.zeros(T, dtype=torch.int64, device="cuda"), L)
    bad = [dict(base=base[:5]), dict(base=base[:, :23]), dict(x=x[:5], base=base[:5]), dict(a=a[:2]), dict(a=a[:, :, :15]),
           dict(b=b[:, :, :3]), dict(b=b[:2]), dict(a=a[0]), dict(b=b[0]), dict(scales=scales[:2]),
           dict(scales=scales.double()), dict(scales=scales.clone().requires_grad_()),
           dict(a=torch.zeros((L, 257, K), device="cuda"), b=torch.zeros((L, N, 257), device="cuda"))]
    for kw in bad:
        args = dict(base=base, x=x, a=a, b=b, scales=scales)
        args.update(kw)
        with pytest.raises(ValueError):
            mod.lora_add(args["base"], args["x"], args["a"], args["b"], batch, args["scales"])
    for kw in (dict(a=a.half()), dict(b=b.bfloat16()), dict(base=base.half()), dict(x=x.double(), a=a.double())):
        args = dict(base=base, x=x, a=a, b=b)
        args.update(kw)
        with pytest.raises(TypeError):
            mod.lora_add(args["base"], args["x"], args["a"], args["b"], batch, scales)
    for index in (torch.zeros(T, device="cuda"), torch.zeros(T, dtype=torch.int16, device="cuda")):
        with pytest.raises(TypeError):
            mod.LoraBatch(index, L)
    for n in (0, -1, 2048):
        with pytest.raises(ValueError):
            mod.LoraBatch(torch.zeros(T, dtype=torch.int32, device="cuda"), n)
    with pytest.raises(ValueError):
        batch.update(torch.zeros(T + 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):
        mod.LoraBatch(torch.zeros(T, dtype=torch.int32), L)
    with pytest.raises(NotImplementedError), torch.no_grad(), torch.autograd.forward_ad.dual_level():
        mod.lora_add(base, torch.autograd.forward_ad.make_dual(x, x), a, b, batch)
    leaf = x.clone().requires_grad_()
    g, = torch.autograd.grad((mod.lora_add(base, leaf, a, b, batch) ** 2).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), leaf)
    # a batch changed between forward and backward
    y = mod.lora_add(base, leaf, a, b, batch)
    batch.update(torch.ones(T, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y.sum(), leaf)
    y = torch.empty_like(base)
    with pytest.raises(f8lin.F8linError):
        f8lin.lora_forward(base, x, a, b, scales, batch.plan, y, None, torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- in use

def test_captured_decoding_and_training(mod):
    """Graphs in which the batch is sorted anew from an index that changes between the replays."""
    T, K, N, R, L = 48, 320, 640, 16, 6
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 10))
    index = torch.from_numpy(index_of(T, L, 1, "single")).cuda()
    batch = mod.LoraBatch(index, L)

    @torch.no_grad()
    def decode():
        return mod.lora_add(base, x, a, b, batch.update(index), scales)

    leaves = [t.clone().requires_grad_() for t in (base, x, a, b)]

    def train(leaves, batch):
        y = mod.lora_add(*leaves, batch, scales)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(), train(leaves, batch)
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = decode()
    with torch.cuda.graph(g2):
        out2 = train(leaves, batch.update(index))
    for seed in range(3):
        index.copy_(torch.from_numpy(index_of(T, L, 20 + seed, "single" if seed else "mixed")))
        with torch.no_grad():
            x.copy_(draw((T, K), torch.bfloat16, 30 + seed))
            leaves[1].copy_(x)
        g1.replay()
        g2.replay()
        got = [y1.clone(), *(t.clone() for t in out2)]
        fresh = mod.LoraBatch(index, L)
        want = train([t.detach().clone().requires_grad_() for t in leaves], fresh)
        assert torch.equal(got[0], want[0]) and all(torch.equal(p, q) for p, q in zip(got[1:], want))
        torch.cuda.synchronize()


def test_streams(mod):
    T, K, N, R, L = 500, 640, 320, 16, 4
    ins = []
    for i in range(2):
        t = [q.cuda() for q in tensors(T, K, N, R, L, torch.bfloat16, 40 + i)]
        ins.append((t, torch.from_numpy(index_of(T, L, i)).cuda()))

    def step(t, index):
        leaves = [q.detach().requires_grad_() for q in t[:4]]
        y = mod.lora_add(*leaves, mod.LoraBatch(index, L), t[5])
        return (y.detach(), *torch.autograd.grad(y, leaves, t[4]))

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(step(*ins[i]))
    torch.cuda.synchronize()
    for i in range(2):
        want = step(*ins[i])
        for got in outs[i]:
            assert all(torch.equal(p, q) for p, q in zip(got, want))


class Block(nn.Module):
    def __init__(self, d, hidden, dtype):
        super().__init__()
        self.norm = nn.LayerNorm(d, dtype=torch.float32)
        self.fc1 = nn.Linear(d, hidden, dtype=dtype)
        self.fc2 = nn.Linear(hidden, d, bias=False, dtype=dtype)

    def forward(self, x):
        return x + self.fc2(torch.relu(self.fc1(self.norm(x))))


@pytest.mark.parametrize("kind", ["plain", "fp8", "mxfp4"])
def test_block_with_norm_and_adapters(mod, kind):
    """norm -> projection + adapters, twice, beside each kind of linear: every layer's output and gradients against
    binary64 on what it really saw; only the adapters (and the norms) train."""
    torch.manual_seed(1)
    d, hidden, L, R = 64, 160, 3, 6
    model = nn.Sequential(Block(d, hidden, torch.bfloat16), Block(d, hidden, torch.bfloat16)).cuda()
    if kind == "fp8":
        mod.convert_to_float8_training(model)
    elif kind == "mxfp4":
        mod.convert_to_mxfp4_training(model)
    mod.convert_layer_norm(model)
    mod.convert_to_lora(model, L, R, scale=2.0)
    assert mod.convert_to_lora(model, L, R) is model  # (what has adapters keeps them)
    layers = [m for m in model.modules() if isinstance(m, mod.LoraLinear)]
    assert len(layers) == 4 and not any(isinstance(m.base, mod.LoraLinear) for m in layers)
    assert {n.split(".")[-1] for n, p in model.named_parameters() if p.requires_grad} == {"lora_a", "lora_b", "weight", "bias"}
    assert not any(p.requires_grad for m in layers for p in m.base.parameters())
    x = draw((3, 50, d), torch.bfloat16, 2).cuda()
    index = torch.from_numpy(index_of(150, L, 4)).view(3, 50).cuda()
    with torch.no_grad():
        plain = model(x)
        mod.set_lora_batch(model, mod.LoraBatch(index, L))
        assert torch.equal(model(x), plain)  # fresh adapters add nothing
        for m in layers:
            m.lora_b.normal_(std=0.2)
        assert not torch.equal(model(x), plain)
    seen = {}
    for m in layers:
        m.register_forward_hook(lambda m, i, o: seen.__setitem__(m, [i[0].detach(), o.detach()]))
        m.base.register_forward_hook(lambda m, i, o: seen.__setitem__(m, [o.detach()]))
        m.register_full_backward_hook(lambda m, gi, go: seen[m].append(go[0].detach()))
    leaf = x.clone().requires_grad_()
    (model(leaf).float() ** 2).mean().backward()
    assert leaf.grad is not None and torch.isfinite(leaf.grad.float()).all()
    flat = index.flatten().cpu().numpy()
    for m in layers:
        inp, out, dy = (t.reshape(150, -1) for t in seen[m])
        base = seen[m.base][0].reshape(150, -1)
        args = [np64(t.to(torch.bfloat16)) for t in (base, inp, m.lora_a, m.lora_b)]
        ref, h, d_y, d_h = lora_bounds(*args, flat, np64(m.lora_scales), torch.bfloat16)
        close(out, ref, d_y, "y")
        refs, errs = lora_grad_bounds(np64(dy), *args[1:], flat, np64(m.lora_scales), h, d_h, torch.bfloat16)
        close(m.lora_a.grad, refs[1], errs[1], "dA")
        close(m.lora_b.grad, refs[2], errs[2], "dB")
    state = model.state_dict()
    assert state["0.fc1.lora_a"].shape == (L, R, d) and "0.fc1.base.weight" in state


def test_serving_frozen_weights_with_adapters(mod):
    """Frozen 4-bit weights shared by requests with adapters of their own: a batch of single tokens gives each token what
    it gets alone."""
    torch.manual_seed(2)
    model = nn.Sequential(nn.LayerNorm(96), nn.Linear(96, 200), nn.ReLU(), nn.Linear(200, 72)).cuda().bfloat16()
    mod.convert_layer_norm(mod.convert_to_mxfp4_training(model))
    mod.freeze_mxfp4(mod.convert_to_lora(model, 5, 8))
    assert model[1].base.frozen and model[1].lora_a.dtype == torch.bfloat16
    with torch.no_grad():
        model[1].lora_b.normal_(std=0.2)
        model[3].lora_b.normal_(std=0.2)
        x = draw((7, 96), torch.bfloat16, 3).cuda()
        index = torch.tensor([0, 4, -1, 2, 2, 9, 1], device="cuda")
        mod.set_lora_batch(model, mod.LoraBatch(index, 5))
        y = model(x)
        for t in range(7):
            mod.set_lora_batch(model, mod.LoraBatch(index[t:t + 1], 5) if 0 <= int(index[t]) < 5 else None)
            one = model(x[t:t + 1])
            # (the few-row products sum in another order: within a step of bf16 of the hidden values' effect)
            assert (one - y[t]).abs().max() <= 2.0 ** -6 * y[t].abs().max()
