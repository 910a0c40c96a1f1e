"""The layer norm and the adapters at their limits: offsets past 32 bits, many rows, every rank's tail in tiles of 16 and
of 64 rows, in place with columns that are no whole blocks, streams that are given."""
import numpy as np
import pytest
import torch

from block_helpers import DTYPES, close, draw, lora_bounds, lora_grad_bounds, norm_bounds, np64
from test_gpu_lora import check, f8lin, index_of, mod, tensors  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [1, 2, 3, 4, 7, 16, 18, 24, 31, 32, 33, 40, 63, 64, 66, 80, 129, 200, 255])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ranks_in_large_tiles(mod, dtype, rank):
    """More than 1024 tokens: 64-row tiles; columns of one block, of several and a tail, and of less than one."""
    for T, K, N, L in ((1100, 100, 150, 2), (1030, 39, 321, 3), (1025, 200, 61, 2)):
        check(mod, T, K, N, rank, L, DTYPES[dtype], index_of(T, L, rank), seed=rank)


@pytest.mark.parametrize("rank", [2, 4, 9, 16, 30, 40, 100])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ranks_in_small_tiles(mod, dtype, rank):
    check(mod, 90, 129, 4500, rank, 20, DTYPES[dtype], index_of(90, 20, rank, "single"), seed=rank)
    check(mod, 33, 7, 63, rank, 2, DTYPES[dtype], index_of(33, 2, rank), seed=rank)


@pytest.mark.parametrize("T,N", [(40, 64), (40, 65), (40, 127), (300, 4803), (1100, 100), (1100, 319), (1100, 1), (40, 50)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_in_place(f8lin, dtype, T, N):
    """y in base's own memory: the same bits as beside it, also where the last columns are read with their neighbours."""
    K, L = 72, 3
    for R in (8, 40, 70):
        base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, DTYPES[dtype], R))
        plan = f8lin.LoraPlan(T, L)
        f8lin.lora_plan(torch.from_numpy(index_of(T, L, R)).cuda(), plan)
        y, z = torch.empty_like(base), base.clone()
        f8lin.lora_forward(base, x, a, b, scales, plan, y)
        f8lin.lora_forward(z, x, a, b, scales, plan, z)
        assert torch.equal(y, z)


def test_layer_norm_past_32_bits(mod, f8lin):
    rows, cols = 70000, 32768  # 2.3e9 elements
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    row = draw((1, cols), torch.bfloat16, 1, 1.0, 0.2).cuda()
    scale = torch.linspace(0.5, 2, rows, device="cuda").to(torch.bfloat16)
    torch.mul(row, scale[:, None], out=x)
    w, b = draw((cols,), torch.float32, 2).cuda(), draw((cols,), torch.float32, 3).cuda()
    y = torch.empty_like(x)
    stats = torch.empty((2, rows), device="cuda")
    f8lin.layer_norm_forward(x, y, w, b, stats=stats)
    picked = torch.tensor([0, 1, 65535, 65536, 65537, rows - 2, rows - 1], device="cuda")
    want = torch.empty((7, cols), dtype=torch.bfloat16, device="cuda")
    st = torch.empty((2, 7), device="cuda")
    few = x[picked].contiguous()
    f8lin.layer_norm_forward(few, want, w, b, stats=st)
    assert torch.equal(y[picked], want) and torch.equal(stats[:, picked], st)
    n = norm_bounds(np64(few), np64(w), np64(b), 1e-5, 7, cols)
    close(want, n["y"], n["d_y"], "y")
    dx = torch.empty_like(x)
    dw, ws = torch.empty(cols, device="cuda"), torch.empty(f8lin.layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8,
                                                           device="cuda")
    f8lin.layer_norm_backward(y, x, w, stats, dx, dw, None, ws)
    dwant = torch.empty_like(few)
    f8lin.layer_norm_backward(want, few, w, st, dwant)
    assert torch.equal(dx[picked], dwant)
    # dw of some columns from the rows' own statistics: two roundings an xhat, one a product, and at most `rows` in a sum
    for c in (0, 1, 16384, cols - 1):
        terms = y[:, c].double() * ((x[:, c].double() - stats[0].double()) * stats[1].double())
        assert abs(float(dw[c]) - float(terms.sum())) <= (rows + 4) * 2.0 ** -24 * float(terms.abs().sum())


def test_layer_norm_many_rows(mod):
    """More rows than one launch takes."""
    rows, cols = (1 << 21) + 5, 12
    x = draw((rows, cols), torch.float32, 1).cuda()
    y = mod.layer_norm(x)
    assert torch.equal(y[-9:], mod.layer_norm(x[-9:])) and torch.equal(y[:9], mod.layer_norm(x[:9]))
    assert torch.equal(y[(1 << 21) - 4:(1 << 21) + 4], mod.layer_norm(x[(1 << 21) - 4:(1 << 21) + 4]))


def test_strides_past_32_bits(mod, f8lin):
    rows, ld, cols = 2200, 1 << 20, 96
    store = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")  # 2.3e9 elements
    x = store[:, 5:5 + cols]
    x.copy_(draw((rows, cols), torch.bfloat16, 1))
    dense = x.contiguous()
    assert torch.equal(mod.layer_norm(x), mod.layer_norm(dense))
    base, _, a, b, dy, scales = (t.cuda() for t in tensors(rows, cols, 80, 8, 2, torch.bfloat16, 2))
    batch = mod.LoraBatch(torch.from_numpy(index_of(rows, 2, 1)).cuda(), 2)
    outs = []
    for v in (x, dense):
        leaves = [t.detach().requires_grad_() for t in (v, a, b)]
        y = mod.lora_add(base, *leaves, batch, scales)
        outs.append((y, *torch.autograd.grad(y, leaves, dy)))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_lora_past_32_bits(mod):
    T, K, N, R, L = 40000, 64, 60000, 4, 2  # 2.4e9 elements of base, y and dy
    x, a, b = draw((T, K), torch.bfloat16, 1).cuda(), draw((L, R, K), torch.bfloat16, 2, 0.1).cuda(), \
        draw((L, N, R), torch.bfloat16, 3).cuda()
    index = torch.from_numpy(index_of(T, L, 5)).cuda()
    base = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    torch.mul(draw((1, N), torch.bfloat16, 4).cuda(), torch.linspace(-1, 1, T, device="cuda").bfloat16()[:, None], out=base)
    leaves = [t.requires_grad_() for t in (x, a, b)]
    y = mod.lora_add(base, *leaves, mod.LoraBatch(index, L))
    tail = torch.arange(T - 40, T, device="cuda")
    args = [np64(t[tail]) for t in (base, x)] + [np64(a), np64(b)]
    ref, h, d_y, _ = lora_bounds(*args, index[tail].cpu().numpy(), np.ones(L), torch.bfloat16)
    close(y[tail], ref, d_y, "y")
    dx, da, db = torch.autograd.grad(y, leaves, base)
    for i in range(L):  # dx of one token in 64 bits; dB of some columns over all tokens
        t = int(torch.nonzero(index == i).flatten()[-1])
        want = (base[t].double() @ b[i].double()) @ a[i].double()
        # N terms in the inner product, its 2^-17 as a pair, R terms after it; bf16 by half a step
        mag = (base[t].double().abs() @ b[i].double().abs()) @ a[i].double().abs()
        assert ((dx[t].double() - want).abs() <= mag * ((N + 24) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * 2.0 ** -8).all()
        rows = torch.nonzero(index == i).flatten()
        inner = torch.matmul(x[rows].double(), a[i].double().t().contiguous())
        cols = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
        part = base[rows][:, cols].double()
        want = torch.matmul(part.t().contiguous(), inner)
        mag = torch.matmul(part.abs().t().contiguous(), torch.matmul(x[rows].double().abs(), a[i].double().abs().t().contiguous()))
        assert ((db[i][cols].double() - want).abs() <= mag * (len(rows) * 2.0 ** -23 + 2.0 ** -16) + want.abs() * 2.0 ** -8).all()


def test_given_streams(f8lin):
    """Every entry point on a stream that is not the current one, by object and by handle."""
    T, K, N, R, L = 500, 96, 130, 8, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 3))
    index = torch.from_numpy(index_of(T, L, 3)).cuda()
    w = draw((K,), torch.bfloat16, 5).cuda()
    torch.cuda.synchronize()

    def run(stream):
        plan = f8lin.LoraPlan(T, L)
        f8lin.lora_plan(index, plan, stream)
        y, dx, da, db = (torch.empty_like(t) for t in (base, x, a, b))
        h = torch.empty(f8lin.lora_h_elements(T, R), device="cuda")
        f8lin.lora_forward(base, x, a, b, scales, plan, y, h, stream=stream)
        f8lin.lora_backward(dy, x, a, b, scales, plan, h, dx, da, db, stream=stream)
        n, stats, g, dw = torch.empty_like(x), torch.empty((2, T), device="cuda"), torch.empty_like(x), torch.empty_like(w)
        f8lin.layer_norm_forward(x, n, w, stats=stats, stream=stream)
        ws = torch.empty(f8lin.layer_norm_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        f8lin.layer_norm_backward(n, x, w, stats, g, dw, None, ws, stream=stream)
        torch.cuda.synchronize()
        return y, dx, da, db, n, g, dw

    want = run(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        assert all(torch.equal(p, q) for p, q in zip(run(stream), want))


def test_overlapping_calls_share_nothing(mod):
    """Two batches in flight at once on two streams, each call with scratch of its own, forward and backward; a batch
    updated on the stream that reads it."""
    T, K, N, R, L = 1500, 320, 256, 16, 4
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, torch.bfloat16, 6))
    indices = [torch.from_numpy(index_of(T, L, s)).cuda() for s in range(4)]
    want = []
    for i in indices:
        leaves = [t.detach().requires_grad_() for t in (x, a, b)]
        y = mod.lora_add(base, *leaves, mod.LoraBatch(i, L), scales)
        want.append((y.detach(), *torch.autograd.grad(y, leaves, dy)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in range(2):
        with torch.cuda.stream(streams[s]):
            batch = mod.LoraBatch(indices[s], L)
            for i in (s, 2 + s, s):
                batch.update(indices[i])
                leaves = [t.detach().requires_grad_() for t in (x, a, b)]
                y = mod.lora_add(base, *leaves, batch, scales)
                got[s].append((i, (y.detach(), *torch.autograd.grad(y, leaves, dy))))
    torch.cuda.synchronize()
    for i, outs in got[0] + got[1]:
        assert all(torch.equal(p, q) for p, q in zip(outs, want[i]))


def test_subnormal_fp16(mod):
    """fp16 data in the subnormal range (small gradients) are not taken as zeros, neither in x and dy nor in the weights."""
    T, K, N, R, L = 1100, 64, 128, 16, 2
    index = index_of(T, L, 1)
    base = torch.zeros((T, N), dtype=torch.float16)
    x = (draw((T, K), torch.float32, 1) * 2.0 ** -18).half()
    dy = (draw((T, N), torch.float32, 2) * 2.0 ** -20).half()
    a, b = draw((L, R, K), torch.float32, 3).half() * 64, draw((L, N, R), torch.float32, 4).half() * 64
    assert float((x.abs() < 2.0 ** -14).float().mean()) > 0.9 and x.any()
    for small in (False, True):
        if small:
            x, a = draw((T, K), torch.float32, 1).half(), (a.float() * 2.0 ** -24).half()
        for t in (T, 90):
            i = index[:t]
            leaves = [q.cuda().requires_grad_() for q in (base[:t], x[:t], a, b)]
            y = mod.lora_add(*leaves, mod.LoraBatch(torch.from_numpy(i).cuda(), L))
            dx, da, db = torch.autograd.grad(y, leaves[1:], dy[:t].cuda())
            args = [np64(q) for q in (base[:t], x[:t], a, b)]
            ref, h, d_y, d_h = lora_bounds(*args, i, np.ones(L), torch.float16)
            close(y, ref, d_y, "y")
            refs, errs = lora_grad_bounds(np64(dy[:t]), *args[1:], i, np.ones(L), h, d_h, torch.float16)
            for got, r, e in zip((dx, da, db), refs, errs):
                close(got, r, e, "gradient")
    rows = (draw((40, 300), torch.float32, 5) * 2.0 ** -20).half()
    n = norm_bounds(np64(rows), None, None, 0.0, 40, 300)
    close(mod.layer_norm(rows.cuda(), eps=0.0), n["y"], n["d_y"], "norm")


def test_inference_mode_and_cast_modules(mod):
    """A batch made and used in inference mode; a module cast to bf16 after its conversion keeps working."""
    lin = torch.nn.Sequential(torch.nn.LayerNorm(48), torch.nn.Linear(48, 80)).cuda()
    mod.convert_to_lora(mod.convert_layer_norm(lin), 3, 4, scale=1.5)
    lin.bfloat16()
    x = draw((20, 48), torch.bfloat16, 1).cuda()
    index = torch.from_numpy(index_of(20, 3, 2, "single")).cuda()
    with torch.no_grad():
        lin[1].lora_b.normal_()
    with torch.inference_mode():
        mod.set_lora_batch(lin, mod.LoraBatch(index, 3))
        y = lin(x)
        lin[1].batch.update(index)
        assert torch.equal(lin(x), y)
    mod.set_lora_batch(lin, mod.LoraBatch(index, 3))
    z = lin(x)
    assert torch.equal(z.detach(), y) and z.dtype == torch.bfloat16
    z.float().sum().backward()
    assert lin[1].lora_a.grad is not None and lin[0].weight.grad is not None
