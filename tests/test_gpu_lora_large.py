"""The adapters where sizes choose other kernels: tiles whose rows several workgroups or one share, every block of ranks
beside them, outer products with waves side by side.  Small whole numbers, few of them not zero: every sum is exact, so
each output is the exact one rounded once."""
import numpy as np
import pytest
import torch

from block_helpers import DTYPES
from test_gpu_lora import f8lin, index_of, mod  # noqa: F401

pytestmark = pytest.mark.gpu


def sparse(rng, shape, top, share, dt):
    v = rng.integers(-top, top + 1, shape).astype(np.float32)
    v *= rng.random(shape, dtype=np.float32) < share
    return torch.from_numpy(v).to(dt).cuda()


def check(mod, T, K, N, R, L, dt, index, shares=(0.5, 0.2, 0.3, 0.02)):
    rng = np.random.default_rng(T + K + R)
    x, a, b = sparse(rng, (T, K), 2, shares[0], dt), sparse(rng, (L, R, K), 1, shares[1], dt), \
        sparse(rng, (L, N, R), 2, shares[2], dt)
    base, dy = sparse(rng, (T, N), 9, 1.0, dt), sparse(rng, (T, N), 1, shares[3], dt)
    scales = torch.tensor([1.0, 2.0, 0.5, 4.0] * L)[:L]
    leaves = [t.requires_grad_() for t in (x, a, b)]
    y = mod.lora_add(base, *leaves, mod.LoraBatch(torch.from_numpy(index).cuda(), L), scales.cuda())
    grads = torch.autograd.grad(y, leaves, dy)
    X, A, B, DY = (t.detach().double() for t in (x, a, b, dy))
    want, dx, da, db = base.double(), torch.zeros_like(X), torch.zeros_like(A), torch.zeros_like(B)
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
        # steps of a half, at most 2^23 of them in any sum of magnitudes
        sums = (torch.matmul(h.abs(), B[i].abs().t().contiguous()).max(), torch.matmul(g.abs(), A[i].abs()).max(),
                torch.matmul(g.abs().t().contiguous(), X[rows].abs()).max(),
                torch.matmul(DY[rows].abs().t().contiguous(), h.abs()).max())
        assert max(float(v) for v in sums) < 2.0 ** 22
    for got, ref, what in zip((y, *grads), (want, dx, da, db), ("y", "dx", "dA", "dB")):
        assert torch.equal(got.detach(), ref.to(torch.float32).to(dt)), what


# 64-row tiles dealt to two workgroups (128 tiles of 64 ranks and more) and to one (512); ranks of every block
@pytest.mark.parametrize("T,K,N", [(9001, 130, 161), (9000, 256, 96), (36000, 65, 200)])
@pytest.mark.parametrize("R", [7, 16, 24, 32, 51, 64, 96, 129, 256])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_tiles(mod, dtype, T, K, N, R):
    check(mod, T, K, N, R, 3, DTYPES[dtype], index_of(T, 3, R))


# 32768 tokens and more: waves of an outer product side by side; fewer: parts of the tokens
@pytest.mark.parametrize("T", [32768, 33001, 32767])
@pytest.mark.parametrize("R", [3, 16, 17, 32, 64, 100, 160])
@pytest.mark.parametrize("K,N", [(129, 700), (1023, 64), (40, 130), (200, 90)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_outer_products(mod, dtype, T, R, K, N):
    check(mod, T, K, N, R, 2, DTYPES[dtype], index_of(T, 2, T + R), (0.05, 0.2, 0.3, 0.02))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_most_tokens(mod, dtype):
    """As many tokens as a plan holds: more tiles than a grid's second dimension."""
    check(mod, 1 << 22, 64, 70, 16, 3, DTYPES[dtype], index_of(1 << 22, 3, 5), (0.5, 0.2, 0.3, 0.0005))


@pytest.mark.parametrize("T", [900, 5000, 33000])
def test_one_gradient_at_a_time(f8lin, mod, T):
    K, N, R, L, dt = 200, 333, 24, 3, torch.bfloat16
    rng = np.random.default_rng(T)
    base, x, dy = (sparse(rng, (T, n), 3, 0.1, dt) for n in (N, K, N))
    a, b = sparse(rng, (L, R, K), 1, 0.2, dt), sparse(rng, (L, N, R), 1, 0.2, dt)
    plan = f8lin.LoraPlan(T, L)
    f8lin.lora_plan(torch.from_numpy(index_of(T, L, 3)).cuda(), plan)
    y, h = torch.empty_like(base), torch.empty(f8lin.lora_h_elements(T, R), device="cuda")
    f8lin.lora_forward(base, x, a, b, None, plan, y, h)
    full = [torch.full_like(t, 5.0) for t in (x, a, b)]
    f8lin.lora_backward(dy, x, a, b, None, plan, h, *full)
    for mask in range(8):
        part = [torch.full_like(t, 5.0) if mask >> k & 1 else None for k, t in enumerate((x, a, b))]
        f8lin.lora_backward(dy, x, a, b, None, plan, h if part[2] is not None else None, *part)
        assert all(p is None or torch.equal(p, f) for p, f in zip(part, full))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_offsets_past_32_bits(mod, dtype):
    """2.4e9 elements of base, y and dy: both gradients of the adapters in whole, every sum of theirs exact."""
    T, K, N, R, L, dt = 40000, 64, 60000, 4, 2, DTYPES[dtype]
    rng = np.random.default_rng(1)
    index = torch.from_numpy(index_of(T, L, 5)).cuda()
    x, a, b = (sparse(rng, s, 2, share, dt).requires_grad_() for s, share in (((T, K), 0.1), ((L, R, K), 0.5), ((L, N, R), 0.3)))
    g = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.empty((T, N), dtype=dt, device="cuda")
    for at in range(0, T, 4000):  # one element in a thousand 1 or -1
        u = torch.rand((4000, N), generator=g, device="cuda")
        dy[at:at + 4000] = ((u < 5e-4).float() - (u > 1 - 5e-4).float()).to(dt)
    base = torch.zeros((T, N), dtype=dt, device="cuda")
    grads = torch.autograd.grad(mod.lora_add(base, x, a, b, mod.LoraBatch(index, L)), (x, a, b), dy)
    del base
    A, B = a.detach().double(), b.detach().double()
    dx, da, db = torch.zeros((T, K), dtype=torch.float64, device="cuda"), torch.zeros_like(A), torch.zeros_like(B)
    for at in range(0, T, 4000):
        d, xs, i = dy[at:at + 4000].double(), x.detach()[at:at + 4000].double(), index[at:at + 4000]
        for k in range(L):
            rows = torch.nonzero(i == k).flatten()
            part, xr = d[rows], xs[rows]
            inner = torch.matmul(part, B[k])
            dx[at + rows] = torch.matmul(inner, A[k])
            da[k] += torch.matmul(inner.t().contiguous(), xr)
            db[k] += torch.matmul(part.t().contiguous(), torch.matmul(xr, A[k].t().contiguous()))
    for got, want, what in zip(grads, (dx, da, db), ("dx", "dA", "dB")):
        assert torch.equal(got, want.float().to(dt)), what
