"""What the adapters' inner products H = s x A^T and G = s dy B keep on their way into the next product: all of their
binary32 bits.  Whole numbers of 20 bits in steps of 2^-14 whose sums cancel, so that an output shows the last ones."""
import numpy as np
import pytest
import torch

from block_helpers import DTYPES, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mod():
    from float8linear_tensorwise_amax_amd import module
    return module


def digits(rng, shape):
    """Weights of three digits: along the last axis 1, 2^-7 and 2^-14 with a sign, thrice in a row of zeros."""
    w = np.zeros(shape)
    flat = w.reshape(-1, shape[-1])
    for row in flat:
        at = rng.choice(shape[-1], 3, replace=False)
        row[at] = rng.choice([-1.0, 1.0], 3) * [1.0, 2.0 ** -7, 2.0 ** -14]
    return w


def pairs(rng, shape, share):
    """Per column of a (rows, ...) matrix: a few rows with +1 and as many with -1."""
    w = np.zeros(shape)
    flat = w.reshape(shape[0], -1)
    for c in range(flat.shape[1]):
        at = rng.choice(shape[0], min(shape[0] // 2 * 2, share), replace=False)
        flat[at, c] = np.tile([1.0, -1.0], len(at) // 2)
    return w


# single tokens in 16-row tiles; 64-row tiles; each block of ranks: 16, 32, 64 and more; waves side by side in the outer
# products (32768 tokens)
@pytest.mark.parametrize("T,L", [(40, 30), (900, 2), (2100, 3), (33000, 2)])
@pytest.mark.parametrize("R", [2, 12, 16, 20, 32, 41, 64, 100, 200])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_all_bits(mod, dtype, T, L, R):
    dt, rng = DTYPES[dtype], np.random.default_rng(T + R)
    K, N = 70, 90
    index = np.sort(rng.integers(0, L, T)) if T > 1000 else rng.integers(-1, L, T)
    rows = [np.flatnonzero(index == i) for i in range(L)]
    batch = mod.LoraBatch(torch.from_numpy(index).cuda(), L)
    put = lambda v: torch.from_numpy(v).to(dt).cuda()  # noqa: E731  (exact in every type)

    # forward: h of 20 bits; y is what h . B leaves of base, dB the differences of a few tokens' h
    x, a = rng.integers(-63, 64, (T, K)).astype(float), digits(rng, (L, R, K))
    b = np.moveaxis(pairs(rng, (R, L * N), 2).reshape(R, L, N), 0, -1).copy()
    dy = np.zeros((T, N))
    h, add = np.zeros((T, R)), np.zeros((T, N))
    for i, at in enumerate(rows):
        h[at] = x[at] @ a[i].T
        add[at] = h[at] @ b[i].T
        if len(at) > 1:
            dy[at] = pairs(rng, (len(at), N), 8)
    base = np64(torch.from_numpy(-add).to(dt))
    assert np.abs(h).max() < 2.0 ** 6.1 and np.all(h * 2.0 ** 14 == np.round(h * 2.0 ** 14))  # (8 of them: 2^24 steps)
    leaves = [put(t).requires_grad_() for t in (x, a, b)]
    y = mod.lora_add(put(base), *leaves, batch)
    want = torch.from_numpy(base + add).to(dt)
    assert torch.equal(y.detach().cpu(), want), "y"
    db = torch.autograd.grad(y, leaves[2], put(dy))[0]
    ref = np.stack([dy[at].T @ h[at] for at in rows])
    assert torch.equal(db.cpu(), torch.from_numpy(ref).to(dt)), "dB"

    # backward: g of 20 bits; dx the differences of a token's g, dA those of a few tokens'
    dy = rng.integers(-63, 64, (T, N)).astype(float)
    b = np.moveaxis(digits(rng, (L, R, N)), 1, 2).copy()
    a = np.moveaxis(pairs(rng, (R, L * K), 2).reshape(R, L, K), 0, 1).copy()
    x = np.zeros((T, K))
    g, dx = np.zeros((T, R)), np.zeros((T, K))
    for i, at in enumerate(rows):
        g[at] = dy[at] @ b[i]
        dx[at] = g[at] @ a[i]
        if len(at) > 1:
            x[at] = pairs(rng, (len(at), K), 8)
    assert np.abs(g).max() < 2.0 ** 6.1
    leaves = [put(t).requires_grad_() for t in (x, a, b)]
    got = torch.autograd.grad(mod.lora_add(put(np.zeros((T, N))), *leaves, batch), leaves[:2], put(dy))
    assert torch.equal(got[0].cpu(), torch.from_numpy(dx).to(dt)), "dx"
    ref = np.stack([g[at].T @ x[at] for at in rows])
    assert torch.equal(got[1].cpu(), torch.from_numpy(ref).to(dt)), "dA"
