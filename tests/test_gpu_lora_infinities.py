"""Infinite values in the adapters' inputs give what the formulas give -- an infinity of the product's sign, NaN where two
of different signs meet or one meets a zero -- and change nothing else's bits."""
import numpy as np
import pytest
import torch

from block_helpers import DTYPES, np64
from oracle import block
from test_gpu_lora import index_of, mod, tensors  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def run(mod, t, index, L):
    leaves = [q.cuda().requires_grad_() for q in t[:4]]
    y = mod.lora_add(*leaves, mod.LoraBatch(torch.from_numpy(index).cuda(), L), t[5].cuda())
    return (y.detach(), *torch.autograd.grad(y, leaves[1:], t[4].cuda()))


def reference(t, index):
    base, x, a, b, dy, scales = (np64(q) for q in t)
    with np.errstate(invalid="ignore"):
        y, h = block.lora(base, x, a, b, index, scales)
        return (y, *block.lora_grads(dy, x, a, b, index, scales, h)[:3])


# what becomes infinite: (tensor, place) in turn; the tokens and adapters are those of the index below
CASES = {
    "base": [(0, (3, 2), -INF)],
    "x": [(1, (0, 1), INF)],
    "x twice": [(1, (0, 1), INF), (1, (2, 0), -INF)],
    "x twice in a token": [(1, (0, 1), INF), (1, (0, 4), -INF)],
    "a": [(2, (0, 1, 3), INF)],
    "b": [(3, (0, 5, 0), -INF)],
    "b twice in a row": [(3, (0, 5, 0), INF), (3, (0, 5, 2), INF)],
    "a and b": [(2, (0, 1, 3), -INF), (3, (0, 5, 2), INF), (3, (1, 0, 0), INF)],
    "dy": [(4, (0, 6), INF)],
    "dy twice": [(4, (0, 6), -INF), (4, (0, 0), -INF), (4, (2, 6), INF)],
    "dy and x": [(4, (0, 6), INF), (1, (2, 1), INF)],
    "nan beside": [(1, (0, 1), INF), (1, (2, 1), NAN), (3, (0, 5, 0), INF)],
}


@pytest.mark.parametrize("T,R", [(1, 4), (50, 3), (50, 16), (700, 20), (90, 64), (90, 100), (1100, 5), (1100, 16), (1200, 24),
                                 (1100, 64), (1100, 130), (32800, 3), (32800, 40)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_infinities(mod, dtype, T, R):
    K, N, L = 40, 70, 3
    index = index_of(T, L, T + R, "single")
    index[:min(T, 4)] = [0, 1, 0, -1][:T]
    t = list(tensors(T, K, N, R, L, DTYPES[dtype], T))
    for name, places in CASES.items():
        places = [p for p in places if p[0] not in (0, 1, 4) or p[1][0] < T]
        bad, clean = [q.clone() for q in t], [q.clone() for q in t]
        for which, at, value in places:
            bad[which][at] = value
            clean[which][at] = 1.0
        got, same, want = run(mod, bad, index, L), run(mod, clean, index, L), reference(bad, index)
        for g, c, w, what in zip(got, same, want, ("y", "dx", "dA", "dB")):
            g = g.cpu()
            w = torch.from_numpy(w)
            finite = torch.isfinite(w)
            assert torch.equal(torch.isnan(g), torch.isnan(w)), (name, what, "nan")
            rest = ~finite & ~torch.isnan(w)
            assert torch.equal(g.double()[rest], w[rest]), (name, what, "inf")
            assert torch.equal(g[finite], c.cpu()[finite]), (name, what, "finite")


@pytest.mark.parametrize("T", [40, 1100])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_beside_small_and_large(mod, dtype, T):
    """An infinite weight beside inner products far below a token's largest; an infinite inner product beside a finite one
    that is large."""
    dt, K, N, R, L = DTYPES[dtype], 4, 64, 8, 1
    index = np.zeros(T, dtype=np.int32)
    base, x = torch.zeros((T, N), dtype=dt), torch.zeros((T, K), dtype=dt)
    a, b = torch.zeros((L, R, K), dtype=dt), torch.zeros((L, N, R), dtype=dt)
    a[0, 0, 0], a[0, 1, 1], a[0, 2, 2] = 256.0, 2.0 ** -12, 1.0
    x[:, 0], x[:, 1] = 256.0, 2.0 ** -12
    b[0, :, 1] = INF
    b[0, :, 0] = 2.0 ** -14
    y = mod.lora_add(base.cuda(), x.cuda(), a.cuda(), b.cuda(), mod.LoraBatch(torch.from_numpy(index).cuda(), L))
    assert bool((y == INF).all())  # 2^16 2^-14 + 2^-24 inf + 0
    # an infinite h of one rank, 2^17 in another (fp16: beyond its largest value), weights of both signs
    x[:, 2] = INF
    a[0, 0, 0], a[0, 1, 1] = 512.0, 0.0
    b[0] = 0.0
    b[0, :, 0], b[0, :, 2] = -2.0 ** -14, 1.0
    got = mod.lora_add(base.cuda(), x.cuda(), a.cuda(), b.cuda(), mod.LoraBatch(torch.from_numpy(index).cuda(), L))
    # (0 times an infinite x is NaN in the other ranks: only with weights of their own)
    ref = reference([base, x, a, b, base, torch.ones(L)], index)[0]
    assert np.isnan(ref).all() and bool(torch.isnan(got).all())
    a[0, :, 2] = 1.0  # every inner product infinite, each of one sign
    a[0, 3, 2] = -1.0
    b[0] = 1.0
    b[0, :, 3] = -2.0 ** -10
    got = mod.lora_add(base.cuda(), x.cuda(), a.cuda(), b.cuda(), mod.LoraBatch(torch.from_numpy(index).cuda(), L))
    assert bool((got == INF).all())
