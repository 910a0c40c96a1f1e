"""The layer norm where its sizes choose other kernels or other loads: very many rows."""
import pytest
import torch

from block_helpers import DTYPES, draw
from test_gpu_layer_norm import f8lin, mod  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_rows_than_a_dimension(mod, dtype):
    """More than 2^22 rows, a head's each: every row as in a small call, dw and db of whole numbers exact."""
    rows, cols, dt = (1 << 22) + 77, 8, DTYPES[dtype]
    x = torch.empty((rows, cols), dtype=dt, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randint(0, 2, (rows, 4), generator=g, device="cuda").repeat(1, 2))
    x[:, 4:] = 1 - x[:, :4]  # four zeros and four ones: xhat is -1 and 1 with eps = 0
    w, b = draw((cols,), dt, 2).cuda().requires_grad_(), draw((cols,), dt, 3).cuda().requires_grad_()
    x.requires_grad_()
    y = mod.layer_norm(x, w, b, eps=0.0)
    dy = torch.zeros((rows, cols), dtype=dt, device="cuda")
    dy[::97] = torch.randint(-1, 2, dy[::97].shape, generator=g, device="cuda").to(dt)
    dy[-5:] = 1
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    xhat = 2 * x.detach().float() - 1
    assert torch.equal(y.detach(), (xhat * w.detach().float() + b.detach().float()).to(dt))
    # (43,000 rows of them: every sum of whole numbers is exact, and rounded once)
    assert torch.equal(dw, (dy.double() * xhat.double()).sum(0).to(dt))
    assert torch.equal(db, dy.double().sum(0).to(dt))
    for at in (slice(0, 9), slice((1 << 21) - 4, (1 << 21) + 4), slice((1 << 22) - 4, rows)):
        part = x.detach()[at].clone().requires_grad_()
        z = mod.layer_norm(part, w, b, eps=0.0)
        assert torch.equal(z, y[at]) and torch.equal(torch.autograd.grad(z, part, dy[at])[0], dx[at])
