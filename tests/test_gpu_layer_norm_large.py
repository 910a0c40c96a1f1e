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


# widths of every entry of the kernels' tables (a wave a row of one, two and four chunks, 256, 512 and 1024 threads), an
# even and an odd one each, with so many rows that the data goes past the caches: more than 256 MB read and written
@pytest.mark.parametrize("cols", [5, 12, 301, 512, 777, 1024, 1601, 2048, 2501, 4096, 4099, 8192, 8195, 16384, 12289])
@pytest.mark.parametrize("types", ["bf16", "fp16", "fp32", "fp32 to bf16"])
def test_past_the_caches(f8lin, cols, types):
    dt, out = DTYPES[types.split()[0]], DTYPES[types.split()[-1]]
    es = dt.itemsize + out.itemsize
    rows = (256 << 20) // (es * cols) + 77
    g = torch.Generator(device="cuda").manual_seed(cols)

    def normal(shape, to):
        t = torch.empty(shape, dtype=to, device="cuda")
        return t.normal_(generator=g)

    for stride in (cols, cols + 3) if types == "bf16" else (cols,):
        x = normal((rows, stride), dt)[:, stride - cols:]
        dy, w, b = normal((rows, cols), out), normal((cols,), torch.float32), normal((cols,), out)
        guard = torch.full((16,), 7.0, dtype=out, device="cuda")
        store = torch.empty(rows * cols + 16, dtype=out, device="cuda")
        store[-16:] = guard
        y, stats, amax = store[:-16].view(rows, cols), torch.empty((2, rows), device="cuda"), torch.empty(1, device="cuda")
        f8lin.layer_norm_forward(x, y, w, b, 1e-5, stats, amax)
        assert torch.equal(store[-16:], guard) and float(amax) == float(y.abs().max())
        dx, dw, db = torch.empty((rows, cols), dtype=dt, device="cuda"), torch.empty_like(w), torch.empty_like(b)
        ws = torch.empty(f8lin.layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        f8lin.layer_norm_backward(dy, x, w, stats, dx, dw, db, ws)
        # rows of all places, as in a small call, whose kernels are held to binary64 elsewhere
        picked = torch.cat([torch.arange(5), torch.randint(5, rows - 5, (40,), generator=torch.Generator().manual_seed(1)),
                            torch.arange(rows - 5, rows)]).cuda()
        few, st = x[picked].contiguous(), torch.empty((2, len(picked)), device="cuda")
        want, dwant = torch.empty((len(picked), cols), dtype=out, device="cuda"), torch.empty_like(few)
        f8lin.layer_norm_forward(few, want, w, b, 1e-5, st)
        f8lin.layer_norm_backward(dy[picked], few, w, st, dwant)
        assert torch.equal(y[picked], want) and torch.equal(stats[:, picked], st) and torch.equal(dx[picked], dwant)
        # dw and db of some columns: two roundings an xhat, one a product, at most `rows` in a sum; then dw's own type
        for c in {0, 1, cols // 2, cols - 1}:
            d = dy[:, c].double()
            terms = d * ((x[:, c].double() - stats[0].double()) * stats[1].double())
            assert abs(float(dw[c]) - float(terms.sum())) <= (rows + 4) * 2.0 ** -24 * float(terms.abs().sum())
            err = (rows + 1) * 2.0 ** -24 * float(d.abs().sum())
            assert abs(float(db[c]) - float(d.sum())) <= err + torch.finfo(out).eps / 2 * (abs(float(d.sum())) + err)
