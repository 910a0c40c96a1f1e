"""Products whose scales differ from block to block, exactly; the quantisation of large calls in each of its forms.

Products: codes are multiples of 1/2 of at most 6.  With scale bytes whose sum, less 254, lies in lo .. hi, a product
is a multiple of 2^(lo - 2) of at most 36 * 2^hi, so a sum of K of them is a whole number of at most K * 144 * 2^(hi -
lo) such units.  Below 2^24 units binary32 holds every partial sum, in whatever order, and the result is exact: a scale
taken from another block, row or place changes it.
"""
import numpy as np
import pytest
import torch

from test_gpu_mxfp4 import DTYPES, GEMMS, MANY, f8lin, mod, mx, np64  # noqa: F401

pytestmark = pytest.mark.gpu

FEW = [(16, 40, 200), (13, 33, 511), (4, 50, 4096), (2, 35, 7000), (1, 96, 14336), (3, 17, 9), (16, 8200, 96), (16, 12300, 100),
       (5, 20001, 64), (17, 4100, 96), (32, 12288, 40), (48, 4800, 1600), (64, 8192, 300), (49, 600, 4100), (20, 600, 8200)]


def operand(f8lin, rows, K, scales, seed):
    """(MXFP4Tensor, values in binary64, on the GPU): any codes, each block's scale byte one of `scales`, and NaN bytes
    behind the last block."""
    gen = torch.Generator("cuda").manual_seed(seed)
    nb = -(-K // 32)
    codes = torch.randint(0, 16, (rows, nb * 32), generator=gen, device="cuda", dtype=torch.uint8)
    codes[:, K:] = 0
    some = torch.tensor(scales, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, -(-nb // 16) * 16), 255, dtype=torch.uint8, device="cuda")
    s[:, :nb] = some[torch.randint(0, len(scales), (rows, nb), generator=gen, device="cuda")]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    v = grid[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3).double())
    v = v * torch.exp2(s[:, :nb].double() - 127).repeat_interleave(32, 1)
    return f8lin.MXFP4Tensor(codes[:, 0::2] | codes[:, 1::2] << 4, s, rows, K), v[:, :K].contiguous()


def check_exact(f8lin, M, N, K, sa, sb):
    lo, hi = min(sa) + min(sb) - 254, max(sa) + max(sb) - 254
    assert K * 144 * 2 ** (hi - lo) < 2 ** 24
    (a, av), (b, bv) = operand(f8lin, M, K, sa, M + K), operand(f8lin, N, K, sb, N + 2 * K)
    want = (av @ bv.t().contiguous()).float()
    c = torch.full((M, N), float("nan"), device="cuda")
    f8lin.mxfp4_gemm([(a, b, c)])
    assert torch.equal(c, want)


@pytest.mark.parametrize("M,N,K", GEMMS + MANY + FEW)
def test_products_with_differing_scales(f8lin, M, N, K):
    """Three neighbouring scales for either operand (two where the contraction is long)."""
    some = (126, 127, 128) if K * 144 * 16 < 2 ** 24 else (127, 128)
    check_exact(f8lin, M, N, K, some, some)


@pytest.mark.parametrize("M,N,K", [(1, 64, 512), (16, 100, 300), (40, 96, 1000), (64, 64, 256), (130, 257, 1311),
                                   (700, 800, 2500), (2100, 2100, 513), (4100, 4100, 200)])
def test_products_with_scales_at_both_ends(f8lin, M, N, K):
    """The smallest scales against the largest: the products are ordinary numbers."""
    check_exact(f8lin, M, N, K, (0, 1), (250, 251, 252, 253, 254))
    check_exact(f8lin, M, N, K, (250, 251, 252, 253, 254), (0, 1))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", [s for s in FEW if s[0] <= 20])
def test_few_rows_of_x_with_differing_scales(f8lin, mod, M, N, K, dtype):
    """X quantised by the call, inside the product or ahead of it: values on the 4-bit grid of their block, whose
    largest is 4 times its scale, so that the codes stand for them exactly."""
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0], device="cuda")
    nb = -(-K // 32)
    x = grid[torch.randint(0, 7, (M, nb, 32), generator=gen, device="cuda")]
    x = x * (1.0 - 2.0 * torch.randint(0, 2, (M, nb, 32), generator=gen, device="cuda"))
    x[:, :, 0] = 4.0
    some = (126, 127, 128) if K * 144 * 16 < 2 ** 24 else (127, 128)
    x = x * torch.exp2(torch.randint(some[0] - 127, 2, (M, nb, 1), generator=gen, device="cuda").float())
    x = x.view(M, nb * 32)[:, :K].to(DTYPES[dtype])
    w, wv = operand(f8lin, N, K, some, N)
    want = x.double() @ wv.t().contiguous()
    y = torch.full((M, N), float("nan"), device="cuda")
    x4 = None if f8lin.mxfp4_forward_fused(M, N, K) else f8lin.new_mxfp4(M, K)
    f8lin.mxfp4_forward(x, None, y, x4, w)
    assert torch.equal(y, want.float())
    assert torch.equal(mod.mxfp4_linear(x, w), want.float().to(DTYPES[dtype]))


def check_in_pieces(f8lin, x, q, qt):
    """q and qt, x's two layouts, against those of x's pieces of 2048 rows, quantised alone."""
    rows, cols = x.shape
    cb = -(-cols // 32)
    for r0 in range(0, rows, 2048):
        n = min(2048, rows - r0)
        p, pt = f8lin.new_mxfp4(n, cols), f8lin.new_mxfp4(cols, n)
        f8lin.mxfp4_quantize(x[r0:r0 + n], p, pt)
        nb = -(-n // 32)
        assert torch.equal(q.codes[r0:r0 + n, :16 * cb], p.codes[:, :16 * cb])
        assert torch.equal(q.scales[r0:r0 + n, :cb], p.scales[:, :cb])
        assert torch.equal(qt.codes[:, r0 // 2:r0 // 2 + 16 * nb], pt.codes[:, :16 * nb])
        assert torch.equal(qt.scales[:, r0 // 32:r0 // 32 + nb], pt.scales[:, :nb])


def normal(shape, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(0.03).to(dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_large_calls(f8lin, mx, dtype, rule):
    """1280 tiles of 256 x 128 and more, with whole and with ragged rows."""
    for rows, cols in ((40960, 1024), (41000, 1030)):
        x = normal((rows, cols), DTYPES[dtype], rows)
        q, qt = f8lin.new_mxfp4(rows, cols), f8lin.new_mxfp4(cols, rows)
        f8lin.mxfp4_quantize(x, q, qt, rule)
        if rule == "floor":
            check_in_pieces(f8lin, x, q, qt)
        assert np.array_equal(np64(q.dequantize(torch.float32)[:300]), mx.rounded(np64(x[:300]), rule))
        assert np.array_equal(np64(qt.dequantize(torch.float32)[:64]), mx.rounded(np64(x[:, :64]).T, rule))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_x_and_weight_in_one_launch(f8lin, dtype):
    """768 tiles of X and 512 of W, both layouts of both; then dY's, with the bias gradient's sums taken on the way."""
    M, N, K = 24576, 16384, 1024
    dt = DTYPES[dtype]
    x, w = normal((M, K), dt, 1), normal((N, K), dt, 2)
    x4, x4t, w4, w4t = (f8lin.new_mxfp4(*s) for s in ((M, K), (K, M), (N, K), (K, N)))
    y = torch.empty((M, N), dtype=dt, device="cuda")
    f8lin.mxfp4_forward(x, w, y, x4, w4, x4t, w4t)
    check_in_pieces(f8lin, x, x4, x4t)
    check_in_pieces(f8lin, w, w4, w4t)
    del y
    M, N = 40960, 1024
    dy = normal((M, N), dt, 3)
    dx, db = torch.empty((M, K), dtype=dt, device="cuda"), torch.empty((N,), device="cuda")
    dy4, dy4t, wt = f8lin.new_mxfp4(M, N), f8lin.new_mxfp4(N, M), f8lin.new_mxfp4(K, N)
    f8lin.mxfp4_quantize(w[:N], None, wt)
    ws = torch.empty(f8lin.mxfp4_dbias_workspace_bytes(M, N) // 4, device="cuda")
    f8lin.mxfp4_backward(dy, None, wt, dx, None, dy4, dy4t, db, ws)
    check_in_pieces(f8lin, dy, dy4, dy4t)
    # an element passes 32 + 2 additions in its tile, tiles / 32 in its group and 31 joining them
    depth = 34 + M // 128 // 32 + 1 + 31
    want, size = dy.double().sum(0), dy.double().abs().sum(0)
    assert (db.double() - want).abs().le(depth * 2.0 ** -24 * 1.01 * size).all()
