"""MXFP4 quantisation, product and linear layer against the binary64 oracle.

Codes, scales and dequantised values are compared bit for bit.  Products: operands hold at most 2 significant bits
each, so products are exact; the K products meet in fp32, and whatever the order each addition is off by at most one
fp32 step (2^-23) of a partial sum that is at most S = sum |a b|, so |error| <= K * 2^-23 * S before the one rounding
to the output type (half a step, eps / 2).  Where every partial sum is a small multiple of 1/4 the result is exact.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def f8lin():
    from float8linear_tensorwise_amax_amd import f8lin
    return f8lin


@pytest.fixture(scope="module")
def mod():
    from float8linear_tensorwise_amax_amd import module
    return module


@pytest.fixture(scope="module")
def mx():
    from oracle import mxfp4
    return mxfp4


def draw(shape, dtype, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * std
    if x.numel() > 64:
        x.view(-1)[::41] *= 50.0
        x.view(-1)[3::97] = 0.0
        x.view(-1)[5::89] = -0.0
    return x.to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def check_mx(mx, q, ref_codes, ref_scales, what):
    """Codes and scales of an MXFP4Tensor equal the oracle's."""
    nb = -(-q.cols // 32)
    codes = mx.unpack(q.codes[:, :16 * nb].cpu().numpy())
    assert np.array_equal(q.scales[:, :nb].cpu().numpy(), ref_scales), f"{what}: scales"
    assert np.array_equal(codes, ref_codes), f"{what}: codes"


def out_half_step(ref, dtype):
    """Half a step of `dtype` at ref (and half its smallest subnormal)."""
    fi = torch.finfo(dtype)
    return np.abs(ref) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def check_product(got, a, b, dtype, bias=None, what=""):
    """got (M, N) against a (M, K) . b (N, K)^T in binary64."""
    ref, s = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        ref, s = ref + bias, s + np.abs(bias)
    tol = (a.shape[1] + 2) * 2.0 ** -23 * s
    tol = tol + out_half_step(np.abs(ref) + tol, dtype)
    err = np.abs(np64(got) - ref)
    assert got.shape == ref.shape
    assert np.all(err <= tol), f"{what}: off by {np.max(err - tol)} over the bound at {np.argmax(err - tol)}"


SIZES = [(1, 1), (1, 32), (1, 4096), (2, 31), (3, 33), (33, 2), (64, 64), (127, 129), (128, 128), (129, 127),
         (257, 96), (31, 1601), (300, 1), (5, 511), (260, 513)]


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(f8lin, mx, rows, cols, dtype, rule):
    x = draw((rows, cols), DTYPES[dtype], rows * 1000 + cols)
    xd = x.cuda()
    for both in (3, 1, 2):
        q = f8lin.new_mxfp4(rows, cols) if both & 1 else None
        qt = f8lin.new_mxfp4(cols, rows) if both & 2 else None
        f8lin.mxfp4_quantize(xd, q, qt, rule)
        if q is not None:
            check_mx(mx, q, *mx.quantize(np64(x), rule), "rows")
            assert np.array_equal(np64(q.dequantize(torch.float32)), mx.rounded(np64(x), rule))
        if qt is not None:
            check_mx(mx, qt, *mx.quantize(np64(x).T, rule), "columns")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_many_tiles(f8lin, mod, mx, dtype):
    """Enough tiles for the taller ones, ragged in both directions; and the column sums a bias gradient takes there."""
    x = draw((4100, 2050), DTYPES[dtype], 7)
    xd = x.cuda()
    q, qt = f8lin.new_mxfp4(4100, 2050), f8lin.new_mxfp4(2050, 4100)
    f8lin.mxfp4_quantize(xd, q, qt)
    check_mx(mx, q, *mx.quantize(np64(x)), "rows")
    check_mx(mx, qt, *mx.quantize(np64(x).T), "columns")
    w = draw((2050, 32), DTYPES[dtype], 8).cuda()
    b = torch.zeros(2050, dtype=DTYPES[dtype], device="cuda", requires_grad=True)
    db, = torch.autograd.grad(mod.mxfp4_linear(draw((4100, 32), DTYPES[dtype], 9).cuda(), w, b), b, xd)
    ref, s = np64(x).sum(0), np.abs(np64(x)).sum(0)
    tol = 4102 * 2.0 ** -23 * s
    assert np.all(np.abs(np64(db) - ref) <= tol + out_half_step(np.abs(ref) + tol, DTYPES[dtype]))


def all_bf16():
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    return x[torch.isfinite(x.float())]


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_every_bf16(f8lin, mx, rule):
    """Every finite bf16 value, next to neighbours of its own size (a block of one binade), of any size (a strided
    block), and below a fixed larger value, so that each meets the top, the middle and the bottom of the grid."""
    x = all_bf16()
    assert x.numel() == 65280
    near = x.view(-1, 32)
    far = x[(torch.arange(65280) * 7919) % 65280].view(-1, 32)
    shifted = near.clone().float()
    for k in range(8):  # the block's maximum 2^k times the largest value there
        shifted[k::8, 0] = shifted[k::8].abs().amax(1) * 2.0 ** k
    shifted = shifted.clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    for name, t in (("near", near), ("far", far), ("below", shifted)):
        q = f8lin.new_mxfp4(*t.shape)
        qt = f8lin.new_mxfp4(t.shape[1], t.shape[0])
        f8lin.mxfp4_quantize(t.cuda(), q, qt, rule)
        check_mx(mx, q, *mx.quantize(np64(t), rule), name)
        check_mx(mx, qt, *mx.quantize(np64(t).T, rule), name + " columns")


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_fp32_borders(f8lin, mx, rule):
    """fp32 values one step on either side of every rounding midpoint and of the saturation and scale borders, at
    exponents from the subnormals to the largest, and all of fp32's own extremes."""
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    rows = []
    for k in (-126, -125, -124, -100, -1, 0, 1, 30, 100, 124):
        base = np.array([m * s for m in (0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9)
                         for s in (1, -1)], dtype=np.float32)
        v = (base.astype(np.float64) * 2.0 ** (k - 2 if k > -100 else k)).astype(np.float32)
        rows += [v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(-np.inf))]
    for top in (6.0, np.nextafter(np.float32(6), np.float32(7)), 7.99, 4.0, np.nextafter(np.float32(4), np.float32(3))):
        v = rows[15].copy()
        v[5] = top
        rows.append(v)
    edge = np.zeros(32, dtype=np.float32)
    edge[:6] = [tiny, -tiny, 3 * tiny, 0.0, -0.0, 5 * tiny]
    rows += [edge, np.full(32, big, np.float32), np.full(32, -0.0, np.float32), np.zeros(32, np.float32)]
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    q, qt = f8lin.new_mxfp4(*x.shape), f8lin.new_mxfp4(x.shape[1], x.shape[0])
    f8lin.mxfp4_quantize(x.cuda(), q, qt, rule)
    check_mx(mx, q, *mx.quantize(np64(x), rule), "rows")
    check_mx(mx, qt, *mx.quantize(np64(x).T, rule), "columns")
    with np.errstate(over="ignore"):  # (4 * 2^126, what the largest values round to, is beyond fp32)
        want = mx.rounded(np64(x), rule).astype(np.float32)
    assert np.array_equal(q.dequantize(torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_nonfinite_blocks(f8lin, mx, dtype):
    """A NaN or an infinity turns its own block, and no other, into NaN."""
    x = draw((70, 130), DTYPES[dtype], 3).float()
    x[0, 5], x[7, 40], x[64, 129], x[69, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    x = x.to(DTYPES[dtype])
    q, qt = f8lin.new_mxfp4(70, 130), f8lin.new_mxfp4(130, 70)
    f8lin.mxfp4_quantize(x.cuda(), q, qt)
    for t, ref in ((q, np64(x)), (qt, np64(x).T)):
        check_mx(mx, t, *mx.quantize(ref), "codes")
        for d in DTYPES.values():
            got, want = np64(t.dequantize(d)), mx.rounded(ref)
            assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(np64(q.dequantize())).sum() == 32 * 3 + 2


def test_quantize_strided_input(f8lin, mx):
    """Rows of a wider buffer, a start that is only element-aligned, and one row and one column of one."""
    for dtype in DTYPES.values():
        base = draw((90, 200), dtype, 11).cuda()
        for x in (base[:, 8:136], base[:, 1:98], base[::2, 3:67], base[4:5, 7:50], base[:, 5:6], base[3:3], base[:, 4:4]):
            q, qt = f8lin.new_mxfp4(*x.shape), f8lin.new_mxfp4(x.shape[1], x.shape[0])
            f8lin.mxfp4_quantize(x, q, qt)
            if x.numel():
                check_mx(mx, q, *mx.quantize(np64(x)), "rows")
                check_mx(mx, qt, *mx.quantize(np64(x).T), "columns")


def test_dequantize_every_code_and_scale(f8lin, mx):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))  # each row: every code twice, at one scale
    scales = np.arange(256, dtype=np.uint8)[:, None]
    pad = np.zeros((256, 16), np.uint8)
    pad[:, :1] = scales
    q = f8lin.MXFP4Tensor(torch.from_numpy(mx.pack(codes)).cuda(), torch.from_numpy(pad).cuda(), 256, 32)
    ref = mx.values(codes, scales, 32)
    for dtype in DTYPES.values():
        with np.errstate(over="ignore"):
            want = torch.from_numpy(ref).to(torch.float64).to(dtype)
        got = q.dequantize(dtype).cpu()
        assert torch.equal(torch.nan_to_num(got.float(), nan=7e37), torch.nan_to_num(want.float(), nan=7e37)), dtype


def random_mx(f8lin, mx, rows, cols, seed, same_scale=False, extra=0):
    """(MXFP4Tensor, its values): uniform codes; scales around one (or all one); rows `extra` bytes longer than needed,
    and everything behind the last block filled with NaN scales and random codes."""
    rng = np.random.default_rng(seed)
    nb = -(-cols // 32)
    codes = rng.integers(0, 16, (rows, nb * 32)).astype(np.uint8)
    codes[:, cols:] = 0
    scales = np.full((rows, nb), 127, np.uint8) if same_scale else rng.integers(115, 128, (rows, nb)).astype(np.uint8)
    buf = rng.integers(0, 256, (rows, 16 * nb + extra)).astype(np.uint8)
    buf[:, :16 * nb] = mx.pack(codes)
    sbuf = np.full((rows, -(-nb // 16) * 16 + extra), 255, np.uint8)
    sbuf[:, :nb] = scales
    return (f8lin.MXFP4Tensor(torch.from_numpy(buf).cuda(), torch.from_numpy(sbuf).cuda(), rows, cols),
            mx.values(codes, scales, cols))


GEMMS = [(1, 1, 1), (1, 17, 33), (1, 4096, 256), (3, 100, 640), (16, 16, 128), (17, 65, 1000), (33, 130, 96),
         (64, 64, 64), (65, 257, 1600), (100, 1, 300), (128, 128, 1024), (129, 255, 1056), (200, 300, 31),
         (256, 256, 2048), (257, 513, 4097), (300, 512, 1311), (512, 256, 1279), (700, 800, 5000), (40, 2000, 4096)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_exact(f8lin, mx, M, N, K):
    """All scales one: every sum is a multiple of 1/4 below 2^22, so fp32 holds it exactly."""
    assert K * 36 < 2 ** 22
    a, av = random_mx(f8lin, mx, M, K, M + K, same_scale=True, extra=16)
    b, bv = random_mx(f8lin, mx, N, K, N + 2 * K, same_scale=True, extra=48)
    c = torch.full((M, N), float("nan"), device="cuda")
    f8lin.mxfp4_gemm([(a, b, c)])
    assert np.array_equal(np64(c), av @ bv.T)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_scales_and_bias(f8lin, mx, M, N, K, dtype):
    a, av = random_mx(f8lin, mx, M, K, M + K)
    b, bv = random_mx(f8lin, mx, N, K, N + 2 * K)
    for bias_dtype in (None, torch.float32, DTYPES[dtype]):
        bias = None if bias_dtype is None else draw((N,), bias_dtype, 5).cuda()
        c = torch.full((M, N), float("nan"), device="cuda", dtype=DTYPES[dtype])
        f8lin.mxfp4_gemm([(a, b, c, bias)])
        check_product(c, av, bv, DTYPES[dtype], None if bias is None else np64(bias), f"{bias_dtype}")


# sizes that take each tile and several of them per workgroup, with odd and even numbers of 256-wide K blocks
MANY = [(4100, 4100, 1000), (4100, 4100, 200), (4096, 4096, 768), (5000, 3900, 513), (2100, 2100, 1300), (1700, 1500, 2050),
        (70, 20000, 600), (20000, 100, 257), (130, 5000, 1000)]


@pytest.mark.parametrize("M,N,K", MANY)
def test_gemm_many_tiles(f8lin, mx, M, N, K):
    """Exact sums over many tiles, in the three output types (bf16 and fp16: rounded once from the exact sum)."""
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    grid = torch.tensor(mx.GRID, device="cuda")

    def operand(rows):
        nb = -(-K // 32)
        codes = torch.randint(0, 16, (rows, nb * 32), generator=gen, device="cuda", dtype=torch.uint8)
        codes[:, K:] = 0
        scales = torch.full((rows, -(-nb // 16) * 16), 255, dtype=torch.uint8, device="cuda")
        scales[:, :nb] = 127
        v = grid[(codes & 7).long()] * (1.0 - 2.0 * (codes >> 3))
        return f8lin.MXFP4Tensor(codes[:, 0::2] | codes[:, 1::2] << 4, scales, rows, K), v[:, :K]

    (a, av), (b, bv) = operand(M), operand(N)
    want = av @ bv.t().contiguous()
    bias = torch.randint(-8, 8, (N,), generator=gen, device="cuda").float()
    for dtype in DTYPES.values():
        c = torch.full((M, N), float("nan"), device="cuda", dtype=dtype)
        f8lin.mxfp4_gemm([(a, b, c)])
        assert torch.equal(c, want.to(dtype))
        f8lin.mxfp4_gemm([(a, b, c, bias)])
        assert torch.equal(c, (want + bias.double()).to(dtype))


def test_gemm_long_contraction_same_bits(f8lin, mx):
    """Few tiles over a long contraction, and twice the same bits."""
    for M, N, K in ((256, 256, 8192), (300, 200, 12000), (1000, 130, 9001), (16, 512, 16384), (1600, 1600, 8200)):
        a, av = random_mx(f8lin, mx, M, K, 1)
        b, bv = random_mx(f8lin, mx, N, K, 2)
        outs = []
        for _ in range(2):
            c = torch.full((M, N), float("nan"), device="cuda")
            f8lin.mxfp4_gemm([(a, b, c)])
            outs.append(c)
        assert torch.equal(outs[0], outs[1])
        check_product(outs[0], av, bv, torch.float32, what=f"{M} {N} {K}")


def test_gemm_pair_equals_singles(f8lin, mx):
    """Two products in one call give what each gives alone."""
    for shapes in (((300, 200, 1000), (200, 1000, 300)), ((1024, 512, 2048), (512, 2048, 1024)), ((5, 70, 4096), (600, 600, 64)),
                   ((0, 70, 32), (65, 64, 0))):
        items, refs = [], []
        for i, (M, N, K) in enumerate(shapes):
            a, av = random_mx(f8lin, mx, M, K, 10 + i)
            b, bv = random_mx(f8lin, mx, N, K, 20 + i)
            c, alone = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
            items.append((a, b, c))
            refs.append(alone)
            f8lin.mxfp4_gemm([(a, b, alone)])
            check_product(alone, av, bv, torch.float32)
        f8lin.mxfp4_gemm(items)
        for (_, _, c), r in zip(items, refs):
            assert torch.equal(c, r)


def test_gemm_nan_scale_reaches_its_rows_only(f8lin, mx):
    for M, N, K in ((70, 90, 300), (300, 300, 4096), (2, 90, 1000)):
        a, av = random_mx(f8lin, mx, M, K, 1)
        b, bv = random_mx(f8lin, mx, N, K, 2)
        a.scales[1, 4] = 255
        b.scales[40, (K - 1) // 32] = 255
        c = torch.zeros((M, N), device="cuda")
        f8lin.mxfp4_gemm([(a, b, c)])
        want = np.zeros((M, N), bool)
        want[1, :] = True
        want[:, 40] = True
        assert np.array_equal(np.isnan(np64(c)), want)


def test_gemm_leaves_what_is_around_c(f8lin, mx):
    for M, N, K in ((33, 47, 200), (300, 301, 2000), (1, 19, 64)):
        a, _ = random_mx(f8lin, mx, M, K, 1)
        b, _ = random_mx(f8lin, mx, N, K, 2)
        for dtype in DTYPES.values():
            buf = torch.full((M * N + 64,), 7.0, device="cuda", dtype=dtype)
            f8lin.mxfp4_gemm([(a, b, buf[32:32 + M * N].view(M, N))])
            assert torch.all(buf[:32] == 7) and torch.all(buf[32 + M * N:] == 7)


LAYERS = [(1, 48, 64, "bf16", True), (3, 4096, 512, "bf16", False), (7, 33, 65, "fp32", True), (16, 256, 4096, "fp16", True),
          (33, 100, 129, "fp16", True), (64, 128, 300, "bf16", True), (257, 130, 250, "bf16", True),
          (300, 513, 1000, "fp32", True), (1, 1, 1, "fp32", True), (130, 1, 31, "fp16", False)]


@pytest.mark.parametrize("M,N,K,dtype,has_bias", LAYERS)
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_linear_training(mod, mx, M, N, K, dtype, has_bias, rule):
    """Y, dX, dW, db of the layer against the formulas in binary64."""
    dt = DTYPES[dtype]
    x, w, dy = draw((M, K), dt, 1), draw((N, K), dt, 2, K ** -0.5), draw((M, N), dt, 3, 0.03)
    b = draw((N,), dt, 4) if has_bias else None
    xs, ws_ = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    bs = None if b is None else b.cuda().requires_grad_()
    y = mod.mxfp4_linear(xs, ws_, bs, rule)
    y.backward(dy.cuda())
    X, W, DY = np64(x), np64(w), np64(dy)
    check_product(y, mx.rounded(X, rule), mx.rounded(W, rule), dt, None if b is None else np64(b), "Y")
    check_product(xs.grad, mx.rounded(DY, rule), mx.rounded(W.T, rule), dt, what="dX")
    check_product(ws_.grad, mx.rounded(DY.T, rule), mx.rounded(X.T, rule), dt, what="dW")
    if b is not None:
        ref, s = DY.sum(0), np.abs(DY).sum(0)
        tol = (M + 2) * 2.0 ** -23 * s
        assert np.all(np.abs(np64(bs.grad) - ref) <= tol + out_half_step(np.abs(ref) + tol, dt))


@pytest.mark.parametrize("M,N,K,dtype,has_bias", LAYERS)
def test_linear_serving(f8lin, mod, mx, M, N, K, dtype, has_bias):
    """A weight quantised before gives what the training forward gives; rows do not depend on their batch."""
    dt = DTYPES[dtype]
    x, w = draw((M, K), dt, 1).cuda(), draw((N, K), dt, 2, K ** -0.5).cuda()
    b = draw((N,), dt, 4).cuda() if has_bias else None
    q = f8lin.new_mxfp4(N, K)
    f8lin.mxfp4_quantize(w, q)
    y = mod.mxfp4_linear(x, q, b)
    check_product(y, mx.rounded(np64(x)), mx.rounded(np64(w)), dt, None if b is None else np64(b), "Y")
    wide = torch.zeros((M, K + 5), dtype=dt, device="cuda")
    wide[:, 3:K + 3] = x
    assert torch.equal(mod.mxfp4_linear(wide[:, 3:K + 3], q, b), y)
    assert torch.equal(mod.mxfp4_linear(x.view(1, M, 1, K), q, b), y.view(1, M, 1, N))


def test_linear_nonfinite_tokens(f8lin, mod):
    """A token with a NaN, in every size class of the product, leaves the other tokens alone."""
    w = draw((96, 256), torch.bfloat16, 2, 1 / 16).cuda()
    q = f8lin.new_mxfp4(96, 256)
    f8lin.mxfp4_quantize(w, q)
    for M in (1, 2, 20, 65, 300):
        x = draw((M, 256), torch.bfloat16, 1).cuda()
        y = mod.mxfp4_linear(x, q)
        x[M - 1, 200] = float("inf")
        z = mod.mxfp4_linear(x, q)
        assert torch.isnan(z[M - 1]).all() and torch.equal(z[:M - 1], y[:M - 1])


def test_gradient_against_differences(mod):
    """Inputs on the 4-bit grid in every direction (all blocks hold a 4, all values on the grid below it), so the layer
    is exactly linear in a step from one grid value to another: the differences are the gradients, exactly."""
    M, N, K = 64, 32, 96
    gen = torch.Generator().manual_seed(0)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0])

    def on_grid(r, c):
        t = grid[torch.randint(0, 6, (r, c), generator=gen)] * (1 - 2 * torch.randint(0, 2, (r, c), generator=gen))
        i = torch.arange(max(r, c))
        for shift in range(0, max(r, c), 16):  # a 4 in every block of every row and column
            t[i % r, (i + shift) % c] = 4.0
        return t.cuda()

    x, w, dy = on_grid(M, K), on_grid(N, K), on_grid(M, N)
    b = torch.zeros(N, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = mod.mxfp4_linear(*leaves)
    assert torch.equal(y.detach().double().cpu(), x.double().cpu() @ w.double().cpu().T)
    dx, dw, db = torch.autograd.grad(y, leaves, dy)

    def loss(x, w, b):
        return float((mod.mxfp4_linear(x, w, b).double() * dy.double()).sum())

    base = loss(x, w, b)
    rng = np.random.default_rng(0)
    for t, g, args in ((x, dx, 0), (w, dw, 1)):
        for _ in range(25):
            i, j = int(rng.integers(t.shape[0])), int(rng.integers(t.shape[1]))
            if float(t[i, j]) == 4.0:
                continue
            new = 1.0 if float(t[i, j]) != 1.0 else 2.0
            moved = t.clone()
            moved[i, j] = new
            call = [x, w, b]
            call[args] = moved
            with torch.no_grad():
                diff = loss(*call) - base
            assert diff == float(g[i, j]) * (new - float(t[i, j]))
    for j in (0, 7, N - 1):
        moved = b.clone()
        moved[j] = 2.0
        assert loss(x, w, moved) - base == 2.0 * float(db[j])


def test_linear_partial_gradients_and_empty(f8lin, mod, mx):
    """Only the gradients that are asked for; no tokens; a sum's broadcast gradient (stride 0)."""
    x, w, b = draw((40, 96), torch.bfloat16, 1).cuda(), draw((50, 96), torch.bfloat16, 2, 0.1).cuda(), \
        draw((50,), torch.bfloat16, 3).cuda()
    dy = draw((40, 50), torch.bfloat16, 4).cuda()
    full = [t.clone().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(mod.mxfp4_linear(*full), full, dy)
    for mask in range(1, 8):
        leaves = [t.clone().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate((x, w, b))]
        ask = [t for t in leaves if t.requires_grad]
        got = torch.autograd.grad(mod.mxfp4_linear(*leaves), ask, dy)
        for g, r in zip(got, [r for i, r in enumerate(want) if mask >> i & 1]):
            assert torch.equal(g, r)
    got = torch.autograd.grad(mod.mxfp4_linear(*full).sum(), full)
    again = torch.autograd.grad(mod.mxfp4_linear(*full), full, torch.ones_like(dy))
    assert all(torch.equal(g, r) for g, r in zip(got, again))
    empty = [t.clone().requires_grad_() for t in (x[:0], w, b)]
    y = mod.mxfp4_linear(*empty)
    gx, gw, gb = torch.autograd.grad(y, empty, torch.zeros_like(y))
    assert y.shape == (0, 50) and gx.shape == (0, 96) and not gw.any() and not gb.any()
    q = f8lin.new_mxfp4(50, 96)
    f8lin.mxfp4_quantize(w, q)
    assert mod.mxfp4_linear(x[:0], q).shape == (0, 50)
    assert mod.mxfp4_linear(x.view(2, 20, 96)[:, :0], q).shape == (2, 0, 50)


def test_refusals(f8lin, mod):
    x = torch.zeros((4, 64), device="cuda")
    q = f8lin.new_mxfp4(4, 64)
    with pytest.raises(TypeError):
        f8lin.mxfp4_quantize(x.double(), q)
    with pytest.raises(ValueError):
        f8lin.mxfp4_quantize(x.t(), f8lin.new_mxfp4(64, 4))
    with pytest.raises(ValueError):
        f8lin.mxfp4_quantize(x, f8lin.new_mxfp4(4, 32))
    with pytest.raises(KeyError):
        f8lin.mxfp4_quantize(x, q, rule="nearest")
    with pytest.raises(f8lin.F8linError):
        f8lin.mxfp4_quantize(x, None)
    with pytest.raises(ValueError):
        f8lin.MXFP4Tensor(q.codes, q.scales, 4, 96)
    with pytest.raises(f8lin.F8linError):  # a scale row stride that is no multiple of 16
        f8lin.mxfp4_dequantize(f8lin.MXFP4Tensor(q.codes, torch.zeros((4, 17), dtype=torch.uint8, device="cuda"), 4, 64), x)
    with pytest.raises(RuntimeError):
        mod.mxfp4_linear(x.cpu(), q)
    with pytest.raises(ValueError):
        mod.mxfp4_linear(x[:, :32], q)
    with pytest.raises(RuntimeError):
        mod.mxfp4_linear(x.clone().requires_grad_(), q)
    with pytest.raises(ValueError):
        f8lin.mxfp4_gemm([(q, q, torch.zeros((4, 5), device="cuda"))])
    with pytest.raises(ValueError):
        f8lin.mxfp4_gemm([(q, q, torch.zeros((4, 8), device="cuda")[:, ::2])])
