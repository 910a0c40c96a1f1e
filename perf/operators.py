"""Workloads of the microscaled 4-bit (MXFP4) operators and of gradient clipping, each with a plain form.

MXFP4: 32 consecutive values along a product's contraction share one e8m0 scale 2^(e - 127); each value is an e2m1
code (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).  With m the block's largest magnitude, the "floor" rule takes
e - 127 = floor(log2 m) - 2 and the "ceil" rule the smallest e - 127 with m <= 6 * 2^(e - 127); codes are rounded to
nearest even and saturate at 6.  Codes are packed two a byte (the even element in the low half), 16 bytes a block;
rows of scales are padded to 16 bytes.

Operators:
  quantize  a tensor to 4 bits along its rows, or along its rows and its columns, given back as the values it stands for
  linear    Y = X W^T + b with W held in 4 bits and X quantised on the way (serving)
  train     Y, dX, dW, db of the layer whose three products run in 4 bits (X, W and dY quantised along each contraction)
  clip      the global norm of a list of gradients, and the gradients scaled to at most max_norm
"""
import math

import numpy as np
import torch

own = False  # True: run() makes the framework's calls; False: the plain form

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's activation on its way into a 4-bit product: latency only
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "bf16", "both": False,
         "rule": "floor"},
        # odd sizes in both directions (last blocks of 1 and 13 values), both layouts, the other scale rule
        {"name": "quantize_odd_fp16", "op": "quantize", "rows": 1805, "cols": 1601, "dtype": "fp16", "both": True,
         "rule": "ceil"},
        # the largest activation of the repository's workloads, both layouts, as a training step quantises it
        {"name": "quantize_large", "op": "quantize", "rows": 65536, "cols": 4096, "dtype": "bf16", "both": True,
         "rule": "floor"},
        # decoding one token through the gated MLP's input projection: bound by reading the weights
        {"name": "linear_token", "op": "linear", "m": 1, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False,
         "rule": "floor"},
        # a ragged decoding batch through the GPT block's qkv projection (K = 1600 is 6.25 tiles), with its bias
        {"name": "linear_batch_fp16", "op": "linear", "m": 51, "n": 4800, "k": 1600, "dtype": "fp16", "bias": True,
         "rule": "floor"},
        # a prompt of 8192 tokens through the same projection: bound by the matrix cores
        {"name": "linear_prompt", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False,
         "rule": "floor"},
        # a training step of a few hundred tokens: few tiles, launches count
        {"name": "train_256", "op": "train", "m": 256, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False,
         "rule": "floor"},
        # odd tokens and features in 32 bits with a bias
        {"name": "train_odd_fp32", "op": "train", "m": 1021, "n": 1601, "k": 2055, "dtype": "fp32", "bias": True,
         "rule": "ceil"},
        # the largest single linear of the repository's workloads
        {"name": "train_65536", "op": "train", "m": 65536, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False,
         "rule": "floor"},
        # the gradients of one small normalised projection: latency only; the largest magnitude is the norm
        {"name": "clip_small_inf", "op": "clip", "sizes": "4096,1600,1600,33,1", "dtype": "fp32", "out": "fp32",
         "norm": math.inf, "share": 0.5},
        # a GPT-1.5B block's weights and biases (qkv, out, fc1, fc2)
        {"name": "clip_gpt_block", "op": "clip",
         "sizes": "7680000,4800,2560000,1600,10240000,6400,10240000,1600", "dtype": "bf16", "out": "bf16",
         "norm": 2.0, "share": 0.25},
        # four Llama-3-8B layers' linears, 32-bit clipped gradients out of 16-bit ones
        {"name": "clip_llama_layers", "op": "clip",
         "sizes": ",".join(["16777216,4194304,4194304,16777216,58720256,58720256,58720256"] * 4), "dtype": "bf16",
         "out": "fp32", "norm": 2.0, "share": 0.1},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "train", "clip"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    rule = rng.choice(("floor", "floor", "ceil"))
    bias = rng.random() < 0.5
    if op == "quantize":
        cols = _log_int(rng, 32, 16384)
        rows = _log_int(rng, 1, min(65536, 2 ** 27 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "both": rng.random() < 0.6, "rule": rule}
    if op == "linear":
        k, n = _log_int(rng, 256, 14336), _log_int(rng, 256, 16384)
        m = _log_int(rng, 1, min(8192, 2 ** 38 // (k * n)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "rule": rule}
    if op == "train":
        k, n = _log_int(rng, 256, 6400), _log_int(rng, 256, 6400)
        m = _log_int(rng, 64, min(65536, 2 ** 38 // (k * n)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "rule": rule}
    count = rng.randint(1, 32)
    sizes = [_log_int(rng, 1, 2 ** 25) for _ in range(count)]
    return {"op": op, "sizes": ",".join(map(str, sizes)), "dtype": dtype, "out": rng.choice((dtype, "fp32")),
            "norm": rng.choice((2.0, 2.0, 1.0, math.inf)), "share": rng.choice((0.03, 0.3, 0.7, 3.0))}


def work(case):
    op, b = case["op"], _BYTES[case["dtype"]]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * b * (3 if case["both"] else 2), "flops": n * (2 if case["both"] else 1)}
    if op == "clip":
        n = sum(map(int, case["sizes"].split(",")))
        return {"bytes": n * (b + _BYTES[case["out"]]), "flops": 3 * n}
    m, n, k = case["m"], case["n"], case["k"]
    bias = n * b if case["bias"] else 0
    if op == "linear":
        return {"bytes": m * k * b + n * k * 17 // 32 + m * n * b + bias, "flops": 2 * m * n * k}
    return {"bytes": 2 * b * (m * k + n * k + m * n) + 2 * bias, "flops": 6 * m * n * k}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _activation(gen, rows, cols, dtype):
    """N(0, 1) with one element in a thousand 20 times as large, and some all-zero rows (padding tokens)."""
    x = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    x.mul_(torch.where(torch.rand((rows, cols), generator=gen, device="cuda") < 1e-3, 20.0, 1.0))
    if rows > 8:
        x[rows // 2] = 0
    return x.to(dtype)


def prepare(case, seed):
    gen = _generator(seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    if op == "quantize":
        return {"case": case, "x": _activation(gen, case["rows"], case["cols"], dtype)}
    if op == "clip":
        sizes = list(map(int, case["sizes"].split(",")))
        total = sum(sizes)
        flat = _normal(gen, (total,), 1e-2, dtype)
        grads = [g.clone() for g in flat.split(sizes)]
        # max_norm as a share of the norm these draws are expected to have (above 1: nothing is clipped)
        expect = {2.0: 1e-2 * math.sqrt(total), 1.0: 1e-2 * math.sqrt(2 / math.pi) * total}.get(
            case["norm"], 1e-2 * math.sqrt(2 * math.log(total + 2)))
        return {"case": case, "grads": grads, "max_norm": case["share"] * expect}
    m, n, k = case["m"], case["n"], case["k"]
    x = _activation(gen, m, k, dtype)
    w = _normal(gen, (n, k), k ** -0.5, dtype)
    bias = _normal(gen, (n,), 0.1, dtype) if case["bias"] else None
    if op == "linear":
        codes, scales = _packed(w, case["rule"])
        return {"case": case, "x": x, "codes": codes, "scales": scales, "bias": bias}
    dy = _normal(gen, (m, n), 1e-3 ** 0.5, dtype)
    leaves = [t.requires_grad_() for t in (x, w, bias) if t is not None]
    return {"case": case, "x": x, "w": w, "bias": bias, "dy": dy, "leaves": leaves}


# ---------------------------------------------------------------- plain form

def _blocks(x):
    """x (rows, cols) in 32 bits, padded with zeros to whole blocks: (rows, blocks, 32)."""
    x = x.float()
    pad = -x.shape[1] % 32
    if pad:
        x = torch.cat([x, x.new_zeros((x.shape[0], pad))], dim=1)
    return x.reshape(x.shape[0], -1, 32)


def _quantised(x, rule):
    """(e2m1 values (rows, blocks, 32), e8m0 exponent bytes (rows, blocks, 1)) of x (rows, cols)."""
    b = _blocks(x)
    m = b.abs().amax(dim=2, keepdim=True)
    bits = m.view(torch.int32)
    e = (bits >> 23) - 2
    if rule == "ceil":
        e = e + ((bits & 0x7FFFFF) > 0x400000)
    e = e.clamp(min=0)
    a = (b * _pow2(127 - e)).clamp(-6, 6)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    return torch.round(a / step) * step, e


def _pow2(e):
    """2^e exactly, for whole -127 <= e <= 127 (put together from its bits)."""
    return torch.where(e < -126, 0x400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _rounded(x, rule):
    """x (rows, cols) as its 4-bit form's values, in 32 bits."""
    v, e = _quantised(x, rule)
    return (v * _pow2(e - 127)).flatten(1)[:, :x.shape[1]]


def _packed(x, rule):
    """(codes (rows, 16 * blocks), scales (rows, blocks padded to 16)), both uint8."""
    v, e = _quantised(x, rule)
    a = v.abs()
    code = (torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
            + 8 * torch.signbit(v).to(torch.uint8))
    codes = (code[:, :, 0::2] | (code[:, :, 1::2] << 4)).flatten(1).contiguous()
    nb = e.shape[1]
    scales = torch.zeros((x.shape[0], -(-nb // 16) * 16), dtype=torch.uint8, device=x.device)
    scales[:, :nb] = e[:, :, 0].to(torch.uint8)
    return codes, scales


def _unpacked(codes, scales, cols):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], dim=2).view(codes.shape[0], -1, 32)
    e = scales[:, :v.shape[1]].int()
    return (v * _pow2(e - 127).unsqueeze(2)).flatten(1)[:, :cols]


def _columns(x, rule):
    """x as the values of its form quantised along the columns, in x's own layout."""
    return _rounded(x.t(), rule).t()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(op, case, state)
    if op == "quantize":
        x, rule = state["x"], case["rule"]
        rows = _rounded(x, rule).to(x.dtype)
        return (rows, _rounded(x.t(), rule).to(x.dtype)) if case["both"] else (rows,)
    if op == "clip":
        grads, p = state["grads"], case["norm"]
        if p == math.inf:
            norm = torch.stack([g.abs().max().float() for g in grads]).max()
        elif p == 1.0:
            norm = torch.stack([g.double().abs().sum() for g in grads]).sum()
        else:
            norm = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
        norm = norm.float()
        factor = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        return norm, [(g.float() * factor).to(_DTYPES[case["out"]]) for g in grads]
    rule = case["rule"]
    if op == "linear":
        x = state["x"]
        y = _rounded(x, rule) @ _unpacked(state["codes"], state["scales"], case["k"]).t()
        if state["bias"] is not None:
            y = y + state["bias"].float()
        return y.to(x.dtype)
    with torch.no_grad():
        x, w, dy, bias = state["x"], state["w"], state["dy"], state["bias"]
        y = _rounded(x, rule) @ _rounded(w, rule).t()
        if bias is not None:
            y = y + bias.float()
        dx = _rounded(dy, rule) @ _columns(w, rule)
        dw = _rounded(dy.t(), rule) @ _columns(x, rule)
        out = [y.to(x.dtype), dx.to(x.dtype), dw.to(w.dtype)]
        return out + [dy.sum(0, dtype=torch.float32).to(bias.dtype)] if bias is not None else out


def _own(op, case, state):
    from float8linear_tensorwise_amax_amd import f8lin, module
    if op == "quantize":
        x = state["x"]
        q = f8lin.new_mxfp4(case["rows"], case["cols"], x.device)
        qt = f8lin.new_mxfp4(case["cols"], case["rows"], x.device) if case["both"] else None
        f8lin.mxfp4_quantize(x, q, qt, case["rule"])
        return tuple(t.dequantize(x.dtype) for t in ((q, qt) if case["both"] else (q,)))
    if op == "clip":
        norm, clipped = module.clip_grads(state["grads"], state["max_norm"], case["norm"], _DTYPES[case["out"]])
        return norm, clipped
    if op == "linear":
        w = f8lin.MXFP4Tensor(state["codes"], state["scales"], case["n"], case["k"])
        return module.mxfp4_linear(state["x"], w, state["bias"], case["rule"])
    y = module.mxfp4_linear(state["x"], state["w"], state["bias"], case["rule"])
    return [y.detach(), *torch.autograd.grad(y, state["leaves"], state["dy"])]


# ---------------------------------------------------------------- 64 bits

_EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # where e2m1 rounding changes value; ties go up at odd places
_UP = (0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0)


def _values64(x, rule):
    """x (rows, cols) through 4 bits, straight from the definition in 64 bits."""
    x = x.detach().double()
    rows, cols = x.shape
    out = torch.zeros((rows, (cols + 31) // 32 * 32), dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    b = out.view(rows, -1, 32)
    m = b.abs().max(dim=2, keepdim=True).values
    mant, expo = torch.frexp(torch.where(m > 0, m, 1.0))  # m = mant * 2^expo, 0.5 <= mant < 1
    e = (expo - 1 - 2).double()
    if rule == "ceil":
        e = e + (mant > 0.75)
    scale = torch.exp2(torch.clamp(e, min=-127.0))
    a = b.abs() / scale
    v = torch.zeros_like(a)
    for i, (edge, up) in enumerate(zip(_EDGES, _UP)):
        v += up * ((a >= edge) if i % 2 else (a > edge))
    return (torch.sign(b) * v * scale).view(rows, -1)[:, :cols]


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "quantize":
        x, rule = s["x"], case["rule"]
        return (_values64(x, rule), _values64(x.t(), rule)) if case["both"] else (_values64(x, rule),)
    if op == "clip":
        p = case["norm"]
        parts = [float(torch.linalg.vector_norm(g.double().flatten(), ord=p)) for g in s["grads"]]
        norm = float(np.linalg.norm(np.array(parts, dtype=np.float64), ord=p))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        return torch.tensor(norm, dtype=torch.float64), [g.double() * factor for g in s["grads"]]
    rule = case["rule"]
    if op == "linear":
        nib = torch.stack([s["codes"] % 16, s["codes"] // 16], dim=2).flatten(1).long()
        size = torch.cat([torch.zeros(1), torch.cumsum(torch.tensor(_UP), 0)]).double().to(nib.device)
        w = torch.where(nib >= 8, -1.0, 1.0).double() * size[nib % 8]
        two = torch.exp2(s["scales"].double() - 127).repeat_interleave(32, dim=1)
        w = (w * two[:, :w.shape[1]])[:, :case["k"]]
        y = torch.matmul(_values64(s["x"], rule), w.t().contiguous())
        return y if s["bias"] is None else y + s["bias"].detach().double()
    x, w, dy = s["x"], s["w"], s["dy"]
    y = torch.matmul(_values64(x, rule), _values64(w, rule).t().contiguous())
    if s["bias"] is not None:
        y = y + s["bias"].detach().double()
    out = [y, torch.matmul(_values64(dy, rule), _values64(w.t(), rule).t().contiguous()),
           torch.matmul(_values64(dy.t(), rule), _values64(x.t(), rule).t().contiguous())]
    return out + [dy.double().sum(0)] if s["bias"] is not None else out
