"""Workloads of the layer norm and of the low-rank adapters beside a shared projection, each with a plain form.

Layer norm of a row x of n values, with weight w and bias b (either may be missing):
    mean = sum(x) / n,  rstd = 1 / sqrt(sum((x - mean)^2) / n + eps),  xhat = (x - mean) * rstd
    y = xhat * w + b
    backward, with g = dy * w:  dx = rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n)
                                dw = sum over rows of dy * xhat,  db = sum over rows of dy

Low-rank adapters: a batch of T tokens belongs to requests that each use one of L adapters, or none.  Beside the shared
projection's output `base` (T, N), whatever made it, a token t of adapter i gets
    y[t] = base[t] + s_i * (x[t] . A_i^T) . B_i^T     A (L, R, K), B (L, N, R), s (L)
    backward:  G[t] = s_i * dy[t] . B_i,  dx[t] = G[t] . A_i,  dA_i = sum over its tokens of G[t]^T x[t],
               dB_i = sum over its tokens of dy[t]^T (s_i * x[t] . A_i^T);  base's gradient is dy itself
and a token without an adapter gets base[t], and a dx of zero.

Operators:
  norm        y
  norm_train  y, dx, dw, db
  lora        y (serving)
  lora_train  y, dx, dA, dB
"""
import math

import torch

own = False  # True: run() makes the framework's calls; False: the plain form

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-5


# ---------------------------------------------------------------- cases

def _text(lengths):
    return ",".join(map(str, lengths))


def listed():
    return [
        # one token in front of its projection: latency only
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "params": "bf16", "bias": True},
        # odd sizes (rows are not whole 16-byte vectors), 32-bit parameters beside 16-bit data, no bias
        {"name": "norm_odd_fp16", "op": "norm", "rows": 1805, "cols": 1601, "dtype": "fp16", "params": "fp32",
         "bias": False},
        # the largest activation of the repository's workloads: bound by memory
        {"name": "norm_65536", "op": "norm", "rows": 65536, "cols": 4096, "dtype": "bf16", "params": "bf16",
         "bias": True},
        # a training step of a few hundred tokens: launches and the parameters' gradients count
        {"name": "norm_train_256", "op": "norm_train", "rows": 256, "cols": 4096, "dtype": "bf16", "params": "bf16",
         "bias": True},
        # odd sizes in 32 bits
        {"name": "norm_train_odd_fp32", "op": "norm_train", "rows": 1021, "cols": 2055, "dtype": "fp32",
         "params": "fp32", "bias": True},
        # a GPT-1.5B block's norm at its training batch, 32-bit parameters
        {"name": "norm_train_gpt", "op": "norm_train", "rows": 12288, "cols": 1600, "dtype": "bf16", "params": "fp32",
         "bias": True},
        # one token of one request beside a 4096 x 4096 projection: latency only
        {"name": "lora_token", "op": "lora", "lengths": "1", "k": 4096, "n": 4096, "rank": 16, "adapters": 8,
         "dtype": "bf16"},
        # a decoding batch, a request a token, most of them with an adapter of their own, beside the gated MLP's input
        # projection: bound by reading the adapters
        {"name": "lora_decode_64", "op": "lora", "lengths": _text([1] * 64), "k": 4096, "n": 14336, "rank": 16,
         "adapters": 64, "dtype": "bf16"},
        # prompts and decoding tokens in one batch, odd sizes and an odd rank
        {"name": "lora_mixed_fp16", "op": "lora", "lengths": _text([1, 1, 517, 1, 1, 33, 1, 129, 1, 1, 2, 1, 260]),
         "k": 1601, "n": 4803, "rank": 12, "adapters": 5, "dtype": "fp16"},
        # 8192 tokens of prompts beside the same wide projection, at a large rank
        {"name": "lora_prompt", "op": "lora", "lengths": _text([1500, 700, 1, 2300, 90, 1100, 1, 333, 1290, 877]),
         "k": 4096, "n": 14336, "rank": 64, "adapters": 6, "dtype": "bf16"},
        # a few sequences of two adapters in 32 bits, odd sizes
        {"name": "lora_train_odd_fp32", "op": "lora_train", "lengths": _text([301, 255, 465]), "k": 1601, "n": 2055,
         "rank": 20, "adapters": 2, "dtype": "fp32"},
        # four adapters trained side by side at the largest batch of the repository's workloads
        {"name": "lora_train_65536", "op": "lora_train", "lengths": _text([8192] * 7 + [8191]), "k": 4096, "n": 4096,
         "rank": 16, "adapters": 4, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_train", "lora", "lora_train"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op.startswith("norm"):
        cols = _log_int(rng, 32, 16384)
        rows = _log_int(rng, 1, min(65536, 2 ** 27 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "params": rng.choice((dtype, "fp32")),
                "bias": rng.random() < 0.7}
    train = op == "lora_train"
    k, n = _log_int(rng, 256, 14336), _log_int(rng, 256, 14336)
    rank = rng.choice((4, 8, 16, 16, 32, 64, _log_int(rng, 1, 128)))
    adapters = _log_int(rng, 1, 8 if train else 64)
    most = min(32768, int(4e9) // ((k + n) * rank), 2 ** 27 // (k + n))
    if not train and rng.random() < 0.4:  # decoding
        lengths = [1] * _log_int(rng, 1, 128)
    else:  # sequences, prompts, or both
        count = rng.randint(1, 12)
        lengths = [max(1, min(_log_int(rng, 1, 8192), most // count)) for _ in range(count)]
    return {"op": op, "lengths": _text(lengths), "k": k, "n": n, "rank": rank, "adapters": adapters, "dtype": dtype}


def _requests(case):
    """[(first token, end, adapter)]; every eighth request has no adapter (-1)."""
    out, at = [], 0
    for i, length in enumerate(map(int, case["lengths"].split(","))):
        out.append((at, at + length, -1 if i % 8 == 7 else i % case["adapters"]))
        at += length
    return out


def work(case):
    b = _BYTES[case["dtype"]]
    if case["op"].startswith("norm"):
        rows, cols, p = case["rows"], case["cols"], _BYTES[case["params"]]
        params = cols * p * (2 if case["bias"] else 1)
        if case["op"] == "norm":
            return {"bytes": 2 * rows * cols * b + params, "flops": 7 * rows * cols}
        return {"bytes": 4 * rows * cols * b + 2 * params, "flops": 20 * rows * cols}
    requests = _requests(case)
    k, n, r = case["k"], case["n"], case["rank"]
    tokens = requests[-1][1]
    adapted = sum(end - at for at, end, i in requests if i >= 0)
    used = len({i for _, _, i in requests if i >= 0}) * r * (k + n)
    if case["op"] == "lora":
        return {"bytes": (adapted * k + 2 * tokens * n + used) * b, "flops": 2 * adapted * r * (k + n)}
    return {"bytes": (adapted * k + tokens * k + 3 * tokens * n + used + case["adapters"] * r * (k + n)) * b,
            "flops": 6 * adapted * r * (k + n)}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _activation(gen, rows, cols, dtype):
    """N(0, 1) with one element in a thousand 20 times as large, and an all-zero row (a padding token)."""
    x = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    x.mul_(torch.where(torch.rand((rows, cols), generator=gen, device="cuda") < 1e-3, 20.0, 1.0))
    if rows > 8:
        x[rows // 2] = 0
    return x.to(dtype)


def prepare(case, seed):
    gen = _generator(seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    if op.startswith("norm"):
        rows, cols, params = case["rows"], case["cols"], _DTYPES[case["params"]]
        x = _activation(gen, rows, cols, torch.float32)
        # a residual stream: columns of differing size, around a mean that is not zero
        x = (x * torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda")) + 0.3).to(dtype)
        w = (1 + _normal(gen, (cols,), 0.1, torch.float32)).to(params)
        bias = _normal(gen, (cols,), 0.1, params) if case["bias"] else None
        if op == "norm":
            return {"case": case, "x": x, "w": w, "bias": bias}
        dy = _normal(gen, (rows, cols), 1e-3 ** 0.5, dtype)
        leaves = [t.requires_grad_() for t in (x, w, bias) if t is not None]
        return {"case": case, "x": x, "w": w, "bias": bias, "dy": dy, "leaves": leaves}
    k, n, r, adapters = case["k"], case["n"], case["rank"], case["adapters"]
    requests = _requests(case)
    tokens = requests[-1][1]
    x = _activation(gen, tokens, k, dtype)
    base = _normal(gen, (tokens, n), 1.0, dtype)
    a = _normal(gen, (adapters, r, k), k ** -0.5, dtype)
    b = _normal(gen, (adapters, n, r), 0.3 * r ** -0.5, dtype)
    scales = 0.5 + 1.5 * torch.rand(adapters, generator=gen, device="cuda")
    state = {"case": case, "x": x, "base": base, "a": a, "b": b, "scales": scales, "requests": requests}
    if own:
        # which token uses which adapter: once a batch, for every projection of the model
        from float8linear_tensorwise_amax_amd import module
        index = torch.tensor([i for at, end, i in requests for _ in range(at, end)], dtype=torch.int32, device="cuda")
        state["batch"] = module.LoraBatch(index, adapters)
    if op == "lora_train":
        state["dy"] = _normal(gen, (tokens, n), 1e-3 ** 0.5, dtype)
        state["leaves"] = [t.requires_grad_() for t in (x, a, b)]
    return state


# ---------------------------------------------------------------- plain form

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(op, state)
    with torch.no_grad():
        return _norm(op, state) if op.startswith("norm") else _lora(op, state)


def _norm(op, state):
    x, w = state["x"].float(), state["w"].float()
    centred = x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((centred * centred).mean(1, keepdim=True) + _EPS)
    xhat = centred * rstd
    y = xhat * w
    if state["bias"] is not None:
        y = y + state["bias"].float()
    y = y.to(state["x"].dtype)
    if op == "norm":
        return y
    dy = state["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    out = [y, dx.to(state["x"].dtype), (dy * xhat).sum(0).to(state["w"].dtype)]
    return out + [dy.sum(0).to(state["bias"].dtype)] if state["bias"] is not None else out


def _lora(op, state):
    x, base, a, b, scales = (state[k] for k in ("x", "base", "a", "b", "scales"))
    train = op == "lora_train"
    y = base.clone()
    if train:
        dx = torch.zeros_like(x)
        da, db = torch.zeros_like(a, dtype=torch.float32), torch.zeros_like(b, dtype=torch.float32)
    for at, end, i in state["requests"]:
        if i < 0:
            continue
        xs, ai, bi, s = x[at:end].float(), a[i].float(), b[i].float(), scales[i]
        h = s * (xs @ ai.t())
        y[at:end] = (base[at:end].float() + h @ bi.t()).to(y.dtype)
        if train:
            ds = state["dy"][at:end].float()
            g = s * (ds @ bi)
            dx[at:end] = (g @ ai).to(dx.dtype)
            da[i] += g.t() @ xs
            db[i] += ds.t() @ h
    return [y, dx, da.to(a.dtype), db.to(b.dtype)] if train else y


def _own(op, state):
    from float8linear_tensorwise_amax_amd import module
    if op.startswith("norm"):
        y = module.layer_norm(state["x"], state["w"], state["bias"], _EPS)
    else:
        y = module.lora_add(state["base"], state["x"], state["a"], state["b"], state["batch"], state["scales"])
    if "dy" not in state:
        return y
    return [y.detach(), *torch.autograd.grad(y, state["leaves"], state["dy"])]


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        x, w = s["x"].detach().double(), s["w"].detach().double()
        n = case["cols"]
        mean = torch.matmul(x, torch.full((n, 1), 1.0 / n, dtype=torch.float64, device=x.device))
        xhat = x - mean
        rstd = torch.rsqrt(torch.linalg.vecdot(xhat, xhat).unsqueeze(1) / n + _EPS)
        xhat = xhat * rstd
        y = torch.addcmul(torch.zeros_like(w) if s["bias"] is None else s["bias"].detach().double(), xhat, w)
        if case["op"] == "norm":
            return y
        dy = s["dy"].double()
        g = dy * w
        # the projection of g off the constant vector and off xhat
        dx = (g - torch.linalg.vecdot(g, torch.ones_like(g)).unsqueeze(1) / n
              - xhat * (torch.linalg.vecdot(g, xhat).unsqueeze(1) / n)) * rstd
        out = [y, dx, torch.linalg.vecdot(dy, xhat, dim=0)]
        return out + [torch.linalg.vecdot(dy, torch.ones_like(dy), dim=0)] if s["bias"] is not None else out
    train = case["op"] == "lora_train"
    index = torch.tensor([i for at, end, i in s["requests"] for _ in range(at, end)], device="cuda")
    x, a, b = (s[k].detach() for k in ("x", "a", "b"))
    y = s["base"].double()
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    da, db = torch.zeros_like(a, dtype=torch.float64), torch.zeros_like(b, dtype=torch.float64)
    for i in range(case["adapters"]):
        rows = torch.nonzero(index == i).flatten()
        if rows.numel() == 0:
            continue
        low, up, s_i = a[i].double(), b[i].double(), float(s["scales"][i])
        xi = x[rows].double()
        inner = torch.matmul(xi, low.t().contiguous())
        y[rows] += s_i * torch.matmul(inner, up.t().contiguous())
        if train:
            di = s["dy"][rows].double()
            back = torch.matmul(di, up)
            dx[rows] = s_i * torch.matmul(back, low)
            da[i] = s_i * torch.matmul(back.t().contiguous(), xi)
            db[i] = s_i * torch.matmul(di.t().contiguous(), inner)
    return [y, dx, da, db] if train else y
