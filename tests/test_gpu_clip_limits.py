"""Clipping without a limit: max_norm = inf only measures."""
import math

import pytest
import torch

from test_gpu_grad_clip import DTYPES, draw, mod, f8lin  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_an_infinite_limit_leaves_the_gradients(mod, f8lin, dtype, p):
    """No gradient is above it, whatever the norm; only a NaN norm makes them NaN, as with any limit."""
    for bad in (0.5, math.inf, -math.inf, math.nan):
        grads = [g.cuda() for g in draw([100, 40001, 7], DTYPES[dtype], 1)]
        grads[1][30000] = bad
        norm, outs = mod.clip_grads(grads, math.inf, p, torch.float32)
        params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
        for q, g in zip(params, grads):
            q.grad = g.clone()
        again = mod.clip_grad_norm_(params, math.inf, p)
        given = [torch.empty_like(g) for g in grads]
        f8lin.grad_clip(grads, math.inf, norm.view(1), None, p, outs=given, norm_given=True)
        assert torch.equal(torch.isfinite(norm), torch.tensor(math.isfinite(bad), device="cuda"))
        for g, o, q, v in zip(grads, outs, params, given):
            if math.isnan(bad):
                assert torch.isnan(o).all() and torch.isnan(q.grad).all() and torch.isnan(v).all()
            else:
                assert torch.equal(o, g.float()) and torch.equal(q.grad, g) and torch.equal(v, g)
        assert math.isnan(bad) or torch.equal(norm, again)
