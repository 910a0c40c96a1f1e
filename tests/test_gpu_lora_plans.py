"""Calls with a plan that is not theirs write nothing, whatever the buffers hold, and read no more of it than its header."""
import ctypes

import pytest
import torch

from test_gpu_lora import f8lin, index_of, tensors  # noqa: F401

pytestmark = pytest.mark.gpu

PATTERN = 5.0


def filled(*shape, dtype=torch.float32):
    return torch.full(shape, PATTERN, dtype=dtype, device="cuda")


@pytest.mark.parametrize("T", [1, 30, 700, 1500])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("R", [4, 40, 100])
def test_nothing_is_written(f8lin, T, dtype, R):
    K, N, L = 40, 50, 3
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, dtype, 7))
    others = [(T + 1, L), (T, L + 1), (max(T - 1, 0), L)]
    for tokens, adapters in others:
        plan = f8lin.LoraPlan(T, L)
        plan.buffer.fill_(-7)
        wide = torch.full((plan.buffer.numel() + 4096,), -7, dtype=torch.int32, device="cuda")
        other = f8lin.LoraPlan(tokens, adapters, buffer=wide)
        f8lin.lora_plan(torch.zeros(tokens, dtype=torch.int32, device="cuda"), other)
        plan.buffer.copy_(wide[:plan.buffer.numel()])
        ws = filled(1 << 19)
        y, dx, da, db = (filled(*t.shape, dtype=dtype) for t in (base, x, a, b))
        h = filled(f8lin.lora_h_elements(T, R))
        f8lin.lora_forward(base, x, a, b, scales, plan, y, h, ws)
        f8lin.lora_backward(dy, x, a, b, scales, plan, h, dx, da, db, ws)
        for t in (y, dx, da, db, h, ws):
            assert bool((t == PATTERN).all())


@pytest.mark.parametrize("T", [20, 1000, 20000])
def test_a_shorter_plan(f8lin, T):
    """Through the C interface, which is given no size of the plan: the plan of one token of one adapter beside a call of
    many tokens."""
    K, N, R, L, dt = 48, 64, 8, 5, torch.bfloat16
    base, x, a, b, dy, scales = (t.cuda() for t in tensors(T, K, N, R, L, dt, 7))
    # (nothing else near it: outputs that a plan of the call's own sizes would reach into are refused)
    room = torch.full((f8lin.LoraPlan(T, L).buffer.numel(),), -7, dtype=torch.int32, device="cuda")
    plan = f8lin.LoraPlan(1, 1, buffer=room)
    f8lin.lora_plan(torch.zeros(1, dtype=torch.int32, device="cuda"), plan)
    y, dx, da, db = (filled(*t.shape, dtype=dt) for t in (base, x, a, b))
    h = filled(f8lin.lora_h_elements(T, R))
    ws = filled(max(f8lin.lora_forward_workspace_bytes(T, K, N, R, L), f8lin.lora_backward_workspace_bytes(T, K, N, R, L)) // 4)
    p = lambda t: t.data_ptr()  # noqa: E731
    fwd = f8lin.LoraFwdArgs(T, K, N, p(x), p(a), p(b), p(base), 0, 0, p(y), p(scales), p(plan.buffer), p(h), p(ws),
                            4 * ws.numel(), R, L, 0)
    bwd = f8lin.LoraBwdArgs(T, K, N, p(dy), p(x), p(a), p(b), 0, 0, p(scales), p(h), p(plan.buffer), p(dx), p(da), p(db),
                            p(ws), 4 * ws.numel(), R, L, 0)
    s = torch.cuda.current_stream().cuda_stream
    assert f8lin._lib.f8lin_lora_forward(ctypes.byref(fwd), s) == 0
    assert f8lin._lib.f8lin_lora_backward(ctypes.byref(bwd), s) == 0
    torch.cuda.synchronize()
    for t in (y, dx, da, db, h, ws):
        assert bool((t == PATTERN).all())
