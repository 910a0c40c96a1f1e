"""PyTorch module surface over the C ABI: a Float8Linear layer, the swap of
nn.Linear for it, and the delayed-scaling sync after backward.

This mirrors the user interface the pages show (pytorch/ao issue #1297,
repro script: convert_to_float8_training(model, config=Float8LinearConfig(
cast_config_input / weight / grad_output = CastConfig(ScalingType...))),
and sync_float8_amax_and_scale_history(model) after loss.backward();
pytorch/ao issue #1199: convert_to_float8_training swapping nn.Linear).
Every step of the forward and backward runs in libf8lin's HIP kernels;
this file only allocates tensors and marshals arguments.

Shapes: in_features and out_features must be multiples of 16.  The token
dimension may be anything: it is zero-padded to a multiple of 16, which is
exact (zero rows raise no amax, add nothing to dW or to the bias gradient,
and their Y / dX rows are dropped).  A bias (the repro's nn.Linear layers
keep theirs) is added in the GEMM epilogue and its gradient is summed in the
backward's cast pass.

Scaling state.  Each layer keeps, per tensor role (input x, weight w,
grad_output dy), the device state the library reads and writes -- amax,
{scale, 1/scale}, the 16-entry amax history and {count, pos} -- as
registered buffers, so model.state_dict() / load_state_dict() save and
restore it and model.to() moves it; which delayed roles have taken their
first step is saved as the module's extra state.

MXFP4.  mxfp4_linear / MXFP4Linear / convert_to_mxfp4_training are the same
layer with 4-bit operands (one 8-bit scale per 32 values along each product's
contraction, so no scaling state); any feature and token counts, in bf16,
fp16 or fp32.  freeze_mxfp4 keeps only the 4-bit weights, for serving.

Gradient clipping.  clip_grad_norm_ (in place), clip_grads (into new tensors)
and get_grad_norm work on a list of gradients after backward.

Layer norm.  layer_norm / LayerNorm / convert_layer_norm: the norm in front of
a block's linears, forward and backward.

Low-rank adapters.  lora_add / LoraLinear / convert_to_lora put adapters
beside a shared projection (any of the linears above); a batch mixes requests
of many adapters, and a LoraBatch says which token uses which.

All of them can be captured into a HIP graph, a whole step under autograd too.  As
with any layer, let no eager graph of the same parameters live on into the
capture of a backward: its gradient nodes belong to another stream.

Delayed scaling, per role:
  * the scale comes from the largest amax of the previous steps (the
    history), and the cast folds this step's amax into the state;
  * a role's first step has no history: it takes its scale from the current
    tensor (amax initialisation).  It runs through the same delayed cast with
    a one-entry history seeded with the current tensor's amax (computed by
    the library's amax pass), so the scale is the dynamic one, bit for bit,
    and the state's amax still collects the maximum over every micro-batch
    of the step;
  * the sync after backward pushes the amax of every delayed role that has
    produced one since the last sync (a forward without backward produces
    none for dy), and only those roles count as initialised.
"""
from dataclasses import dataclass, field
from typing import Dict, Iterable, List, Optional, Tuple, Union

import torch
import torch.nn as nn
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import f8lin

_ROLES = ("x", "w", "dy")
_STATE_FIELDS = (("amax", (1,), torch.float32), ("scale", (2,), torch.float32),
                 ("history", (f8lin.HISTORY_LEN,), torch.float32), ("hist_meta", (2,), torch.int32))


@dataclass
class CastConfig:
    scaling_type: str = "dynamic"  # "dynamic" or "delayed"

    def __post_init__(self):
        if self.scaling_type not in ("dynamic", "delayed"):
            raise ValueError(f"scaling_type must be 'dynamic' or 'delayed', got {self.scaling_type!r}")


@dataclass
class Float8LinearConfig:
    cast_config_input: CastConfig = field(default_factory=CastConfig)
    cast_config_weight: CastConfig = field(default_factory=CastConfig)
    cast_config_grad_output: CastConfig = field(default_factory=CastConfig)
    amax_algo: str = "twopass"  # "atomic" or "twopass"
    # Opt-in: reuse the weight's fp8 copies while the weight tensor and its
    # version counter are unchanged (e.g. the micro-batches of one optimizer
    # step).  Updates through .data (p.data.copy_, EMA, checkpoint loading)
    # do not move the version counter: after such an update call
    # invalidate_weight_cast(model).  The cache is also dropped at every
    # sync_float8_amax_and_scale_history.
    reuse_weight_cast: bool = False


def _pad_rows(t: torch.Tensor) -> torch.Tensor:
    m = t.shape[0]
    pad = (-m) % 16
    if pad == 0:
        return t.contiguous()
    return torch.cat([t, t.new_zeros((pad, t.shape[1]))], dim=0)


class _Float8LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, weight, bias, layer):
        M0 = x2d.shape[0]
        x = _pad_rows(x2d.to(torch.bfloat16))
        b = None if bias is None else bias.to(torch.bfloat16).contiguous()
        M, K = x.shape
        N = weight.shape[0]
        dev = x.device
        u8 = dict(dtype=torch.uint8, device=dev)
        x8 = torch.empty((M, K), **u8)
        x8t = f8lin.new_transposed(K, M, dev)
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        key = (weight.data_ptr(), weight._version, weight.dtype, str(dev), layer._mode("w"))
        cached = layer._w_cache if (layer.config.reuse_weight_cast and layer._w_cache is not None
                                    and layer._w_cache[0] == key) else None
        mode_x, sx = layer._prepare("x", x)
        if cached is not None:
            # unchanged weight: its fp8 copies and scale (in the w state) are still valid
            w, w8, w8t = None, cached[1], cached[2]
            mode_w, sw = "dynamic", layer.state("w")
            layer.weight_cast_reuses += 1
        else:
            # fresh copies: an earlier forward's backward may still read the old ones
            w = weight.to(torch.bfloat16).contiguous()
            w8 = torch.empty((N, K), **u8)
            w8t = f8lin.new_transposed(K, N, dev)
            mode_w, sw = layer._prepare("w", w)
        f8lin.forward(x, w, y, x8, x8t, w8, w8t, sx, sw, layer.fp8_workspace, mode_x, mode_w,
                      layer.config.amax_algo, bias=b, w_cast_valid=cached is not None)
        if cached is None and layer.config.reuse_weight_cast:
            layer._w_cache = (key, w8, w8t)
        # backward must use the scales these fp8 copies were made with, even if
        # the layer runs forward again before it (micro-batches, recomputation)
        ctx.save_for_backward(x8t, w8t, sx.scale.clone(), sw.scale.clone())
        ctx.layer = layer
        ctx.M0 = M0
        ctx.w_dtype = weight.dtype
        ctx.b_dtype = None if bias is None else bias.dtype
        return y[:M0]

    @staticmethod
    def backward(ctx, dy2d):
        x8t, w8t, sx_scale, sw_scale = ctx.saved_tensors
        layer = ctx.layer
        dy = _pad_rows(dy2d.to(torch.bfloat16))
        M, N = dy.shape
        K = x8t.shape[0]
        dev = dy.device
        dy8 = torch.empty((M, N), dtype=torch.uint8, device=dev)
        dy8t = f8lin.new_transposed(N, M, dev)
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
        db = db_ws = None
        if ctx.b_dtype is not None:
            db = torch.empty((N,), dtype=torch.bfloat16, device=dev)
            db_ws = f8lin.new_dbias_workspace(M, N, dev)
        # scratch for GEMMs split along their contraction (None when none splits at this shape)
        gemm_ws = f8lin.new_backward_gemm_workspace(M, N, K, dev)
        mode_dy, sdy = layer._prepare("dy", dy)
        f8lin.backward(dy, x8t, w8t, dx, dw, dy8, dy8t, f8lin.ScaleView(sx_scale), f8lin.ScaleView(sw_scale),
                       sdy, layer.fp8_workspace, mode_dy, layer.config.amax_algo, dbias=db, dbias_ws=db_ws,
                       gemm_ws=gemm_ws)
        return dx[:ctx.M0], dw.to(ctx.w_dtype), (None if db is None else db.to(ctx.b_dtype)), None


class Float8Linear(nn.Module):
    """nn.Linear whose forward and backward GEMMs run in fp8 with tensorwise
    scaling: X and W cast to e4m3, dY to e5m2, per-tensor scales from the
    current amax (dynamic) or a 16-step amax history (delayed)."""

    def __init__(self, in_features: int, out_features: int, config: Optional[Float8LinearConfig] = None,
                 weight: Optional[torch.Tensor] = None, device=None, dtype=torch.bfloat16, bias=False):
        super().__init__()
        if in_features % 16 or out_features % 16:
            raise ValueError("Float8Linear needs in_features and out_features that are multiples of 16")
        self.in_features = in_features
        self.out_features = out_features
        self.config = config or Float8LinearConfig()
        if weight is None:
            weight = torch.empty((out_features, in_features), device=device, dtype=dtype)
            nn.init.kaiming_uniform_(weight, a=5 ** 0.5)
        self.weight = weight if isinstance(weight, nn.Parameter) else nn.Parameter(weight)
        # bias: False / True (a zero-initialised bias), or an existing tensor / Parameter to share
        if isinstance(bias, torch.Tensor):
            if tuple(bias.shape) != (out_features,):
                raise ValueError("bias must have shape (out_features,)")
            self.bias = bias if isinstance(bias, nn.Parameter) else nn.Parameter(bias)
        elif bias:
            self.bias = nn.Parameter(torch.zeros(out_features, device=self.weight.device, dtype=self.weight.dtype))
        else:
            self.register_parameter("bias", None)
        dev = self.weight.device
        for role in _ROLES:
            for name, shape, dt in _STATE_FIELDS:
                self.register_buffer(f"fp8_{role}_{name}", torch.zeros(shape, dtype=dt, device=dev))
        # the library's workspace, and one history per role whose slot 0 holds
        # the current amax during a delayed role's first step (slots 1-15 stay 0)
        self.register_buffer("fp8_workspace", torch.zeros(f8lin.workspace_bytes(), dtype=torch.uint8, device=dev),
                             persistent=False)
        self.register_buffer("fp8_seed_history", torch.zeros((len(_ROLES), f8lin.HISTORY_LEN), dtype=torch.float32,
                                                             device=dev), persistent=False)
        self._initialized: Dict[str, bool] = {r: False for r in _ROLES}
        self._produced: Dict[str, bool] = {r: False for r in _ROLES}
        self._w_cache = None  # (key, w8, w8t) of the weight's last cast
        self.weight_cast_reuses = 0

    # ---- scaling state
    def state(self, role: str) -> f8lin.ScalingState:
        """The role's device state (views of this module's buffers)."""
        return f8lin.ScalingState(tensors=tuple(getattr(self, f"fp8_{role}_{n}") for n, _, _ in _STATE_FIELDS))

    sx = property(lambda self: self.state("x"))
    sw = property(lambda self: self.state("w"))
    sdy = property(lambda self: self.state("dy"))

    def _cfg(self, role):
        return {"x": self.config.cast_config_input, "w": self.config.cast_config_weight,
                "dy": self.config.cast_config_grad_output}[role]

    def _mode(self, role):
        """How the role's scale is taken this step: "delayed" (from the
        history) once the role has been synced, else "dynamic" (the current
        tensor's amax; for a delayed role this is its first step)."""
        if self._cfg(role).scaling_type == "delayed" and self._initialized[role]:
            return "delayed"
        return "dynamic"

    def _prepare(self, role, t: torch.Tensor):
        """(mode, state) for casting tensor t of `role`, and marks the role as
        having produced an amax since the last sync."""
        self._produced[role] = True
        st = self.state(role)
        if self._cfg(role).scaling_type == "dynamic" or self._initialized[role]:
            return self._mode(role), st
        # a delayed role's first step: the delayed cast with a history seeded
        # with this tensor's amax (the dynamic scale; the cast folds the amax
        # into the state, max over micro-batches)
        seed = self.fp8_seed_history[_ROLES.index(role)]
        f8lin.amax(t, seed[0:1], self.fp8_workspace, self.config.amax_algo)
        return "delayed", f8lin.ScalingState(tensors=(st.amax, st.scale, seed, st.hist_meta))

    def delayed_states(self):
        """States of the delayed roles that produced an amax since the last sync."""
        return [self.state(r) for r in self._sync_roles()]

    def _sync_roles(self):
        return [r for r in _ROLES if self._cfg(r).scaling_type == "delayed" and self._produced[r]]

    def _mark_synced(self, roles=None):
        for r in (self._sync_roles() if roles is None else roles):
            self._initialized[r] = True
            self._produced[r] = False
        self._w_cache = None  # the weight's scale may move with its history; the step is over

    def invalidate_weight_cast(self):
        """Drop the cached weight cast (after changing the weight through .data)."""
        self._w_cache = None

    # ---- checkpointing: the buffers are saved by nn.Module; the flags here
    def get_extra_state(self):
        return {"initialized": [bool(self._initialized[r]) for r in _ROLES]}

    def set_extra_state(self, state):
        flags = state["initialized"]
        self._initialized = {r: bool(f) for r, f in zip(_ROLES, flags)}
        self._produced = {r: False for r in _ROLES}
        self._w_cache = None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if not x.is_cuda:
            raise RuntimeError("Float8Linear runs on the GPU only (libf8lin has no CPU path)")
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        if self.fp8_x_amax.device != x.device:
            raise RuntimeError(f"Float8Linear's scaling state is on {self.fp8_x_amax.device}, the input on "
                               f"{x.device}: move the module with .to()")
        lead = x.shape[:-1]
        y = _Float8LinearFn.apply(x.reshape(-1, self.in_features), self.weight, self.bias, self)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        c = self.config
        return (f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, "
                f"input={c.cast_config_input.scaling_type}, weight={c.cast_config_weight.scaling_type}, "
                f"grad_output={c.cast_config_grad_output.scaling_type}, amax_algo={c.amax_algo}")


def convert_to_float8_training(module: nn.Module, config: Optional[Float8LinearConfig] = None,
                               module_filter_fn=None) -> nn.Module:
    """Replaces every nn.Linear whose dimensions are multiples of 16 (and that
    module_filter_fn(fqn, module) accepts, if given) by a Float8Linear sharing
    its weight and bias Parameters.  Returns the module."""
    config = config or Float8LinearConfig()

    def swap(parent: nn.Module, prefix: str):
        for name, child in list(parent.named_children()):
            fqn = f"{prefix}.{name}" if prefix else name
            if (type(child) is nn.Linear and child.in_features % 16 == 0 and child.out_features % 16 == 0
                    and (module_filter_fn is None or module_filter_fn(fqn, child))):
                setattr(parent, name, Float8Linear(child.in_features, child.out_features, config,
                                                   weight=child.weight,
                                                   bias=child.bias if child.bias is not None else False))
            else:
                swap(child, fqn)

    if type(module) is nn.Linear:
        raise ValueError("convert the parent module, not a bare nn.Linear")
    swap(module, "")
    return module


def invalidate_weight_cast(module: nn.Module) -> None:
    """Drops every Float8Linear's cached weight cast (call it after changing
    weights through .data when reuse_weight_cast is on)."""
    for m in module.modules():
        if isinstance(m, Float8Linear):
            m.invalidate_weight_cast()


def sync_float8_amax_and_scale_history(module: nn.Module, check: bool = False) -> None:
    """After backward: pushes the amax of this step of every delayed-scaling
    role that produced one into its 16-entry history (one launch for all
    layers' states).  check=True also reads back the library's per-state
    status (a host synchronisation) and raises if a state's {count, pos}
    was corrupt (such a state is left untouched)."""
    states, layers = [], []
    for m in module.modules():
        if isinstance(m, Float8Linear):
            roles = m._sync_roles()
            states.extend(m.state(r) for r in roles)
            layers.append((m, roles))
    status = None
    if states:
        if check:
            status = torch.empty(len(states), dtype=torch.int32, device=states[0].amax.device)
        f8lin.delayed_update(states, status=status)
    for m, roles in layers:
        m._mark_synced(roles)
    if status is not None:
        bad = torch.nonzero(status).flatten().tolist()
        if bad:
            raise RuntimeError(f"sync_float8_amax_and_scale_history: {len(bad)} corrupt delayed-scaling "
                               f"state(s) (invalid count/pos), left unchanged: state indices {bad}")


# ------------------------------------------------------------------- MXFP4

def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as a 2-D tensor with contiguous rows (a copy only where its strides need one)."""
    if t.dim() == 2 and t.is_contiguous():
        return t
    t = t.reshape(-1, t.shape[-1])
    if t.numel() and ((t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1])):
        t = t.contiguous()
    return t


def _refuse_tangents(what: str, *tensors: Optional[torch.Tensor]) -> None:
    """Raises where a tensor has a forward-mode tangent: a call that takes no part in autograd would drop it, and its
    result would read as having a derivative of zero."""
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{what} has no forward-mode derivative")


def _present(*pairs):
    """The shapes of the pairs (asked for, shape) that are asked for."""
    return [shape for ask, shape in pairs if ask]


def _mxfp4_forward(x, weight, bias, rule, need_x, need_w):
    """(y, buffer of the transposed copies that the gradients asked for will need, or None)."""
    M, K = x.shape
    N = weight.shape[0]
    dev = x.device
    y = torch.empty((M, N), dtype=x.dtype, device=dev)
    _, (x4, w4) = f8lin.new_mxfp4s(((M, K), (N, K)), dev)
    x4t = w4t = saved = None
    if need_x or need_w:
        saved, copies = f8lin.new_mxfp4s(_present((need_w, (K, M)), (need_x, (K, N))), dev)
        x4t = copies[0] if need_w else None
        w4t = copies[-1] if need_x else None
    f8lin.mxfp4_forward(x, weight if weight.is_contiguous() else weight.contiguous(), y, x4, w4, x4t, w4t,
                        bias if bias is None or bias.is_contiguous() else bias.contiguous(), rule)
    return y, saved


class _MXFP4LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, rule):
        y, saved = _mxfp4_forward(x, weight, bias, rule, *ctx.needs_input_grad[:2])
        if saved is not None:
            ctx.save_for_backward(saved)
        ctx.args = (x.shape[0], weight.shape[0], x.shape[1], rule, x.dtype, weight.dtype,
                    None if bias is None else bias.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        M, N, K, rule, x_dtype, w_dtype, b_dtype = ctx.args
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        dev = dy.device
        dy = _rows(dy)
        x4t = w4t = dx = dw = db = db_ws = None
        if need_x or need_w:
            copies = f8lin.new_mxfp4s(_present((need_w, (K, M)), (need_x, (K, N))), dev, ctx.saved_tensors[0])[1]
            x4t = copies[0] if need_w else None
            w4t = copies[-1] if need_x else None
        if need_x:
            dx = torch.empty((M, K), dtype=x_dtype, device=dev)
        if need_w:
            dw = torch.empty((N, K), dtype=w_dtype, device=dev)
        if need_b:
            db = torch.empty((N,), dtype=b_dtype, device=dev)
            db_ws = torch.empty(max(1, f8lin.mxfp4_dbias_workspace_bytes(M, N) // 4), dtype=torch.float32, device=dev)
        cols = need_w or need_b
        _, copies = f8lin.new_mxfp4s(_present((need_x, (M, N)), (cols, (N, M))), dev)
        f8lin.mxfp4_backward(dy, x4t, w4t, dx, dw, copies[0] if need_x else None, copies[-1] if cols else None, db, db_ws,
                             rule)
        return dx, dw, db, None


def mxfp4_linear(x: torch.Tensor, weight: Union[torch.Tensor, f8lin.MXFP4Tensor], bias: Optional[torch.Tensor] = None,
                 rule: str = "floor") -> torch.Tensor:
    """y = x . weight^T (+ bias) with both operands of the product in MXFP4; y has x's dtype.

    weight a (out, in) tensor: it is quantised by the call, and the call is differentiable in x, weight and bias
    (the two backward products run in MXFP4 too, on operands quantised along their own contractions).
    weight an f8lin.MXFP4Tensor of (out, in): for serving; x must not need a gradient.
    Forward-mode derivatives are refused (NotImplementedError), whatever the grad mode."""
    if not x.is_cuda:
        raise RuntimeError("mxfp4_linear runs on the GPU only (libf8lin has no CPU path)")
    packed = isinstance(weight, f8lin.MXFP4Tensor)
    N, K = (weight.rows, weight.cols) if packed else weight.shape
    if x.dim() < 1 or x.shape[-1] != K:
        raise ValueError(f"expected last dimension {K}, got {tuple(x.shape)}")
    lead = x.shape[:-1]
    # (an empty last dimension leaves reshape nothing to infer the rows from)
    x2 = _rows(x) if x.numel() else x.reshape(lead.numel(), K)
    # (torch.jit.trace sees a Function, and of the library's own call nothing but the empty output)
    traced = torch._C._get_tracing_state() is not None
    if not packed and (traced or torch.is_grad_enabled()):
        return _MXFP4LinearFn.apply(x2, weight, bias, rule).reshape(*lead, N)
    _refuse_tangents("mxfp4_linear", x, bias, None if packed else weight)
    if traced:
        raise RuntimeError("mxfp4_linear: a call with a quantised weight cannot be traced")
    if not packed:
        return _mxfp4_forward(x2, weight, bias, rule, False, False)[0].reshape(*lead, N)
    if torch.is_grad_enabled() and (x.requires_grad or (bias is not None and bias.requires_grad)):
        raise RuntimeError("mxfp4_linear: a quantised weight has no backward; call it under torch.no_grad()")
    M = x2.shape[0]
    y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    fused = f8lin.mxfp4_forward_fused(M, N, K)  # X is quantised inside the product: no buffers
    f8lin.mxfp4_forward(x2, None, y, None if fused else f8lin.new_mxfp4(M, K, x.device), weight,
                        bias=bias if bias is None or bias.is_contiguous() else bias.contiguous(), rule=rule)
    return y if x.dim() == 2 else y.reshape(*lead, N)


class MXFP4Linear(nn.Module):
    """nn.Linear whose products run in MXFP4 (mxfp4_linear).  freeze() replaces the weight by its 4-bit form, kept in
    the buffers weight_codes and weight_scales, after which the layer only serves: its bias is no longer trained, and
    an input that needs a gradient is refused.  (A frozen layer's state dict loads into a frozen layer.)"""

    def __init__(self, in_features: int, out_features: int, rule: str = "floor", weight: Optional[torch.Tensor] = None,
                 device=None, dtype=torch.bfloat16, bias=False):
        super().__init__()
        if rule not in ("floor", "ceil"):
            raise ValueError(f"rule must be 'floor' or 'ceil', got {rule!r}")
        self.in_features, self.out_features, self.rule = in_features, out_features, rule
        if weight is None:
            weight = torch.empty((out_features, in_features), device=device, dtype=dtype)
            nn.init.kaiming_uniform_(weight, a=5 ** 0.5)
        if tuple(weight.shape) != (out_features, in_features):
            raise ValueError("weight must have shape (out_features, in_features)")
        self.weight = weight if isinstance(weight, nn.Parameter) else nn.Parameter(weight)
        if isinstance(bias, torch.Tensor):
            if tuple(bias.shape) != (out_features,):
                raise ValueError("bias must have shape (out_features,)")
            self.bias = bias if isinstance(bias, nn.Parameter) else nn.Parameter(bias)
        elif bias:
            self.bias = nn.Parameter(torch.zeros(out_features, device=self.weight.device, dtype=self.weight.dtype))
        else:
            self.register_parameter("bias", None)
        self.register_buffer("weight_codes", None)
        self.register_buffer("weight_scales", None)

    @property
    def frozen(self) -> bool:
        return self.weight_codes is not None

    @torch.no_grad()
    def freeze(self) -> "MXFP4Linear":
        """Quantises the weight once and drops its full form."""
        if not self.frozen:
            q = f8lin.new_mxfp4(self.out_features, self.in_features, self.weight.device)
            f8lin.mxfp4_quantize(self.weight.detach().contiguous(), q, None, self.rule)
            self.weight_codes, self.weight_scales = q.codes.clone(), q.scales.clone()
            self.weight = None
            if self.bias is not None:
                self.bias = nn.Parameter(self.bias.detach(), requires_grad=False)
        return self

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if not self.frozen:
            return mxfp4_linear(x, self.weight, self.bias, self.rule)
        q = f8lin.MXFP4Tensor(self.weight_codes, self.weight_scales, self.out_features, self.in_features)
        return mxfp4_linear(x, q, self.bias, self.rule)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, "
                f"rule={self.rule}, frozen={self.frozen}")


def convert_to_mxfp4_training(module: nn.Module, rule: str = "floor", module_filter_fn=None) -> nn.Module:
    """Replaces every nn.Linear (that module_filter_fn(fqn, module) accepts, if given) by an MXFP4Linear sharing its
    weight and bias Parameters.  A linear that stands in several places becomes one MXFP4Linear in all of them; the
    filter is asked for each (for the places inside a shared parent, once, under that parent's first name).  Returns the
    module."""
    if type(module) is nn.Linear:
        raise ValueError("convert the parent module, not a bare nn.Linear")
    made: Dict[nn.Linear, MXFP4Linear] = {}
    for prefix, parent in list(module.named_modules()):
        # (not named_children, which names a child once)
        for name, child in list(parent._modules.items()):
            fqn = f"{prefix}.{name}" if prefix else name
            if type(child) is nn.Linear and (module_filter_fn is None or module_filter_fn(fqn, child)):
                if child not in made:
                    made[child] = MXFP4Linear(child.in_features, child.out_features, rule, weight=child.weight,
                                              bias=child.bias if child.bias is not None else False)
                setattr(parent, name, made[child])
    return module


def freeze_mxfp4(module: nn.Module) -> nn.Module:
    """freeze() on every MXFP4Linear of the module: 4-bit weights only, for serving.  Returns the module."""
    for m in module.modules():
        if isinstance(m, MXFP4Linear):
            m.freeze()
    return module


# --------------------------------------------------- gradient norm and clipping

def _dense_copy(g: torch.Tensor) -> torch.Tensor:
    return g if f8lin._is_dense(g) else g.contiguous()


def _gradients(parameters: Union[torch.Tensor, Iterable[torch.Tensor]]) -> List[torch.Tensor]:
    params = [parameters] if isinstance(parameters, torch.Tensor) else parameters
    return [p.grad for p in params if p.grad is not None]


def get_grad_norm(grads: Iterable[torch.Tensor], norm_type: float = 2.0) -> torch.Tensor:
    """The norm (2, 1 or inf) of all the gradients' elements as one vector: a float32 scalar on their GPU, outside any
    autograd graph (a forward-mode tangent is refused)."""
    grads = list(grads)
    _refuse_tangents("get_grad_norm", *grads)
    grads = [_dense_copy(g) for g in grads]
    if not grads:
        return torch.zeros((), dtype=torch.float32)
    dev = grads[0].device
    norm = torch.empty((), dtype=torch.float32, device=dev)
    f8lin.grad_norm(grads, norm, f8lin.new_grad_workspace(dev), norm_type)
    return norm


def clip_grads(grads: Iterable[torch.Tensor], max_norm: float, norm_type: float = 2.0,
               out_dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """(norm, clipped): the gradients times min(1, max_norm / (norm + 1e-6)) in new tensors (of out_dtype, e.g.
    float32 for a full-precision optimiser behind 16-bit gradients; default their own), outside any autograd graph (a
    forward-mode tangent is refused)."""
    grads = list(grads)
    _refuse_tangents("clip_grads", *grads)
    grads = [_dense_copy(g) for g in grads]
    if not grads:
        return torch.zeros((), dtype=torch.float32), []
    dev = grads[0].device
    norm = torch.empty((), dtype=torch.float32, device=dev)
    outs = [torch.empty_like(g, dtype=out_dtype) for g in grads]
    f8lin.grad_clip(grads, max_norm, norm, f8lin.new_grad_workspace(dev), norm_type, outs)
    return norm, outs


@torch.no_grad()
def clip_grad_norm_(parameters: Union[torch.Tensor, Iterable[torch.Tensor]], max_norm: float, norm_type: float = 2.0,
                    error_if_nonfinite: bool = False) -> torch.Tensor:
    """Scales the parameters' gradients in place so that the norm of all of them together is at most max_norm;
    returns the norm they had.  A NaN norm makes every gradient NaN; error_if_nonfinite=True reads the norm back
    instead (a host synchronisation) and raises before anything is scaled.  max_norm=inf only measures the norm.  A
    gradient may be there once: a parameter listed twice is refused."""
    grads = _gradients(parameters)
    if not grads:
        return torch.zeros((), dtype=torch.float32)
    _refuse_tangents("clip_grad_norm_", *grads)
    if any(st == 0 and n > 1 for g in grads for st, n in zip(g.stride(), g.shape)):
        raise ValueError("clip_grad_norm_: an expanded gradient cannot be scaled in place")
    flat = [_dense_copy(g) for g in grads]
    dev = flat[0].device
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws = f8lin.new_grad_workspace(dev)
    if error_if_nonfinite:
        f8lin.grad_norm(flat, norm, ws, norm_type)
        if not torch.isfinite(norm).item():
            raise RuntimeError(f"the norm of order {norm_type} of the gradients is not finite, so they cannot be "
                               "clipped")
        f8lin.grad_clip(flat, max_norm, norm, None, norm_type, norm_given=True)
    else:
        f8lin.grad_clip(flat, max_norm, norm, ws, norm_type)
    for g, f in zip(grads, flat):
        if f is not g:
            g.copy_(f)
    return norm


# -------------------------------------------------------------- layer norm

def _needs_graph(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether a call on these tensors has to pass through autograd.  (torch.jit.trace too sees a Function, and of the
    library's own call nothing but the empty output.)"""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return torch._C._get_tracing_state() is not None


def _vector_of(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return t if t is None or t.is_contiguous() else t.contiguous()


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        rows, cols = x.shape
        dev = x.device
        weight = _vector_of(weight)
        y = torch.empty((rows, cols), dtype=out_dtype, device=dev)
        stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
        f8lin.layer_norm_forward(x, y, weight, _vector_of(bias), eps, stats)
        ctx.save_for_backward(x, weight, stats)
        ctx.b_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        rows, cols = x.shape
        dev = x.device
        dx = torch.empty((rows, cols), dtype=x.dtype, device=dev) if need_x else None
        dw = torch.empty((cols,), dtype=weight.dtype, device=dev) if need_w else None
        db = torch.empty((cols,), dtype=ctx.b_dtype, device=dev) if need_b else None
        ws = None
        if need_w or need_b:
            ws = torch.empty(f8lin.layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev)
        f8lin.layer_norm_backward(_rows(dy), x, weight, stats, dx, dw, db, ws)
        return dx, dw, db, None, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The layer norm of x over its last dimension, times weight plus bias (vectors of that length, of any of the three
    types, or None): (x - mean) / sqrt(var + eps) * weight + bias, computed in float32 and rounded once.

    The result has x's dtype, or with a float32 x the given out_dtype (bfloat16 for the linears behind a float32
    residual stream, say).  Differentiable once in x, weight and bias; forward-mode derivatives are refused
    (NotImplementedError)."""
    if not x.is_cuda:
        raise RuntimeError("layer_norm runs on the GPU only (libf8lin has no CPU path)")
    if x.dim() < 1:
        raise ValueError("layer_norm needs a dimension to normalise over")
    cols = x.shape[-1]
    for what, t in (("weight", weight), ("bias", bias)):
        if t is not None and tuple(t.shape) != (cols,):
            raise ValueError(f"{what} must have shape ({cols},), got {tuple(t.shape)}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    dtype = x.dtype if out_dtype is None else out_dtype
    if dtype != x.dtype and (x.dtype != torch.float32 or dtype not in f8lin._DTYPE):
        raise TypeError(f"out_dtype must be {x.dtype} (only a float32 x allows another type), got {dtype}")
    # (an empty last dimension leaves reshape nothing to infer the rows from)
    x2 = _rows(x) if x.numel() else x.reshape(x.shape[:-1].numel(), cols)
    if _needs_graph(x, weight, bias):
        y = _LayerNormFn.apply(x2, weight, bias, eps, dtype)
    else:
        _refuse_tangents("layer_norm", x, weight, bias)
        y = torch.empty(x2.shape, dtype=dtype, device=x.device)
        f8lin.layer_norm_forward(x2, y, _vector_of(weight), _vector_of(bias), eps)
    return y if x.dim() == 2 else y.reshape(x.shape)


class LayerNorm(nn.Module):
    """nn.LayerNorm on this library's kernels (layer_norm).  weight and bias: True (new), False (none), or existing
    tensors / Parameters to share."""

    def __init__(self, normalized_shape, eps: float = 1e-5, weight=True, bias=True, device=None, dtype=torch.float32):
        super().__init__()
        shape = (normalized_shape,) if isinstance(normalized_shape, int) else tuple(normalized_shape)
        if not shape:
            raise ValueError("LayerNorm needs a shape to normalise over")
        self.normalized_shape, self.eps = shape, eps
        for name, given, fill in (("weight", weight, 1.0), ("bias", bias, 0.0)):
            if isinstance(given, torch.Tensor):
                if tuple(given.shape) != shape:
                    raise ValueError(f"{name} must have shape {shape}")
                given = given if isinstance(given, nn.Parameter) else nn.Parameter(given)
            elif given:
                given = nn.Parameter(torch.full(shape, fill, device=device, dtype=dtype))
            else:
                given = None
            self.register_parameter(name, given)

    def forward(self, x: torch.Tensor, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        n = len(self.normalized_shape)
        if tuple(x.shape[-n:]) != self.normalized_shape:
            raise ValueError(f"expected last dimensions {self.normalized_shape}, got {tuple(x.shape)}")
        if n == 1:
            return layer_norm(x, self.weight, self.bias, self.eps, out_dtype)
        flat = [None if p is None else p.reshape(-1) for p in (self.weight, self.bias)]
        lead = x.shape[:-n]
        return layer_norm(x.reshape(lead.numel(), -1) if x.numel() else x.reshape(lead.numel(), self._numel()), *flat,
                          self.eps, out_dtype).reshape(x.shape)

    def _numel(self) -> int:
        return torch.Size(self.normalized_shape).numel()

    def extra_repr(self):
        return (f"{self.normalized_shape}, eps={self.eps}, weight={self.weight is not None}, "
                f"bias={self.bias is not None}")


def _swap(module: nn.Module, accepts, make, module_filter_fn) -> nn.Module:
    """Replaces every child that `accepts` and the filter take by make(child); a child that stands in several places is
    made once.  What lies inside a LoraLinear is left as it is."""
    made: Dict[nn.Module, nn.Module] = {}
    for prefix, parent in list(module.named_modules()):
        if isinstance(parent, LoraLinear):
            continue
        # (not named_children, which names a child once)
        for name, child in list(parent._modules.items()):
            fqn = f"{prefix}.{name}" if prefix else name
            if child is not None and accepts(child) and (module_filter_fn is None or module_filter_fn(fqn, child)):
                if child not in made:
                    made[child] = make(child)
                setattr(parent, name, made[child])
    return module


def convert_layer_norm(module: nn.Module, module_filter_fn=None) -> nn.Module:
    """Replaces every nn.LayerNorm (that module_filter_fn(fqn, module) accepts, if given) by a LayerNorm sharing its
    weight and bias Parameters; one that stands in several places becomes one in all of them.  Returns the module."""
    if type(module) is nn.LayerNorm:
        raise ValueError("convert the parent module, not a bare nn.LayerNorm")
    return _swap(module, lambda m: type(m) is nn.LayerNorm,
                 lambda m: LayerNorm(m.normalized_shape, m.eps, m.weight if m.weight is not None else False,
                                     m.bias if m.bias is not None else False), module_filter_fn)


# ------------------------------------------------------- low-rank adapters

class LoraBatch:
    """Which token of a batch uses which adapter, sorted on the GPU once for all the projections that the batch passes.

    index: int32 or int64 tensor on the GPU, one entry a token (any shape; the tokens in its order); a value outside
    0 .. adapters - 1 means no adapter.  Tokens may come in any order."""

    def __init__(self, index: torch.Tensor, adapters: int):
        if not index.is_cuda:
            raise RuntimeError("LoraBatch runs on the GPU only (libf8lin has no CPU path)")
        self.plan = f8lin.LoraPlan(index.numel(), adapters, index.device)
        f8lin.lora_plan(index if index.is_contiguous() else index.contiguous(), self.plan)

    tokens = property(lambda self: self.plan.tokens)
    adapters = property(lambda self: self.plan.adapters)

    def update(self, index: torch.Tensor) -> "LoraBatch":
        """Another batch of as many tokens, in place (in a captured graph: from what index holds at the replay)."""
        f8lin.lora_plan(index if index.is_contiguous() else index.contiguous(), self.plan)
        return self


def _lora_forward(base, x, a, b, plan, scales, keep):
    """(y, the inner products if they are to be kept)."""
    y = torch.empty(base.shape, dtype=x.dtype, device=x.device)
    h = None
    if keep:
        h = torch.empty(f8lin.lora_h_elements(plan.tokens, b.shape[2]), dtype=torch.float32, device=x.device)
    f8lin.lora_forward(base, x, a, b, scales, plan, y, h)
    return y, h


class _LoraAddFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, base, x, a, b, plan, scales):
        a, b = a.contiguous(), b.contiguous()
        y, h = _lora_forward(base, x, a, b, plan, scales, ctx.needs_input_grad[3])
        # (the plan first: activation checkpointing compares what a forward and its recomputation save, one after the
        # other, and no other layer saves the like)
        ctx.save_for_backward(plan.buffer, plan.mark(), x, a, b, h, scales)
        ctx.sizes, ctx.serial = (plan.tokens, plan.adapters), plan.serial
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_base, need_x, need_a, need_b = ctx.needs_input_grad[:4]
        buffer, mark, x, a, b, h, scales = ctx.saved_tensors
        # Under checkpointing these tensors are the recomputation's, the node is the forward's.
        if int(mark) != ctx.serial:
            raise RuntimeError("low-rank adapters were recomputed for the backward with another batch than their forward "
                               "had (set or updated in between): pass the batch in the call")
        dx = da = db = None
        if need_x or need_a or need_b:
            plan = f8lin.LoraPlan(*ctx.sizes, buffer=buffer)
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_x else None
            da = torch.empty_like(a) if need_a else None
            db = torch.empty_like(b) if need_b else None
            f8lin.lora_backward(_rows(dy), x, a, b, scales, plan, h, dx, da, db)
        return dy if need_base else None, dx, da, db, None, None


class _InsideBackward(torch.autograd.Function):
    """Identity.  Its backward only runs where the forward that a backward made (a recomputation) is itself
    differentiated: no node of the first forward is there then to compare its batch with."""

    @staticmethod
    def forward(ctx, y):
        return y.view_as(y)

    @staticmethod
    def backward(ctx, dy):
        _refuse_unclear()


def _refuse_unclear():
    raise RuntimeError("low-rank adapters were recomputed inside a backward with a batch that need not be their forward's: "
                       "use checkpoint(..., use_reentrant=False), or pass a LoraBatch in the call that is not updated")


def _inside_backward() -> bool:
    """Whether this is a forward under autograd inside a backward pass: a recomputation."""
    return torch._C._current_graph_task_id() != -1 and torch.is_grad_enabled()


def _unclear(y: torch.Tensor) -> torch.Tensor:
    """y of a recomputation whose batch is not known to be the forward's; refused where no node can find out."""
    if not y.requires_grad:
        _refuse_unclear()
    return _InsideBackward.apply(y)


def lora_add(base: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, batch: LoraBatch,
             scales: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A shared projection's output with each token's low-rank adapter added:
        y[t] = base[t] + scales[i] * (x[t] . a[i]^T) . b[i]^T     for a token t of adapter i, base[t] without one.

    base (..., N) and x (..., K) with batch.tokens tokens; a (adapters, rank, K), b (adapters, N, rank); all of one
    dtype.  scales: float32 (adapters) or None (1), outside the graph.  Differentiable once in base, x, a and b (an
    adapter that no token uses gets a gradient of zero); forward-mode derivatives are refused (NotImplementedError).
    The order of a token's sums depends on the batch it comes in, within their rounding; the same batch gives the same
    bits."""
    if not x.is_cuda:
        raise RuntimeError("lora_add runs on the GPU only (libf8lin has no CPU path)")
    sx, sb = x.shape, base.shape
    if len(sx) < 1 or len(sb) != len(sx) or sb[:-1] != sx[:-1] or b.dim() != 3 or sb[-1] != b.shape[1]:
        raise ValueError(f"base must be x's tokens by the adapters' N, got {tuple(sb)} beside {tuple(sx)} and "
                         f"{tuple(b.shape)}")
    if scales is not None and scales.requires_grad:
        raise ValueError("scales take no part in the graph: detach them")
    base2, x2 = base, x
    if len(sx) != 2 and not (x.numel() and base.numel()):
        # (an empty last dimension leaves reshape nothing to infer the rows from)
        tokens = sx[:-1].numel()
        base2, x2 = base.reshape(tokens, sb[-1]), x.reshape(tokens, sx[-1])
    base2, x2 = _rows(base2), _rows(x2)
    if _needs_graph(base, x, a, b):
        y = _LoraAddFn.apply(base2, x2, a, b, batch.plan, scales)
    else:
        _refuse_tangents("lora_add", base, x, a, b, scales)
        y = _lora_forward(base2, x2, a if a.is_contiguous() else a.contiguous(),
                          b if b.is_contiguous() else b.contiguous(), batch.plan, scales, False)[0]
    if batch.plan.writes > 1 and _inside_backward():
        y = _unclear(y)
    return y if len(sx) == 2 else y.reshape(sb)


_SET = object()  # the batch that is set on the layer


class LoraLinear(nn.Module):
    """A linear layer with low-rank adapters beside it: base(x), then lora_add for the batch in the call, or else the one
    set in `batch` (a LoraBatch; None: the base alone).  A batch in the call belongs to that call: threads that serve one
    model at once, and what is recomputed in a backward after another batch was set, need it there.  Under activation
    checkpointing a layer whose set batch is another one by then raises RuntimeError (with use_reentrant=True, which
    leaves nothing to compare, any set batch does).

    base: nn.Linear, Float8Linear or MXFP4Linear (also a frozen one, for serving).  lora_a starts random and lora_b at
    zero, so that a new adapter adds nothing.  They are kept in `dtype` (default: the weight's, bfloat16 beside a frozen
    one) and used in the base output's."""

    def __init__(self, base: nn.Module, adapters: int, rank: int, scale: float = 1.0, dtype: Optional[torch.dtype] = None):
        super().__init__()
        if not 1 <= adapters <= f8lin.LORA_MAX_ADAPTERS or not 1 <= rank <= f8lin.LORA_MAX_RANK:
            raise ValueError(f"adapters must be 1 to {f8lin.LORA_MAX_ADAPTERS} and rank 1 to {f8lin.LORA_MAX_RANK}, got "
                             f"{adapters} and {rank}")
        self.base, self.adapters, self.rank = base, adapters, rank
        self.in_features, self.out_features = base.in_features, base.out_features
        weight = base.weight if base.weight is not None else base.weight_codes
        if dtype is None:
            dtype = weight.dtype if weight.is_floating_point() else torch.bfloat16
        a = torch.empty((adapters, rank, self.in_features), dtype=dtype, device=weight.device)
        self.lora_a = nn.Parameter(a.normal_(std=self.in_features ** -0.5))
        self.lora_b = nn.Parameter(torch.zeros((adapters, self.out_features, rank), dtype=dtype, device=weight.device))
        self.register_buffer("lora_scales", torch.full((adapters,), scale, dtype=torch.float32, device=weight.device))

    _batch: Optional[LoraBatch] = None
    _had_batch = False

    @property
    def batch(self) -> Optional[LoraBatch]:
        return self._batch

    @batch.setter
    def batch(self, batch: Optional[LoraBatch]) -> None:
        self._batch = batch
        self._had_batch = self._had_batch or batch is not None

    def forward(self, x: torch.Tensor, batch=_SET) -> torch.Tensor:
        unclear = batch is _SET and self._had_batch and _inside_backward()
        if batch is _SET:
            batch = self._batch
        y = self.base(x)
        if batch is not None:
            # (casting the module casts its scales too)
            y = lora_add(y, x.to(y.dtype), self.lora_a.to(y.dtype), self.lora_b.to(y.dtype), batch,
                         self.lora_scales.float())
        return _unclear(y) if unclear else y

    def extra_repr(self):
        return f"adapters={self.adapters}, rank={self.rank}"


def convert_to_lora(module: nn.Module, adapters: int, rank: int, scale: float = 1.0, module_filter_fn=None) -> nn.Module:
    """Puts adapters beside every nn.Linear, Float8Linear and MXFP4Linear (that module_filter_fn(fqn, module) accepts, if
    given) and takes that layer's own parameters out of training.  A linear that stands in several places has one set of
    adapters.  Returns the module."""
    kinds = (nn.Linear, Float8Linear, MXFP4Linear)
    if type(module) in kinds:
        raise ValueError("convert the parent module, not a bare linear")
    return _swap(module, lambda m: type(m) in kinds,
                 lambda m: LoraLinear(m.requires_grad_(False), adapters, rank, scale), module_filter_fn)


def set_lora_batch(module: nn.Module, batch: Optional[LoraBatch]) -> None:
    """The batch that every LoraLinear of the module serves next, where the call brings none (None: the bases alone)."""
    for m in module.modules():
        if isinstance(m, LoraLinear):
            m.batch = batch
