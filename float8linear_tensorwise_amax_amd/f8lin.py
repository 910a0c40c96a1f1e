"""Thin Python binding of libf8lin.so (include/f8lin.h), same names as the C ABI.

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  PyTorch supplies device memory (tensors) and streams; this module
checks dtypes / devices / contiguity, passes raw pointers and the current HIP
stream, and raises F8linError on a non-zero status.  Importing it fails
loudly if the library is not built -- there is no fallback.  Outputs are
written behind autograd's back: only grad_norm and grad_clip, whose tensors
are gradients, move the version counters of what they write.
"""
import array
import ctypes
import functools
import itertools
import math
import os
import struct
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libf8lin.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                      "from the repository root")

_lib = ctypes.CDLL(LIB_PATH)

E4M3 = 0
E5M2 = 1
AMAX_ATOMIC = 0
AMAX_TWOPASS = 1
DYNAMIC = 0
DELAYED = 1
HISTORY_LEN = 16

_FMT = {"e4m3": E4M3, "e5m2": E5M2, E4M3: E4M3, E5M2: E5M2}
_ALGO = {"atomic": AMAX_ATOMIC, "twopass": AMAX_TWOPASS, AMAX_ATOMIC: AMAX_ATOMIC, AMAX_TWOPASS: AMAX_TWOPASS}
_MODE = {"dynamic": DYNAMIC, "delayed": DELAYED, DYNAMIC: DYNAMIC, DELAYED: DELAYED}

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int


class State(ctypes.Structure):
    _fields_ = [("amax", _vp), ("scale", _vp), ("history", _vp), ("hist_meta", _vp)]


class GemmDesc(ctypes.Structure):
    _fields_ = [("a", _vp), ("b", _vp), ("inv_scale_a", _vp), ("inv_scale_b", _vp), ("c", _vp),
                ("M", _i64), ("N", _i64), ("K", _i64), ("lda", _i64), ("ldb", _i64)]


MAX_BATCH = 4


class FwdArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("x", _vp), ("w", _vp), ("y", _vp),
                ("x8", _vp), ("x8t", _vp), ("w8", _vp), ("w8t", _vp), ("sx", State), ("sw", State),
                ("mode_x", _int), ("mode_w", _int), ("algo", _int), ("ws", _vp), ("ws_bytes", ctypes.c_size_t),
                ("bias", _vp), ("w_cast_valid", _int), ("ev_gemm_begin", _vp), ("ev_gemm_end", _vp),
                ("y_amax", _vp), ("x_amax_given", _int)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("dy", _vp), ("x8t", _vp), ("w8t", _vp),
                ("dx", _vp), ("dw", _vp), ("dy8", _vp), ("dy8t", _vp), ("sx", State), ("sw", State),
                ("sdy", State), ("mode_dy", _int), ("algo", _int), ("ws", _vp), ("ws_bytes", ctypes.c_size_t),
                ("dbias", _vp), ("dbias_ws", _vp), ("dbias_ws_bytes", ctypes.c_size_t), ("gemm_ws", _vp),
                ("gemm_ws_bytes", ctypes.c_size_t), ("ev_gemm_begin", _vp), ("ev_gemm_end", _vp),
                ("dx_amax", _vp), ("dy_amax_given", _int)]


_lib.f8lin_transposed_ld.argtypes = [_i64]
_lib.f8lin_transposed_ld.restype = _i64
_lib.f8lin_workspace_bytes.argtypes = []
_lib.f8lin_workspace_bytes.restype = ctypes.c_size_t
_lib.f8lin_dbias_workspace_bytes.argtypes = [_i64, _i64]
_lib.f8lin_dbias_workspace_bytes.restype = ctypes.c_size_t
_lib.f8lin_backward_gemm_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.f8lin_backward_gemm_workspace_bytes.restype = ctypes.c_size_t
_lib.f8lin_status_str.argtypes = [_int]
_lib.f8lin_status_str.restype = ctypes.c_char_p
_lib.f8lin_amax.argtypes = [_vp, _i64, _int, _vp, _vp, ctypes.c_size_t, _vp]
_lib.f8lin_cast_transpose.argtypes = [_vp, _i64, _i64, _int, _int, ctypes.POINTER(State), _vp, _vp, _vp]
_lib.f8lin_cast_f32.argtypes = [_vp, _i64, _int, _vp, _vp]
_lib.f8lin_gemm.argtypes = [_vp, _int, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
_lib.f8lin_gemm_batch.argtypes = [ctypes.POINTER(GemmDesc), _int, _int, _int, _vp]
_lib.f8lin_forward.argtypes = [ctypes.POINTER(FwdArgs), _vp]
_lib.f8lin_forward_shared_x.argtypes = [ctypes.POINTER(FwdArgs), _int, _vp]
_lib.f8lin_backward.argtypes = [ctypes.POINTER(BwdArgs), _vp]
_lib.f8lin_backward_noalloc.argtypes = [ctypes.POINTER(BwdArgs), _vp]
_lib.f8lin_delayed_update.argtypes = [ctypes.POINTER(State), _int, _vp, _vp]
for _name in ("f8lin_amax", "f8lin_cast_transpose", "f8lin_cast_f32", "f8lin_gemm", "f8lin_forward",
              "f8lin_backward", "f8lin_backward_noalloc", "f8lin_delayed_update"):
    getattr(_lib, _name).restype = _int


class F8linError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(_lib.f8lin_status_str(status).decode())


def _check(status: int):
    if status != 0:
        raise F8linError(status)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor], dtype=None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("f8lin: tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("f8lin: tensors must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"f8lin: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def transposed_ld(rows: int) -> int:
    """Row stride (bytes) of the transposed fp8 copy of a tensor with `rows` rows."""
    return int(_lib.f8lin_transposed_ld(rows))


def new_transposed(cols: int, rows: int, device="cuda") -> torch.Tensor:
    """A (cols, rows) uint8 tensor laid out as the library's transposed copies
    are: a view into a (cols, transposed_ld(rows)) buffer (uninitialised)."""
    ld = transposed_ld(rows)
    buf = torch.empty((cols, ld), dtype=torch.uint8, device=device)
    return buf[:, :rows] if ld != rows else buf


def _ptr_t(t: Optional[torch.Tensor]) -> Optional[int]:
    """Pointer of a transposed fp8 copy: a (cols, rows) uint8 tensor whose rows
    are transposed_ld(rows) bytes apart (see new_transposed)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("f8lin: tensors must be on the GPU")
    if t.dtype != torch.uint8 or t.dim() != 2:
        raise TypeError("f8lin: a transposed fp8 copy is a 2-D uint8 tensor")
    if t.numel() > 0 and (t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) != transposed_ld(t.shape[1]))):
        raise ValueError(f"f8lin: a transposed copy with rows of {t.shape[1]} codes needs a row stride of "
                         f"{transposed_ld(t.shape[1])} bytes (allocate it with new_transposed)")
    return t.data_ptr()


def _ptr_ld(t: torch.Tensor):
    """(pointer, row stride) of a 2-D uint8 GEMM operand whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("f8lin: tensors must be on the GPU")
    if t.dtype != torch.uint8 or t.dim() != 2 or (t.numel() > 0 and t.stride(1) != 1):
        raise TypeError("f8lin: a GEMM operand is a 2-D uint8 tensor with contiguous rows")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def workspace_bytes() -> int:
    return int(_lib.f8lin_workspace_bytes())


def dbias_workspace_bytes(M: int, N: int) -> int:
    return int(_lib.f8lin_dbias_workspace_bytes(M, N))


def backward_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.f8lin_backward_gemm_workspace_bytes(M, N, K))


def new_backward_gemm_workspace(M: int, N: int, K: int, device="cuda") -> Optional[torch.Tensor]:
    """Scratch for split backward GEMMs (uninitialised), or None when no GEMM of this shape splits."""
    n = backward_gemm_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def new_dbias_workspace(M: int, N: int, device="cuda") -> torch.Tensor:
    """Scratch (float32, no initialisation needed) for the bias gradient of an (M, N) dY."""
    return torch.empty(max(1, dbias_workspace_bytes(M, N) // 4), dtype=torch.float32, device=device)


def status_str(status: int) -> str:
    return _lib.f8lin_status_str(status).decode()


def new_workspace(device="cuda") -> torch.Tensor:
    """A zero-filled workspace (uint8) of workspace_bytes()."""
    return torch.zeros(workspace_bytes(), dtype=torch.uint8, device=device)


class ScalingState:
    """Device-resident scaling state of one tensor role (f8lin_state):
    amax [1] f32, scale [2] f32 = {scale, 1/scale}, history [16] f32,
    hist_meta [2] i32 = {count, pos}; all zero-initialised."""

    def __init__(self, device="cuda", tensors=None):
        """tensors: optional (amax, scale, history, hist_meta) tensors to wrap
        instead of allocating new ones (e.g. a module's buffers)."""
        if tensors is not None:
            self.amax, self.scale, self.history, self.hist_meta = tensors
            return
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.scale = torch.zeros(2, dtype=torch.float32, device=device)
        self.history = torch.zeros(HISTORY_LEN, dtype=torch.float32, device=device)
        self.hist_meta = torch.zeros(2, dtype=torch.int32, device=device)

    def c_struct(self) -> State:
        return State(self.amax.data_ptr(), self.scale.data_ptr(), self.history.data_ptr(), self.hist_meta.data_ptr())

    @property
    def inv_scale(self) -> torch.Tensor:
        return self.scale[1:2]

    def state_dict(self):
        """Host copies of the state (for checkpointing)."""
        return {k: getattr(self, k).detach().cpu().clone() for k in ("amax", "scale", "history", "hist_meta")}

    def load_state_dict(self, sd):
        for k in ("amax", "scale", "history", "hist_meta"):
            getattr(self, k).copy_(sd[k])


class ScaleView:
    """A state that only carries {scale, 1/scale} (what backward reads of the
    forward's X and W states), e.g. a snapshot taken at forward time."""

    def __init__(self, scale: torch.Tensor):
        if scale.numel() != 2 or scale.dtype != torch.float32 or not scale.is_contiguous():
            raise ValueError("ScaleView needs a contiguous float32 tensor of 2 elements")
        self.scale = scale

    def c_struct(self) -> State:
        return State(None, self.scale.data_ptr(), None, None)


# ----------------------------------------------------------------- entry points

def amax(x: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, algo="atomic", stream=None):
    _check(_lib.f8lin_amax(_ptr(x, torch.bfloat16), x.numel(), _ALGO[algo], _ptr(out, torch.float32),
                           _ptr(ws), _nbytes(ws), _stream(stream)))


def cast_transpose(x: torch.Tensor, fmt, mode, state: ScalingState, q: torch.Tensor,
                   qt: Optional[torch.Tensor] = None, stream=None):
    if x.dim() != 2:
        raise ValueError("cast_transpose takes a 2-D tensor")
    st = state.c_struct()
    _check(_lib.f8lin_cast_transpose(_ptr(x, torch.bfloat16), x.shape[0], x.shape[1], _FMT[fmt], _MODE[mode],
                                     ctypes.byref(st), _ptr(q, torch.uint8), _ptr_t(qt), _stream(stream)))


def cast_f32(v: torch.Tensor, fmt, q: torch.Tensor, stream=None):
    _check(_lib.f8lin_cast_f32(_ptr(v, torch.float32), v.numel(), _FMT[fmt], _ptr(q, torch.uint8),
                               _stream(stream)))


def gemm(a: torch.Tensor, fmt_a, b: torch.Tensor, fmt_b, inv_a: torch.Tensor, inv_b: torch.Tensor,
         c: torch.Tensor, stream=None):
    """c (M, N) bf16 = a (M, K) . b (N, K)^T * inv_a[0] * inv_b[0]."""
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K or tuple(c.shape) != (M, N):
        raise ValueError("gemm: shape mismatch")
    _check(_lib.f8lin_gemm(_ptr(a, torch.uint8), _FMT[fmt_a], _ptr(b, torch.uint8), _FMT[fmt_b], M, N, K,
                           _ptr(inv_a, torch.float32), _ptr(inv_b, torch.float32), _ptr(c, torch.bfloat16),
                           _stream(stream)))


def gemm_batch(items, fmt_a, fmt_b, stream=None):
    """Up to MAX_BATCH GEMMs in one launch; items: (a, b, inv_a, inv_b, c) tuples
    as for gemm(), all with the operand formats fmt_a / fmt_b."""
    arr = (GemmDesc * max(1, len(items)))()
    for i, (a, b, inv_a, inv_b, c) in enumerate(items):
        M, K = a.shape
        N = b.shape[0]
        if b.shape[1] != K or tuple(c.shape) != (M, N):
            raise ValueError("gemm_batch: shape mismatch")
        pa, lda = _ptr_ld(a)
        pb, ldb = _ptr_ld(b)
        arr[i] = GemmDesc(pa, pb, _ptr(inv_a, torch.float32), _ptr(inv_b, torch.float32), _ptr(c, torch.bfloat16),
                          M, N, K, lda, ldb)
    _check(_lib.f8lin_gemm_batch(arr, len(items), _FMT[fmt_a], _FMT[fmt_b], _stream(stream)))


def _event(ev) -> Optional[int]:
    """Raw hipEvent_t of a torch.cuda.Event (created by recording it once), or None."""
    if ev is None:
        return None
    if not ev.cuda_event:
        ev.record()
    return ev.cuda_event


def _amax_word(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() < 1:
        raise TypeError("f8lin: an amax output is a float32 tensor")
    return _ptr(t)


def _fwd_args(x, w, y, x8, x8t, w8, w8t, sx, sw, ws, mode_x, mode_w, algo, bias, w_cast_valid, gemm_events=None,
              y_amax=None, x_amax_given=False):
    M, K = x.shape
    N = w8.shape[0]
    if (w is not None and tuple(w.shape) != (N, K)) or tuple(w8.shape) != (N, K) or tuple(y.shape) != (M, N):
        raise ValueError("forward: shape mismatch")
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError("forward: bias must have shape (N,)")
    ev0, ev1 = (None, None) if gemm_events is None else gemm_events
    return FwdArgs(M, N, K, _ptr(x, torch.bfloat16), _ptr(w, torch.bfloat16), _ptr(y, torch.bfloat16),
                   _ptr(x8, torch.uint8), _ptr_t(x8t), _ptr(w8, torch.uint8), _ptr_t(w8t),
                   sx.c_struct(), sw.c_struct(), _MODE[mode_x], _MODE[mode_w], _ALGO[algo], _ptr(ws),
                   _nbytes(ws), None if bias is None else _ptr(bias, torch.bfloat16),
                   1 if w_cast_valid else 0, _event(ev0), _event(ev1), _amax_word(y_amax),
                   1 if x_amax_given else 0)


def forward(x, w, y, x8, x8t, w8, w8t, sx: ScalingState, sw: ScalingState, ws, mode_x="dynamic",
            mode_w="dynamic", algo="atomic", stream=None, bias=None, w_cast_valid=False, gemm_events=None,
            y_amax=None, x_amax_given=False):
    """w_cast_valid: w8, w8t and sw's scale already hold W's cast (unchanged
    weight); W's amax and cast are skipped and w may be None.
    gemm_events: optional (begin, end) torch.cuda.Event pair recorded around
    the call's GEMM launch.  y_amax: optional float32 tensor that receives
    amax(Y) from the GEMM epilogue.  x_amax_given: sx.amax already holds
    amax(X) (dynamic mode), so X's amax pass is skipped."""
    a = _fwd_args(x, w, y, x8, x8t, w8, w8t, sx, sw, ws, mode_x, mode_w, algo, bias, w_cast_valid, gemm_events,
                  y_amax, x_amax_given)
    _check(_lib.f8lin_forward(ctypes.byref(a), _stream(stream)))


def forward_shared_x(x, x8, x8t, sx: ScalingState, ws, linears, mode_x="dynamic", algo="atomic", stream=None,
                     gemm_events=None, x_amax_given=False):
    """Linears reading the same X: linears is a list of dicts with keys w, y,
    w8, w8t, sw and optionally mode_w, bias, w_cast_valid, y_amax.  X is cast
    once; the GEMMs share one launch."""
    arr = (FwdArgs * max(1, len(linears)))()
    for i, l in enumerate(linears):
        arr[i] = _fwd_args(x, l.get("w"), l["y"], x8, x8t, l["w8"], l["w8t"], sx, l["sw"], ws, mode_x,
                           l.get("mode_w", "dynamic"), algo, l.get("bias"), l.get("w_cast_valid", False),
                           gemm_events, l.get("y_amax"), x_amax_given)
    _check(_lib.f8lin_forward_shared_x(arr, len(linears), _stream(stream)))


def backward(dy, x8t, w8t, dx, dw, dy8, dy8t, sx: ScalingState, sw: ScalingState, sdy: ScalingState, ws,
             mode_dy="dynamic", algo="atomic", stream=None, dbias=None, dbias_ws=None, gemm_ws=None,
             gemm_events=None, dx_amax=None, dy_amax_given=False):
    """gemm_ws: optional scratch (backward_gemm_workspace_bytes(M, N, K) bytes) with which GEMMs that have
    few output tiles and a long contraction run split along K.  gemm_events, dx_amax, dy_amax_given: as
    forward's gemm_events, y_amax, x_amax_given, for the dgrad + wgrad launch, dX and dY."""
    M, N = dy.shape
    K = x8t.shape[0]
    if tuple(dx.shape) != (M, K) or tuple(dw.shape) != (N, K) or tuple(w8t.shape) != (K, N):
        raise ValueError("backward: shape mismatch")
    if dbias is not None and tuple(dbias.shape) != (N,):
        raise ValueError("backward: dbias must have shape (N,)")
    a = BwdArgs(M, N, K, _ptr(dy, torch.bfloat16), _ptr_t(x8t), _ptr_t(w8t),
                _ptr(dx, torch.bfloat16), _ptr(dw, torch.bfloat16), _ptr(dy8, torch.uint8), _ptr_t(dy8t),
                sx.c_struct(), sw.c_struct(), sdy.c_struct(), _MODE[mode_dy], _ALGO[algo], _ptr(ws),
                _nbytes(ws), None if dbias is None else _ptr(dbias, torch.bfloat16),
                None if dbias_ws is None else _ptr(dbias_ws, torch.float32),
                0 if dbias_ws is None else dbias_ws.numel() * 4, _ptr(gemm_ws), _nbytes(gemm_ws),
                *((None, None) if gemm_events is None else (_event(gemm_events[0]), _event(gemm_events[1]))),
                _amax_word(dx_amax), 1 if dy_amax_given else 0)
    _check(_lib.f8lin_backward(ctypes.byref(a), _stream(stream)))


def backward_noalloc(dy, x8t, w8t, dx, dw, dy8, dy8t, sx: ScalingState, sw: ScalingState, sdy: ScalingState,
                     mode_dy="dynamic", algo="atomic", stream=None, dbias=None, gemm_events=None, dx_amax=None,
                     dy_amax_given=False):
    """backward() for callers that cannot allocate: no workspace, bias-gradient
    scratch or split scratch is passed; the library's static per-device scratch
    (8 KB + 16 MiB) takes their place.  Calls that overlap in time on one GPU race."""
    M, N = dy.shape
    K = x8t.shape[0]
    if tuple(dx.shape) != (M, K) or tuple(dw.shape) != (N, K) or tuple(w8t.shape) != (K, N):
        raise ValueError("backward_noalloc: shape mismatch")
    if dbias is not None and tuple(dbias.shape) != (N,):
        raise ValueError("backward_noalloc: dbias must have shape (N,)")
    a = BwdArgs(M, N, K, _ptr(dy, torch.bfloat16), _ptr_t(x8t), _ptr_t(w8t),
                _ptr(dx, torch.bfloat16), _ptr(dw, torch.bfloat16), _ptr(dy8, torch.uint8), _ptr_t(dy8t),
                sx.c_struct(), sw.c_struct(), sdy.c_struct(), _MODE[mode_dy], _ALGO[algo], None, 0,
                None if dbias is None else _ptr(dbias, torch.bfloat16), None, 0, None, 0,
                *((None, None) if gemm_events is None else (_event(gemm_events[0]), _event(gemm_events[1]))),
                _amax_word(dx_amax), 1 if dy_amax_given else 0)
    _check(_lib.f8lin_backward_noalloc(ctypes.byref(a), _stream(stream)))


NOALLOC_REGION_BYTES = 16 << 20  # the static scratch's region for bias-gradient sums and split partials


def delayed_update(states: Sequence[ScalingState], stream=None, status: Optional[torch.Tensor] = None):
    """status: optional int32 device tensor of len(states); entry i becomes 0
    when state i was updated and 1 (F8LIN_EINVAL) when its {count, pos} was
    not a reachable one, in which case that state is left untouched."""
    arr = (State * max(1, len(states)))(*[s.c_struct() for s in states])
    if status is not None and (status.dtype != torch.int32 or status.numel() < len(states)):
        raise ValueError("delayed_update: status must be an int32 tensor of at least len(states) entries")
    _check(_lib.f8lin_delayed_update(arr, len(states), _ptr(status), _stream(stream)))


# ------------------------------------------------------------ layer buffers

class LinearBuffers:
    """Every device buffer one Float8Linear forward + backward needs, for
    X (M, K), W (N, K), dY (M, N); allocated once with torch (plumbing)."""

    def __init__(self, M: int, N: int, K: int, device="cuda", with_bias: bool = False):
        u8 = dict(dtype=torch.uint8, device=device)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.M, self.N, self.K = M, N, K
        self.y = torch.empty((M, N), **bf)
        self.dx = torch.empty((M, K), **bf)
        self.dw = torch.empty((N, K), **bf)
        self.x8 = torch.empty((M, K), **u8)
        self.x8t = new_transposed(K, M, device)
        self.w8 = torch.empty((N, K), **u8)
        self.w8t = new_transposed(K, N, device)
        self.dy8 = torch.empty((M, N), **u8)
        self.dy8t = new_transposed(N, M, device)
        self.sx = ScalingState(device)
        self.sw = ScalingState(device)
        self.sdy = ScalingState(device)
        self.ws = new_workspace(device)
        self.dbias = torch.empty((N,), **bf) if with_bias else None
        self.dbias_ws = new_dbias_workspace(M, N, device) if with_bias else None
        self.gemm_ws = new_backward_gemm_workspace(M, N, K, device)

    def forward(self, x, w, mode="dynamic", algo="atomic", stream=None, bias=None, gemm_events=None):
        forward(x, w, self.y, self.x8, self.x8t, self.w8, self.w8t, self.sx, self.sw, self.ws, mode, mode, algo,
                stream, bias, gemm_events=gemm_events)
        return self.y

    def backward(self, dy, mode="dynamic", algo="atomic", stream=None, gemm_events=None):
        backward(dy, self.x8t, self.w8t, self.dx, self.dw, self.dy8, self.dy8t, self.sx, self.sw, self.sdy,
                 self.ws, mode, algo, stream, self.dbias, self.dbias_ws, self.gemm_ws, gemm_events=gemm_events)
        return self.dx, self.dw

    def states(self):
        return [self.sx, self.sw, self.sdy]


# ------------------------------------------------------------------- MXFP4

MX_FLOOR = 0
MX_CEIL = 1
_RULE = {"floor": MX_FLOOR, "ceil": MX_CEIL, MX_FLOOR: MX_FLOOR, MX_CEIL: MX_CEIL}
_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MXFP4_BLOCK = 32


class MxStruct(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("ld", _i64), ("scale_ld", _i64)]


class MxGemmDesc(ctypes.Structure):
    _fields_ = [("a", MxStruct), ("b", MxStruct), ("c", _vp), ("bias", _vp), ("M", _i64), ("N", _i64), ("K", _i64),
                ("c_dtype", _int), ("bias_dtype", _int)]


class MxFwdArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("x", _vp), ("w", _vp), ("ldx", _i64), ("y", _vp),
                ("bias", _vp), ("x_dtype", _int), ("w_dtype", _int), ("y_dtype", _int), ("bias_dtype", _int),
                ("x4", MxStruct), ("x4t", MxStruct), ("w4", MxStruct), ("w4t", MxStruct), ("rule", _int)]


class MxBwdArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("dy", _vp), ("lddy", _i64), ("dx", _vp), ("dw", _vp),
                ("dbias", _vp), ("dy_dtype", _int), ("dx_dtype", _int), ("dw_dtype", _int), ("dbias_dtype", _int),
                ("x4t", MxStruct), ("w4t", MxStruct), ("dy4", MxStruct), ("dy4t", MxStruct), ("rule", _int),
                ("dbias_ws", _vp), ("dbias_ws_bytes", ctypes.c_size_t)]


class Grad(ctypes.Structure):
    _fields_ = [("g", _vp), ("out", _vp), ("n", _i64), ("dtype", _int), ("out_dtype", _int)]


_lib.f8lin_mxfp4_ld.argtypes = [_i64]
_lib.f8lin_mxfp4_ld.restype = _i64
_lib.f8lin_mxfp4_scale_ld.argtypes = [_i64]
_lib.f8lin_mxfp4_scale_ld.restype = _i64
_lib.f8lin_mxfp4_quantize.argtypes = [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _vp]
_lib.f8lin_mxfp4_dequantize.argtypes = [_vp, _i64, _i64, _int, _vp, _vp]
_lib.f8lin_mxfp4_gemm.argtypes = [_vp, _int, _vp]
_lib.f8lin_mxfp4_forward.argtypes = [_vp, _vp]
_lib.f8lin_mxfp4_forward_fused.argtypes = [_i64, _i64, _i64]
_lib.f8lin_mxfp4_forward_fused.restype = _int
_lib.f8lin_mxfp4_backward.argtypes = [_vp, _vp]
_lib.f8lin_mxfp4_dbias_workspace_bytes.argtypes = [_i64, _i64]
_lib.f8lin_mxfp4_dbias_workspace_bytes.restype = ctypes.c_size_t
_lib.f8lin_grad_workspace_bytes.argtypes = []
_lib.f8lin_grad_workspace_bytes.restype = ctypes.c_size_t
_lib.f8lin_grad_norm.argtypes = [_vp, _int, _int, _vp, _vp, ctypes.c_size_t, _vp]
_lib.f8lin_grad_clip.argtypes = [_vp, _int, _int, ctypes.c_float, _vp, _int, _vp, ctypes.c_size_t, _vp]
for _name in ("f8lin_mxfp4_quantize", "f8lin_mxfp4_dequantize", "f8lin_mxfp4_gemm", "f8lin_mxfp4_forward",
              "f8lin_mxfp4_backward", "f8lin_grad_norm", "f8lin_grad_clip"):
    getattr(_lib, _name).restype = _int


# The argument structures as bytes: packing one costs a fraction of filling a ctypes.Structure field by field.
_MX = struct.Struct("@4q")
_MX_FWD = struct.Struct("@8q4i16qi4x")
_MX_BWD = struct.Struct("@8q4i16qi4x2q")
for _fmt, _cls in ((_MX, MxStruct), (_MX_FWD, MxFwdArgs), (_MX_BWD, MxBwdArgs)):
    assert _fmt.size == ctypes.sizeof(_cls)


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current hipStream_t of a device, without a Stream object
_current_device = torch._C._cuda_getDevice


def _call(fn, device: torch.device, stream, *args):
    """Calls fn(*args, stream) with `device` current: the stream is the given one, or the device's current one."""
    index = device.index
    raw = _raw_stream(index) if stream is None else _stream(stream)
    if index == _current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        raise F8linError(status)


def _stream_object(stream, device: torch.device) -> torch.cuda.Stream:
    """The stream as an object that torch allocates under (ExternalStream would take a handle of 0 for no stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = _stream(stream)
    return torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)


def _refuse(t: torch.Tensor, what: str, device: Optional[torch.device]):
    if not t.is_cuda:
        raise ValueError("f8lin: tensors must be on the GPU")
    if device is not None and t.device != device:
        raise ValueError(f"f8lin: {what} is on {t.device}, expected {device}")
    if t.dtype not in _DTYPE:
        raise TypeError(f"f8lin: {what} must be bfloat16, float16 or float32, got {t.dtype}")


def _same_device(t: Optional[torch.Tensor], what: str, device: torch.device):
    if t is not None and t.device != device:
        raise ValueError(f"f8lin: {what} is on {t.device}, expected {device}")


def _dense(t: torch.Tensor, what: str, device: Optional[torch.device] = None) -> int:
    """Pointer of a contiguous bf16 / fp16 / fp32 GPU tensor (on `device`, if given)."""
    if not t.is_cuda or t.dtype not in _DTYPE or (device is not None and t.device != device):
        _refuse(t, what, device)
    if not t.is_contiguous():
        raise ValueError(f"f8lin: {what} must be contiguous")
    return t.data_ptr()


def _dense_ld(t: torch.Tensor, what: str, device: Optional[torch.device] = None):
    """(pointer, row stride in elements) of a 2-D bf16 / fp16 / fp32 tensor whose rows are contiguous."""
    if t.is_contiguous():
        return _dense(t, what, device), t.shape[1]
    _refuse(t, what, device)
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if t.numel() and ((cols > 1 and t.stride(1) != 1) or ld < cols):
        raise ValueError(f"f8lin: {what}'s rows must be contiguous and must not overlap")
    return t.data_ptr(), max(ld, cols)


class MXFP4Tensor:
    """A (rows, cols) tensor of 4-bit codes with one 8-bit scale per 32
    consecutive elements of a row (f8lin_mxfp4).

    codes  (rows, >= 16 * ceil(cols / 32)) uint8: two e2m1 codes a byte, the even element in its low half; the
           codes past cols in the last block are zero
    scales (rows, >= ceil(cols / 32) rounded up to 16) uint8: e8m0, 2^(byte - 127), 255 for NaN
    Both with contiguous rows 16 bytes aligned.  A row's codes and scales are views into what you pass."""

    __slots__ = ("_codes", "_scales", "rows", "cols", "device", "_buffer", "_at", "_c")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        nb = -(-cols // MXFP4_BLOCK)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.dim() != 2 or scales.dim() != 2:
            raise TypeError("MXFP4Tensor: codes and scales must be 2-D uint8 tensors")
        if not codes.is_cuda or scales.device != codes.device:
            raise ValueError("MXFP4Tensor: codes and scales must be on one GPU")
        self._codes, self._scales, self.rows, self.cols = codes, scales, rows, cols
        self.device, self._buffer = codes.device, None
        if rows and cols:
            (cr, cw), (sr, sw) = codes.shape, scales.shape
            sn = -(-nb // 16) * 16
            if cr != rows or sr != rows or cw < 16 * nb or sw < sn or codes.stride(1) != 1 or scales.stride(1) != 1:
                raise ValueError(f"MXFP4Tensor: a ({rows}, {cols}) tensor has codes ({rows}, >= {16 * nb}) and scales "
                                 f"({rows}, >= {sn}) with contiguous rows")
            # (a single row has no stride to speak of)
            self._c = (codes.data_ptr(), scales.data_ptr(), codes.stride(0) if rows > 1 else 16 * nb,
                       scales.stride(0) if rows > 1 else sn)
        else:
            self._c = _NO_MX

    @classmethod
    def _of(cls, buffer: torch.Tensor, at: int, rows: int, cols: int, ld: int, scale_ld: int) -> "MXFP4Tensor":
        """The tensor whose codes, then scales, lie `at` bytes into a flat buffer."""
        t = cls.__new__(cls)
        t._codes = t._scales = None
        t.rows, t.cols, t.device, t._buffer, t._at = rows, cols, buffer.device, buffer, at
        p = buffer.data_ptr() + at
        t._c = (p, p + rows * ld, ld, scale_ld)
        return t

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            n, ld, at = self.rows, self._c[2], self._at
            self._codes = self._buffer[at:at + n * ld].view(n, ld)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            n, ld, sld = self.rows, self._c[2], self._c[3]
            at = self._at + n * ld
            self._scales = self._buffer[at:at + n * sld].view(n, sld)
        return self._scales

    def dequantize(self, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
        """The values this tensor stands for, rounded to `dtype`.  A given stream owns the result's memory, as of a tensor
        made under it; the current stream may read it once it has waited for that stream."""
        if stream is None:
            out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.device)
        else:
            stream = _stream_object(stream, self.device)
            with torch.cuda.stream(stream):
                out = torch.empty((self.rows, self.cols), dtype=dtype, device=self.device)
            current = torch.cuda.current_stream(self.device)
            if stream != current:
                out.record_stream(current)
        mxfp4_dequantize(self, out, stream)
        return out


_NO_MX = (0, 0, 0, 0)


def _mx(t: Optional[MXFP4Tensor], rows: int, cols: int, what: str, device=None):
    """(codes, scales, ld, scale_ld) as f8lin_mxfp4 has them."""
    if t is None:
        return _NO_MX
    if t.rows != rows or t.cols != cols:
        raise ValueError(f"f8lin: {what} must be a ({rows}, {cols}) MXFP4 tensor, got ({t.rows}, {t.cols})")
    if device is not None and t.device != device:
        raise ValueError(f"f8lin: {what} is on {t.device}, expected {device}")
    return t._c


def new_mxfp4s(shapes, device="cuda", buffer: Optional[torch.Tensor] = None):
    """(flat buffer, [MXFP4Tensor]): uninitialised tensors of the (rows, cols) shapes, with the library's strides, in
    one allocation -- or the tensors that such a buffer (flat, contiguous, 16-byte aligned, as long or longer) holds."""
    ld, sld = _lib.f8lin_mxfp4_ld, _lib.f8lin_mxfp4_scale_ld
    laid, at = [], 0
    for rows, cols in shapes:
        a, b = ld(cols), sld(cols)
        laid.append((at, rows, cols, a, b))
        at += rows * (a + b)
    if buffer is None:
        buffer = torch.empty(at, dtype=torch.uint8, device=device)
    elif (buffer.dtype != torch.uint8 or buffer.dim() != 1 or buffer.numel() < at or not buffer.is_contiguous()
          or buffer.data_ptr() % 16):
        raise ValueError(f"new_mxfp4s: these tensors need a flat, contiguous, 16-byte aligned uint8 buffer of {at} bytes")
    return buffer, [MXFP4Tensor._of(buffer, *l) for l in laid]


def new_mxfp4(rows: int, cols: int, device="cuda") -> MXFP4Tensor:
    """An uninitialised MXFP4 tensor with the library's strides."""
    return new_mxfp4s(((rows, cols),), device)[1][0]


def mxfp4_quantize(x: torch.Tensor, q: Optional[MXFP4Tensor], qt: Optional[MXFP4Tensor] = None, rule="floor",
                   stream=None):
    """x (rows, cols) -> q (rows, cols), blocks along the rows, and / or qt (cols, rows), the transposed tensor with
    blocks along x's columns.  rule, with m a block's largest magnitude: "floor" (exponent floor(log2 m) - 2) or "ceil"
    (ceil(log2(m / 6)): nothing saturates)."""
    if x.dim() != 2:
        raise ValueError("mxfp4_quantize takes a 2-D tensor")
    rows, cols = x.shape
    p, ld = _dense_ld(x, "x")
    dev = x.device
    _call(_lib.f8lin_mxfp4_quantize, dev, stream, p, _DTYPE[x.dtype], rows, cols, ld,
          _MX.pack(*_mx(q, rows, cols, "q", dev)), _MX.pack(*_mx(qt, cols, rows, "qt", dev)), _RULE[rule])


def mxfp4_dequantize(q: MXFP4Tensor, out: torch.Tensor, stream=None):
    """out (rows, cols) = the values q stands for."""
    if tuple(out.shape) != (q.rows, q.cols):
        raise ValueError("mxfp4_dequantize: shape mismatch")
    p = _dense(out, "out", q.device)
    _call(_lib.f8lin_mxfp4_dequantize, out.device, stream, _MX.pack(*q._c), q.rows, q.cols, _DTYPE[out.dtype], p)


def mxfp4_gemm(items, stream=None):
    """One or two products c (M, N) = a (M, K) . b (N, K)^T (+ bias) in one call; items: (a, b, c) or (a, b, c, bias)
    tuples, a and b MXFP4Tensors."""
    arr = (MxGemmDesc * max(1, len(items)))()
    dev = None
    for i, item in enumerate(items):
        a, b, c = item[:3]
        bias = item[3] if len(item) > 3 else None
        M, K, N = a.rows, a.cols, b.rows
        dev = c.device if dev is None else dev
        if b.cols != K or tuple(c.shape) != (M, N) or (bias is not None and tuple(bias.shape) != (N,)):
            raise ValueError("mxfp4_gemm: shape mismatch")
        arr[i] = MxGemmDesc(MxStruct(*_mx(a, M, K, "a", dev)), MxStruct(*_mx(b, N, K, "b", dev)), _dense(c, "c", dev),
                            None if bias is None else _dense(bias, "bias", dev), M, N, K, _DTYPE[c.dtype],
                            0 if bias is None else _DTYPE[bias.dtype])
    if dev is None:
        raise ValueError("mxfp4_gemm: no products given")
    _call(_lib.f8lin_mxfp4_gemm, dev, stream, arr, len(items))


def mxfp4_forward_fused(M: int, N: int, K: int) -> bool:
    """Whether mxfp4_forward with a quantised weight can quantise X inside the product (x4 and x4t may be None)."""
    return bool(_lib.f8lin_mxfp4_forward_fused(M, N, K))


def mxfp4_forward(x, w, y, x4: Optional[MXFP4Tensor], w4: MXFP4Tensor, x4t=None, w4t=None, bias=None, rule="floor",
                  stream=None):
    """y (M, N) = x4 . w4^T (+ bias).  w (N, K): quantised into w4 (and w4t); None: w4 already holds the weight.
    x4 (and x4t, if the backward is to follow) receive X's codes; x4 may be None where mxfp4_forward_fused says so."""
    M, K = x.shape
    N = w4.rows
    dev = x.device
    if tuple(y.shape) != (M, N) or (w is not None and tuple(w.shape) != (N, K)) or \
            (bias is not None and tuple(bias.shape) != (N,)):
        raise ValueError("mxfp4_forward: shape mismatch")
    px, ldx = _dense_ld(x, "x")
    a = _MX_FWD.pack(M, N, K, px, 0 if w is None else _dense(w, "w", dev), ldx, _dense(y, "y", dev),
                     0 if bias is None else _dense(bias, "bias", dev), _DTYPE[x.dtype],
                     0 if w is None else _DTYPE[w.dtype], _DTYPE[y.dtype], 0 if bias is None else _DTYPE[bias.dtype],
                     *_mx(x4, M, K, "x4", dev), *_mx(x4t, K, M, "x4t", dev), *_mx(w4, N, K, "w4", dev),
                     *_mx(w4t, K, N, "w4t", dev), _RULE[rule])
    _call(_lib.f8lin_mxfp4_forward, dev, stream, a)


def mxfp4_dbias_workspace_bytes(M: int, N: int) -> int:
    return int(_lib.f8lin_mxfp4_dbias_workspace_bytes(M, N))


def mxfp4_backward(dy, x4t, w4t, dx, dw, dy4, dy4t, dbias=None, dbias_ws=None, rule="floor", stream=None):
    """dx (M, K), dw (N, K) and dbias (N) -- each may be None -- of the layer whose forward left x4t (K, M) and
    w4t (K, N).  dy4 (M, N; for dx) and dy4t (N, M; for dw or dbias) receive dY's two layouts; dbias_ws: float32
    scratch of mxfp4_dbias_workspace_bytes(M, N)."""
    M, N = dy.shape
    K = (dx if dx is not None else dw).shape[1] if dx is not None or dw is not None else 0
    dev = dy.device
    if (dx is not None and tuple(dx.shape) != (M, K)) or (dw is not None and tuple(dw.shape) != (N, K)) or \
            (dbias is not None and tuple(dbias.shape) != (N,)):
        raise ValueError("mxfp4_backward: shape mismatch")
    p, ld = _dense_ld(dy, "dy")
    _same_device(dbias_ws, "dbias_ws", dev)
    opt = lambda t, what: 0 if t is None else _dense(t, what, dev)  # noqa: E731
    dt = lambda t: 0 if t is None else _DTYPE[t.dtype]  # noqa: E731
    a = _MX_BWD.pack(M, N, K, p, ld, opt(dx, "dx"), opt(dw, "dw"), opt(dbias, "dbias"), _DTYPE[dy.dtype], dt(dx), dt(dw),
                     dt(dbias), *_mx(x4t if dw is not None else None, K, M, "x4t", dev),
                     *_mx(w4t if dx is not None else None, K, N, "w4t", dev), *_mx(dy4, M, N, "dy4", dev),
                     *_mx(dy4t, N, M, "dy4t", dev), _RULE[rule], _ptr(dbias_ws, torch.float32) or 0, _nbytes(dbias_ws))
    _call(_lib.f8lin_mxfp4_backward, dev, stream, a)


# --------------------------------------------------- gradient norm and clipping

_NORM = {2.0: 0, 1.0: 1, math.inf: 2}


def grad_workspace_bytes() -> int:
    return int(_lib.f8lin_grad_workspace_bytes())


def new_grad_workspace(device="cuda") -> torch.Tensor:
    """Scratch for grad_norm / grad_clip (uninitialised; one for each call that may overlap another in time)."""
    return torch.empty(grad_workspace_bytes(), dtype=torch.uint8, device=device)


def _is_dense(t: torch.Tensor) -> bool:
    """Whether t covers numel() consecutive elements of memory exactly once, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != want:
            return False
        want *= size
    return True


def _norm_type(norm_type) -> int:
    code = _NORM.get(float(norm_type))
    if code is None:
        raise ValueError(f"f8lin: norm_type must be 2, 1 or inf, got {norm_type!r}")
    return code


def _grad_table(grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]], device: torch.device):
    """The list as the C ABI takes it: four 64-bit words a tensor (g, out, n, dtype | out_dtype << 32)."""
    words: List[int] = []
    outs = grads if outs is None else outs
    if len(outs) != len(grads):
        raise ValueError("f8lin: as many outputs as gradients")
    for g, o in zip(grads, outs):
        dt, odt = _DTYPE.get(g.dtype), _DTYPE.get(o.dtype)
        if dt is None or odt is None:
            raise TypeError("f8lin: gradients must be bfloat16, float16 or float32")
        if g.device != device or o.device != device:
            raise ValueError(f"f8lin: gradients must all be on {device}")
        if g.layout is not torch.strided or not _is_dense(g) or \
                (o is not g and (o.shape != g.shape or (g.numel() > 0 and o.stride() != g.stride()))):
            raise ValueError("f8lin: gradients must be dense, and an output laid out as its gradient")
        words += (g.data_ptr(), o.data_ptr(), g.numel(), dt | odt << 32)
    return array.array("q", words)


def grad_norm(grads: Sequence[torch.Tensor], out: torch.Tensor, ws: torch.Tensor, norm_type: float = 2.0, stream=None):
    """out[0] (float32) = the norm of all gradients' elements as one vector; norm_type 2, 1 or inf."""
    code = _norm_type(norm_type)
    tab = _grad_table(grads, None, out.device)
    _same_device(ws, "ws", out.device)
    _call(_lib.f8lin_grad_norm, out.device, stream, tab.buffer_info()[0], len(grads), code,
          _ptr(out, torch.float32), _ptr(ws), _nbytes(ws))
    torch.autograd.graph.increment_version(out)


def grad_clip(grads: Sequence[torch.Tensor], max_norm: float, norm: torch.Tensor, ws: Optional[torch.Tensor],
              norm_type: float = 2.0, outs: Optional[Sequence[torch.Tensor]] = None, norm_given: bool = False,
              stream=None):
    """norm[0] (float32) = the norm as grad_norm gives it (norm_given: it is read instead), then every gradient times
    min(1, max_norm / (norm + 1e-6)), in place or into outs (laid out alike; any of the three types).  max_norm may be
    inf: no limit."""
    code = _norm_type(norm_type)
    tab = _grad_table(grads, outs, norm.device)
    _same_device(ws, "ws", norm.device)
    _call(_lib.f8lin_grad_clip, norm.device, stream, tab.buffer_info()[0], len(grads), code, float(max_norm),
          _ptr(norm, torch.float32), 1 if norm_given else 0, _ptr(ws), _nbytes(ws))
    written = list(grads if outs is None else outs)
    torch.autograd.graph.increment_version(written if norm_given else written + [norm])


# -------------------------------------------------------------- layer norm

class LayerNormFwdArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("x", _vp), ("ldx", _i64), ("weight", _vp), ("bias", _vp), ("y", _vp),
                ("stats", _vp), ("y_amax", _vp), ("x_dtype", _int), ("weight_dtype", _int),
                ("bias_dtype", _int), ("y_dtype", _int), ("eps", ctypes.c_float)]


class LayerNormBwdArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("dy", _vp), ("x", _vp), ("lddy", _i64), ("ldx", _i64),
                ("weight", _vp), ("stats", _vp), ("dx", _vp), ("dweight", _vp), ("dbias", _vp),
                ("dy_dtype", _int), ("x_dtype", _int), ("weight_dtype", _int), ("dweight_dtype", _int),
                ("dbias_dtype", _int), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


_LN_FWD = struct.Struct("@9q4if4x")
_LN_BWD = struct.Struct("@11q5i4x2q")
for _fmt, _cls in ((_LN_FWD, LayerNormFwdArgs), (_LN_BWD, LayerNormBwdArgs)):
    assert _fmt.size == ctypes.sizeof(_cls)

_lib.f8lin_layer_norm_forward.argtypes = [_vp, _vp]
_lib.f8lin_layer_norm_backward.argtypes = [_vp, _vp]
_lib.f8lin_layer_norm_workspace_bytes.argtypes = [_i64, _i64]
_lib.f8lin_layer_norm_workspace_bytes.restype = ctypes.c_size_t
for _name in ("f8lin_layer_norm_forward", "f8lin_layer_norm_backward"):
    getattr(_lib, _name).restype = _int


def _f32(t: Optional[torch.Tensor], n: int, what: str, device: torch.device) -> int:
    """Pointer of a contiguous float32 tensor of n elements on `device` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not torch.float32 or t.device != device or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"f8lin: {what} must be a contiguous float32 tensor of {n} elements on {device}")
    return t.data_ptr()


def _vector(t: Optional[torch.Tensor], n: int, what: str, device: torch.device):
    """(pointer, dtype code) of a contiguous bf16 / fp16 / fp32 vector of n elements on `device` (0, 0 for None)."""
    if t is None:
        return 0, 0
    if t.numel() != n:
        raise ValueError(f"f8lin: {what} must have {n} elements, got {tuple(t.shape)}")
    return _dense(t, what, device), _DTYPE[t.dtype]


def _pair_types(x: torch.Tensor, y: torch.Tensor, what: str):
    if y.dtype != x.dtype and x.dtype != torch.float32:
        raise TypeError(f"f8lin: {what} must be {x.dtype} like x (only a float32 x allows another type), got {y.dtype}")


def layer_norm_forward(x, y, weight=None, bias=None, eps: float = 1e-5, stats=None, y_amax=None, stream=None):
    """y (rows, cols) = the layer norm of each row of x, times weight plus bias (each (cols) or None).  stats: optional
    float32 (2, rows) tensor that receives the rows' mean and rstd for the backward.  y_amax: optional float32 tensor
    that receives max |y|."""
    if x.dim() != 2 or y.shape != x.shape:
        raise ValueError("layer_norm_forward: x and y must be 2-D tensors of one shape")
    rows, cols = x.shape
    px, ldx = _dense_ld(x, "x")
    dev = x.device
    py = _dense(y, "y", dev)
    if y.dtype is not x.dtype:
        _pair_types(x, y, "y")
    pw = wt = pb = bt = 0
    if weight is not None:
        pw, wt = _vector(weight, cols, "weight", dev)
    if bias is not None:
        pb, bt = _vector(bias, cols, "bias", dev)
    a = _LN_FWD.pack(rows, cols, px, ldx, pw, pb, py, 0 if stats is None else _f32(stats, 2 * rows, "stats", dev),
                     0 if y_amax is None else _f32(y_amax, 1, "y_amax", dev), _DTYPE[x.dtype], wt, bt, _DTYPE[y.dtype], eps)
    _call(_lib.f8lin_layer_norm_forward, dev, stream, a)


@functools.lru_cache(maxsize=1024)
def layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib.f8lin_layer_norm_workspace_bytes(rows, cols))


def layer_norm_backward(dy, x, weight, stats, dx=None, dweight=None, dbias=None, ws=None, stream=None):
    """dx (rows, cols; x's type), dweight (cols) and dbias (cols) -- each may be None -- from dy, x, weight (or None) and
    the forward's mean and rstd.  ws: layer_norm_workspace_bytes(rows, cols) bytes, for dweight or dbias."""
    if x.dim() != 2 or dy.shape != x.shape or (dx is not None and dx.shape != x.shape):
        raise ValueError("layer_norm_backward: dy, x and dx must be 2-D tensors of one shape")
    rows, cols = x.shape
    px, ldx = _dense_ld(x, "x")
    dev = x.device
    pdy, lddy = _dense_ld(dy, "dy", dev)
    _pair_types(x, dy, "dy")
    pdx = 0 if dx is None else _dense(dx, "dx", dev)
    if dx is not None and dx.dtype != x.dtype:
        raise TypeError(f"f8lin: dx must be {x.dtype} like x, got {dx.dtype}")
    pw, wt = _vector(weight, cols, "weight", dev)
    pdw, dwt = _vector(dweight, cols, "dweight", dev)
    pdb, dbt = _vector(dbias, cols, "dbias", dev)
    _same_device(ws, "ws", dev)
    a = _LN_BWD.pack(rows, cols, pdy, px, lddy, ldx, pw, _f32(stats, 2 * rows, "stats", dev), pdx, pdw, pdb,
                     _DTYPE[dy.dtype], _DTYPE[x.dtype], wt, dwt, dbt, _ptr(ws) or 0, _nbytes(ws))
    _call(_lib.f8lin_layer_norm_backward, dev, stream, a)


# ------------------------------------------------------- low-rank adapters

LORA_MAX_ADAPTERS = 2047
LORA_MAX_RANK = 256


class LoraFwdArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("K", _i64), ("N", _i64), ("x", _vp), ("a", _vp), ("b", _vp), ("base", _vp),
                ("ldx", _i64), ("ldbase", _i64), ("y", _vp), ("scales", _vp), ("plan", _vp), ("h", _vp), ("ws", _vp),
                ("ws_bytes", ctypes.c_size_t), ("rank", _int), ("adapters", _int), ("dtype", _int)]


class LoraBwdArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("K", _i64), ("N", _i64), ("dy", _vp), ("x", _vp), ("a", _vp), ("b", _vp),
                ("lddy", _i64), ("ldx", _i64), ("scales", _vp), ("h", _vp), ("plan", _vp), ("dx", _vp), ("da", _vp),
                ("db", _vp), ("ws", _vp), ("ws_bytes", ctypes.c_size_t), ("rank", _int), ("adapters", _int),
                ("dtype", _int)]


_LORA_FWD = struct.Struct("@15q3i4x")
_LORA_BWD = struct.Struct("@17q3i4x")
for _fmt, _cls in ((_LORA_FWD, LoraFwdArgs), (_LORA_BWD, LoraBwdArgs)):
    assert _fmt.size == ctypes.sizeof(_cls)

_lib.f8lin_lora_plan_bytes.argtypes = [_i64, _int]
_lib.f8lin_lora_plan.argtypes = [_vp, _int, _i64, _int, _vp, ctypes.c_size_t, _vp]
_lib.f8lin_lora_forward.argtypes = [_vp, _vp]
_lib.f8lin_lora_backward.argtypes = [_vp, _vp]
for _name in ("f8lin_lora_forward_workspace_bytes", "f8lin_lora_backward_workspace_bytes"):
    getattr(_lib, _name).argtypes = [_i64, _i64, _i64, _int, _int]
    getattr(_lib, _name).restype = ctypes.c_size_t
_lib.f8lin_lora_plan_bytes.restype = ctypes.c_size_t
for _name in ("f8lin_lora_plan", "f8lin_lora_forward", "f8lin_lora_backward"):
    getattr(_lib, _name).restype = _int


_lora_serials = itertools.count(1)


class LoraPlan:
    """The buffer of a plan (lora_plan writes it) for a batch of `tokens` tokens over `adapters` adapters.  `serial` is
    another number each time that any plan is written, 0 before; `writes` counts this one's."""

    __slots__ = ("tokens", "adapters", "device", "buffer", "serial", "writes", "_mark")

    def __init__(self, tokens: int, adapters: int, device="cuda", buffer: Optional[torch.Tensor] = None):
        """buffer: an int32 tensor to use instead of a new one."""
        if not 1 <= adapters <= LORA_MAX_ADAPTERS:
            raise ValueError(f"f8lin: a plan holds 1 to {LORA_MAX_ADAPTERS} adapters, got {adapters}")
        need = int(_lib.f8lin_lora_plan_bytes(tokens, adapters))
        if need == 0:
            raise ValueError(f"f8lin: a plan holds 0 to 2^22 tokens, got {tokens}")
        if buffer is None:
            buffer = torch.empty(need // 4, dtype=torch.int32, device=device)
        elif buffer.dtype != torch.int32 or not buffer.is_contiguous() or buffer.numel() < need // 4 or not buffer.is_cuda:
            raise ValueError(f"f8lin: this plan needs a contiguous int32 GPU buffer of {need // 4} elements")
        self.tokens, self.adapters, self.device, self.buffer = tokens, adapters, buffer.device, buffer
        self.serial, self.writes, self._mark = 0, 0, None

    def written(self) -> None:
        self.serial, self.writes, self._mark = next(_lora_serials), self.writes + 1, None

    def mark(self) -> torch.Tensor:
        """The serial as a tensor in host memory, to be saved beside the tensors of a graph."""
        if self._mark is None:
            self._mark = torch.tensor(self.serial, device="cpu")
        return self._mark


def lora_plan(index: torch.Tensor, plan: LoraPlan, stream=None):
    """Writes the plan of a batch: index (tokens) int32 or int64 holds each token's adapter, a value outside
    0 .. adapters - 1 none."""
    if index.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"f8lin: index must be int32 or int64, got {index.dtype}")
    if index.numel() != plan.tokens:
        raise ValueError(f"f8lin: the plan is of {plan.tokens} tokens, got {index.numel()} indices")
    p = _ptr(index) or 0
    if index.device != plan.device:
        raise ValueError(f"f8lin: index is on {index.device}, the plan on {plan.device}")
    _call(_lib.f8lin_lora_plan, plan.device, stream, p, index.element_size(), plan.tokens, plan.adapters,
          plan.buffer.data_ptr(), 4 * plan.buffer.numel())
    torch.autograd.graph.increment_version(plan.buffer)
    plan.written()


@functools.lru_cache(maxsize=1024)
def lora_forward_workspace_bytes(T: int, K: int, N: int, rank: int, adapters: int) -> int:
    return int(_lib.f8lin_lora_forward_workspace_bytes(T, K, N, rank, adapters))


@functools.lru_cache(maxsize=1024)
def lora_backward_workspace_bytes(T: int, K: int, N: int, rank: int, adapters: int) -> int:
    return int(_lib.f8lin_lora_backward_workspace_bytes(T, K, N, rank, adapters))


def lora_h_elements(T: int, rank: int) -> int:
    """Float32 elements of the inner products that lora_forward keeps for lora_backward."""
    return T * (16 if rank <= 16 else -(-rank // 32) * 32)


def _lora_refuse(x_rows: int, K: int, a: torch.Tensor, b: torch.Tensor, plan: LoraPlan):
    """Raises for adapters a (adapters, rank, K), b (adapters, N, rank) that do not fit x and the plan."""
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != plan.adapters or b.shape[0] != plan.adapters or \
            a.shape[2] != K or b.shape[2] != a.shape[1]:
        raise ValueError(f"f8lin: adapters must be ({plan.adapters}, rank, {K}) and ({plan.adapters}, N, rank), got "
                         f"{tuple(a.shape)} and {tuple(b.shape)}")
    if not 1 <= a.shape[1] <= LORA_MAX_RANK:
        raise ValueError(f"f8lin: the rank must be 1 to {LORA_MAX_RANK}, got {a.shape[1]}")
    raise ValueError(f"f8lin: the plan is of {plan.tokens} tokens, got {x_rows} rows")


def _lora_sizes(x_rows: int, K: int, a: torch.Tensor, b: torch.Tensor, plan: LoraPlan):
    """(rank, N) of the adapters beside the plan."""
    sa, sb = a.shape, b.shape
    if len(sa) != 3 or len(sb) != 3:
        _lora_refuse(x_rows, K, a, b, plan)
    (la, rank, ka), (lb, N, rb) = sa, sb
    if la != plan.adapters or lb != la or ka != K or rb != rank or x_rows != plan.tokens or not 1 <= rank <= LORA_MAX_RANK:
        _lora_refuse(x_rows, K, a, b, plan)
    return rank, N


def _one_dtype(dtype: torch.dtype, *named):
    """Raises unless every (name, tensor or None) has this dtype."""
    for what, t in named:
        if t is not None and t.dtype is not dtype:
            raise TypeError(f"f8lin: {what} must be {dtype} like x, got {t.dtype}")


def _workspace(nbytes: int, device: torch.device, stream) -> torch.Tensor:
    """Scratch for one call, of the stream that the call runs on."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def lora_forward(base, x, a, b, scales, plan: LoraPlan, y, h=None, ws=None, stream=None):
    """y (T, N) = base (T, N; None: 0) + what each token's adapter adds: scales[i] * (x[t] . a[i]^T) . b[i]^T.
    scales: float32 (adapters), or None for 1.  h: optional float32 tensor of lora_h_elements(T, rank) that receives the
    inner products for lora_backward.  ws: lora_forward_workspace_bytes(T, K, N, rank, adapters) bytes, or None to
    allocate them.  y may be base."""
    T, K = x.shape
    rank, N = _lora_sizes(T, K, a, b, plan)
    if y.shape != (T, N) or (base is not None and base.shape != y.shape):
        raise ValueError("lora_forward: shape mismatch")
    px, ldx = _dense_ld(x, "x")
    dev = x.device
    dt = x.dtype
    if a.dtype is not dt or b.dtype is not dt or y.dtype is not dt or (base is not None and base.dtype is not dt):
        _one_dtype(dt, ("a", a), ("b", b), ("base", base), ("y", y))
    pbase, ldbase = (0, 0) if base is None else _dense_ld(base, "base", dev)
    if plan.device != dev:
        raise ValueError(f"f8lin: the plan is on {plan.device}, expected {dev}")
    if ws is None:
        nbytes = lora_forward_workspace_bytes(T, K, N, rank, plan.adapters)
        pws = (ws := _workspace(nbytes, dev, stream)).data_ptr()
    else:
        _same_device(ws, "ws", dev)
        pws, nbytes = _ptr(ws) or 0, _nbytes(ws)
    args = _LORA_FWD.pack(T, K, N, px, _dense(a, "a", dev), _dense(b, "b", dev), pbase, ldx, ldbase, _dense(y, "y", dev),
                          _f32(scales, plan.adapters, "scales", dev), plan.buffer.data_ptr(),
                          0 if h is None else _f32(h, lora_h_elements(T, rank), "h", dev), pws, nbytes, rank,
                          plan.adapters, _DTYPE[dt])
    _call(_lib.f8lin_lora_forward, dev, stream, args)


def lora_backward(dy, x, a, b, scales, plan: LoraPlan, h, dx=None, da=None, db=None, ws=None, stream=None):
    """dx (T, K), da like a and db like b -- each may be None -- of lora_forward; h as it left it (needed for db).
    ws: lora_backward_workspace_bytes(T, K, N, rank, adapters) bytes, or None to allocate them."""
    T, K = x.shape
    rank, N = _lora_sizes(T, K, a, b, plan)
    if tuple(dy.shape) != (T, N) or (dx is not None and dx.shape != x.shape) or \
            (da is not None and da.shape != a.shape) or (db is not None and db.shape != b.shape):
        raise ValueError("lora_backward: shape mismatch")
    px, ldx = _dense_ld(x, "x")
    dev = x.device
    _one_dtype(x.dtype, ("dy", dy), ("a", a), ("b", b), ("dx", dx), ("da", da), ("db", db))
    pdy, lddy = _dense_ld(dy, "dy", dev)
    if plan.device != dev:
        raise ValueError(f"f8lin: the plan is on {plan.device}, expected {dev}")
    if ws is None:
        ws = _workspace(lora_backward_workspace_bytes(T, K, N, rank, plan.adapters), dev, stream)
    _same_device(ws, "ws", dev)
    opt = lambda t, what: 0 if t is None else _dense(t, what, dev)  # noqa: E731
    args = _LORA_BWD.pack(T, K, N, pdy, px, _dense(a, "a", dev), _dense(b, "b", dev), lddy, ldx,
                          _f32(scales, plan.adapters, "scales", dev),
                          0 if h is None else _f32(h, lora_h_elements(T, rank), "h", dev), plan.buffer.data_ptr(),
                          opt(dx, "dx"), opt(da, "da"), opt(db, "db"), _ptr(ws) or 0, _nbytes(ws), rank, plan.adapters,
                          _DTYPE[x.dtype])
    _call(_lib.f8lin_lora_backward, dev, stream, args)
