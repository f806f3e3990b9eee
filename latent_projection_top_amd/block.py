"""Python binding of the layer's operators (include/block.h in libroute.so):
layer norm, the gated feed-forward product and the linear product with bias,
activation and residual, each forward and backward. Argument marshalling only.

Like the route's binding: every function checks types, shapes and placement,
then calls the C entry point of the same operator; a non-zero status raises
RouteError and there is no fallback. Matrices of rows may have any row stride
(`t.stride(0)`), weights are contiguous [K][N].
"""
from __future__ import annotations

import ctypes

import torch

from .route import LIB, OK, RouteError

ABI_VERSION = 1
MAX_ROWS = 1 << 20
MAX_SIZE = 1 << 17
MAX_STRIDE = 1 << 20
WORKSPACE_ZEROED = 1 << 17

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

SYMBOLS = tuple(f"block_{op}{call}" for op in ("norm", "gated", "linear")
                for call in ("_prepare", "_workspace_bytes", "", "_backward", "_destroy"))


class NormConfig(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("width", ctypes.c_int32), ("dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class GatedConfig(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("inputs", ctypes.c_int32), ("inner", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("training", ctypes.c_int32)]


class LinearConfig(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("inputs", ctypes.c_int32), ("outputs", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("training", ctypes.c_int32)]


def _declare() -> None:
    p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    mat = [p, i64]  # a matrix of rows and its stride
    args = {
        "block_norm": [p, *mat, p, p, *mat, p, p, i32, p],
        "block_norm_backward": [p, *mat, *mat, p, p, p, *mat, p, p, p, i32, p],
        "block_gated": [p, *mat, p, p, *mat, p, p, p, i32, p],
        "block_gated_backward": [p, *mat, *mat, p, p, p, p, *mat, p, p, p, i32, p],
        "block_linear": [p, *mat, p, p, *mat, *mat, p, p, i32, p],
        "block_linear_backward": [p, *mat, *mat, p, p, *mat, p, p, p, i32, p],
    }
    for name, types in args.items():
        fn = getattr(LIB, name)
        fn.argtypes, fn.restype = types, ctypes.c_int
    for op, config in (("norm", NormConfig), ("gated", GatedConfig), ("linear", LinearConfig)):
        fn = getattr(LIB, f"block_{op}_prepare")
        fn.argtypes, fn.restype = [ctypes.POINTER(config), ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int
        fn = getattr(LIB, f"block_{op}_workspace_bytes")
        fn.argtypes, fn.restype = [p], ctypes.c_size_t
        fn = getattr(LIB, f"block_{op}_destroy")
        fn.argtypes, fn.restype = [p], None


_declare()


def prepare_raw(op: str, cfg) -> tuple[int, int]:
    """Call block_<op>_prepare; returns (status, plan handle or 0). cfg may be None."""
    out = ctypes.c_void_p(0)
    st = getattr(LIB, f"block_{op}_prepare")(ctypes.byref(cfg) if cfg is not None else None,
                                             ctypes.byref(out))
    return st, (out.value or 0)


def _code(table, key, what: str) -> int:
    if key not in table:
        raise ValueError(f"{what}: expected one of {list(table)}, got {key!r}")
    return table[key]


class _Plan:
    """A prepared plan (owns the C plan; freed on close/GC)."""

    OP = ""

    def _prepare(self, cfg) -> None:
        st, handle = prepare_raw(self.OP, cfg)
        if st != OK:
            raise RouteError(st, f"block_{self.OP}_prepare")
        self.handle = handle
        self.rows = cfg.rows
        self.device = cfg.device
        self.workspace_bytes = int(getattr(LIB, f"block_{self.OP}_workspace_bytes")(handle))

    def new_workspace(self) -> torch.Tensor:
        """A workspace tensor of the size this plan needs, zero where it has to be."""
        ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=f"cuda:{self.device}")
        if self.OP != "norm":
            ws[:WORKSPACE_ZEROED].zero_()
        return ws

    def close(self) -> None:
        if getattr(self, "handle", 0):
            getattr(LIB, f"block_{self.OP}_destroy")(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _device(device) -> int:
    return torch.cuda.current_device() if device is None else int(device)


class NormPlan(_Plan):
    """Layer norm of up to `rows` rows of `width` values."""

    OP = "norm"

    def __init__(self, rows: int, width: int, dtype=torch.bfloat16, param_dtype=torch.float32,
                 eps: float = 1e-5, device: int | None = None):
        self.width, self.dtype, self.param_dtype = width, dtype, param_dtype
        self._prepare(NormConfig(ABI_VERSION, _device(device), rows, width, _code(DTYPES, dtype, "dtype"),
                                 _code(DTYPES, param_dtype, "param_dtype"), eps))


class GatedPlan(_Plan):
    """h = act(x w_gate) * (x w_up) of up to `rows` rows; `training` sizes the
    workspace for the backward call as well."""

    OP = "gated"

    def __init__(self, rows: int, inputs: int, inner: int, activation: str = "silu", dtype=torch.bfloat16,
                 training: bool = False, device: int | None = None):
        self.inputs, self.inner, self.dtype, self.activation = inputs, inner, dtype, activation
        self.training = bool(training)
        self._prepare(GatedConfig(ABI_VERSION, _device(device), rows, inputs, inner,
                                  _code(DTYPES, dtype, "dtype"), _code(ACTIVATIONS, activation, "activation"),
                                  int(self.training)))


class LinearPlan(_Plan):
    """y = act(x w + bias) + residual of up to `rows` rows; `training` sizes
    the workspace for the backward call as well."""

    OP = "linear"

    def __init__(self, rows: int, inputs: int, outputs: int, activation: str = "none", dtype=torch.bfloat16,
                 training: bool = False, device: int | None = None):
        self.inputs, self.outputs, self.dtype, self.activation = inputs, outputs, dtype, activation
        self.training = bool(training)
        self._prepare(LinearConfig(ABI_VERSION, _device(device), rows, inputs, outputs,
                                   _code(DTYPES, dtype, "dtype"),
                                   _code(ACTIVATIONS, activation, "activation"), int(self.training)))


# The checks run on every call, in front of kernels of a few microseconds, so
# they read each property of a tensor once.


def _check(t: torch.Tensor, dtype, plan: _Plan, name: str) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != plan.device:
        raise ValueError(f"{name}: on {t.device}, the plan is for cuda:{plan.device}")


def _rows_of(t, dtype, plan: _Plan, rows: int, width: int, name: str) -> tuple[int | None, int]:
    """Pointer and row stride of a matrix of rows; None gives (NULL, width)."""
    if t is None:
        return None, width
    if t.dtype is not dtype or t.get_device() != plan.device:
        _check(t, dtype, plan, name)
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name}: expected [rows][{width}], got {tuple(shape)}")
    if shape[0] < rows:
        raise ValueError(f"{name}: needs at least {rows} rows, has {shape[0]}")
    if strides[1] != 1 and width > 1 and rows > 0:
        raise ValueError(f"{name}: the values of a row must be adjacent")
    if rows <= 1:  # the stride of a single row is never used
        return t.data_ptr(), width
    if strides[0] < width:
        raise ValueError(f"{name}: rows overlap (row stride {strides[0]}, width {width})")
    return t.data_ptr(), strides[0]


def _dense(t, dtype, plan: _Plan, shape, name: str) -> int | None:
    """Pointer of a contiguous tensor of exactly this shape."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != plan.device:
        _check(t, dtype, plan, name)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _per_row(t, dtype, plan: _Plan, shape, name: str) -> int | None:
    """Like _dense for what is kept per row: spare rows at the end are allowed."""
    if t is not None and t.dim() == len(shape) and t.shape[0] > shape[0]:
        t = t[:shape[0]]
    return _dense(t, dtype, plan, shape, name)


def _workspace(plan: _Plan, workspace) -> int:
    if workspace.dtype is not torch.uint8 or workspace.get_device() != plan.device:
        _check(workspace, torch.uint8, plan, "workspace")
    if workspace.numel() < plan.workspace_bytes or not workspace.is_contiguous():
        raise ValueError(f"workspace: needs {plan.workspace_bytes} contiguous bytes")
    return workspace.data_ptr()


def _stream(plan: _Plan, stream) -> int | None:
    if stream is not None:
        return stream.cuda_stream or None
    return _current_stream(plan.device) or None


# the current stream's handle alone (torch.cuda.current_stream builds an object)
_current_stream = torch._C._cuda_getCurrentRawStream


def _run(fn, name: str, plan: _Plan, *args) -> None:
    st = fn(plan.handle, *args)
    if st != OK:
        raise RouteError(st, name)


def layer_norm(plan: NormPlan, x, weight, bias, y, mean=None, rstd=None, rows: int | None = None,
               stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias; weight and bias may be None; mean
    and rstd (FP32, one per row) are kept for layer_norm_backward if given."""
    rows = x.shape[0] if rows is None else rows
    dt, pdt, w = plan.dtype, plan.param_dtype, plan.width
    _run(LIB.block_norm, "block_norm", plan, *_rows_of(x, dt, plan, rows, w, "x"),
         _dense(weight, pdt, plan, (w,), "weight"), _dense(bias, pdt, plan, (w,), "bias"),
         *_rows_of(y, dt, plan, rows, w, "y"), _per_row(mean, torch.float32, plan, (rows,), "mean"),
         _per_row(rstd, torch.float32, plan, (rows,), "rstd"), rows, _stream(plan, stream))


def layer_norm_backward(plan: NormPlan, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                        rows: int | None = None, stream=None) -> None:
    """Gradients of layer_norm; dx, dweight or dbias None is not computed."""
    rows = dy.shape[0] if rows is None else rows
    dt, pdt, w = plan.dtype, plan.param_dtype, plan.width
    _run(LIB.block_norm_backward, "block_norm_backward", plan, *_rows_of(dy, dt, plan, rows, w, "dy"),
         *_rows_of(x, dt, plan, rows, w, "x"), _dense(weight, pdt, plan, (w,), "weight"),
         _per_row(mean, torch.float32, plan, (rows,), "mean"),
         _per_row(rstd, torch.float32, plan, (rows,), "rstd"), *_rows_of(dx, dt, plan, rows, w, "dx"),
         _dense(dweight, pdt, plan, (w,), "dweight"), _dense(dbias, pdt, plan, (w,), "dbias"),
         _workspace(plan, workspace), rows, _stream(plan, stream))


def gated(plan: GatedPlan, x, w_gate, w_up, h, workspace, d_gate=None, d_up=None, rows: int | None = None,
          stream=None) -> None:
    """h = act(x w_gate) * (x w_up). For training, d_gate and d_up receive the
    derivatives of h by the two products, for gated_backward."""
    rows = x.shape[0] if rows is None else rows
    dt, k, n = plan.dtype, plan.inputs, plan.inner
    _run(LIB.block_gated, "block_gated", plan, *_rows_of(x, dt, plan, rows, k, "x"),
         _dense(w_gate, dt, plan, (k, n), "w_gate"), _dense(w_up, dt, plan, (k, n), "w_up"),
         *_rows_of(h, dt, plan, rows, n, "h"), _per_row(d_gate, dt, plan, (rows, n), "d_gate"),
         _per_row(d_up, dt, plan, (rows, n), "d_up"), _workspace(plan, workspace), rows, _stream(plan, stream))


def gated_backward(plan: GatedPlan, dh, x, w_gate, w_up, d_gate, d_up, dx, dw_gate, dw_up, workspace,
                   rows: int | None = None, stream=None) -> None:
    """Gradients of gated; dx None, or dw_gate and dw_up None, is not computed."""
    rows = dh.shape[0] if rows is None else rows
    dt, k, n = plan.dtype, plan.inputs, plan.inner
    _run(LIB.block_gated_backward, "block_gated_backward", plan, *_rows_of(dh, dt, plan, rows, n, "dh"),
         *_rows_of(x, dt, plan, rows, k, "x"), _dense(w_gate, dt, plan, (k, n), "w_gate"),
         _dense(w_up, dt, plan, (k, n), "w_up"), _per_row(d_gate, dt, plan, (rows, n), "d_gate"),
         _per_row(d_up, dt, plan, (rows, n), "d_up"), *_rows_of(dx, dt, plan, rows, k, "dx"),
         _dense(dw_gate, dt, plan, (k, n), "dw_gate"), _dense(dw_up, dt, plan, (k, n), "dw_up"),
         _workspace(plan, workspace), rows, _stream(plan, stream))


def linear(plan: LinearPlan, x, w, y, workspace, bias=None, residual=None, slope=None,
           rows: int | None = None, stream=None) -> None:
    """y = act(x w + bias) + residual; `residual` may be `y` itself. For
    training with an activation, `slope` receives act' for linear_backward."""
    rows = x.shape[0] if rows is None else rows
    dt, k, n = plan.dtype, plan.inputs, plan.outputs
    _run(LIB.block_linear, "block_linear", plan, *_rows_of(x, dt, plan, rows, k, "x"), _dense(w, dt, plan, (k, n), "w"),
         _dense(bias, dt, plan, (n,), "bias"), *_rows_of(residual, dt, plan, rows, n, "residual"),
         *_rows_of(y, dt, plan, rows, n, "y"), _per_row(slope, dt, plan, (rows, n), "slope"),
         _workspace(plan, workspace), rows, _stream(plan, stream))


def linear_backward(plan: LinearPlan, dy, x, w, slope, dx, dw, dbias, workspace, rows: int | None = None,
                    stream=None) -> None:
    """Gradients of linear (the residual's is dy itself); dx, dw or dbias None
    is not computed. `slope` is None when the plan has no activation."""
    rows = dy.shape[0] if rows is None else rows
    dt, k, n = plan.dtype, plan.inputs, plan.outputs
    _run(LIB.block_linear_backward, "block_linear_backward", plan, *_rows_of(dy, dt, plan, rows, n, "dy"),
         *_rows_of(x, dt, plan, rows, k, "x"), _dense(w, dt, plan, (k, n), "w"),
         _per_row(slope, dt, plan, (rows, n), "slope"), *_rows_of(dx, dt, plan, rows, k, "dx"),
         _dense(dw, dt, plan, (k, n), "dw"), _dense(dbias, dt, plan, (n,), "dbias"),
         _workspace(plan, workspace), rows, _stream(plan, stream))
