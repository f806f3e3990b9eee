"""Python binding of the routed half of a layer (include/experts.h in
libroute.so): choices sorted by expert, rows taken to that order and back with
their gradients, and the experts' products in 8-bit integers. Argument
marshalling only.

Like the other bindings: every function checks types, shapes and placement,
then calls the C entry point of the same operator; a non-zero status raises
RouteError and there is no fallback. A buffer in sorted order (`token`, `xs`,
`ys`, `dxs`, `dys`) of fewer than rows * topk rows drops the choices placed
beyond its end.
"""
from __future__ import annotations

import ctypes

import torch

from .block import ACTIVATIONS, DTYPES, _code, _dense, _device, _per_row, _Plan, _rows_of, _run, _stream, _workspace
from .route import LIB, OK, RouteError

ABI_VERSION = 1
MAX_COUNT = 4096
MAX_TOPK = 64
MAX_CHOICES = 1 << 24
MAX_INPUTS = 131071
WORKSPACE_ZEROED = 65536

_CALLS = {"sort": ("_workspace_bytes", ""), "combine": ("", "_backward"),
          "linear8": ("_workspace_bytes", "_packed_bytes", "_quantize", "_pack", ""),
          "gated8": ("_workspace_bytes", "_packed_bytes", "_quantize", "_pack", "")}
SYMBOLS = tuple(f"experts_{op}{call}" for op, calls in _CALLS.items()
                for call in ("_prepare", *calls, "_destroy")) + ("experts_gather", "experts_gather_backward")


class SortConfig(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("experts", ctypes.c_int32), ("first", ctypes.c_int32)]


class CombineConfig(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Linear8Config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("tokens", ctypes.c_int32), ("inputs", ctypes.c_int32), ("outputs", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class Gated8Config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("device", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("tokens", ctypes.c_int32), ("inputs", ctypes.c_int32), ("inner", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


_CONFIG = {"sort": SortConfig, "combine": CombineConfig, "linear8": Linear8Config, "gated8": Gated8Config}


def _declare() -> None:
    p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    mat = [p, i64]  # a matrix of rows and its stride
    args = {
        "experts_sort": [p, p, p, p, p, p, i32, i32, p],
        "experts_gather": [p, *mat, p, *mat, i32, i32, p],
        "experts_gather_backward": [p, *mat, p, *mat, i32, i32, p],
        "experts_combine": [p, *mat, p, p, *mat, *mat, i32, i32, p],
        "experts_combine_backward": [p, *mat, *mat, p, p, *mat, p, i32, i32, p],
        "experts_linear8_quantize": [p, p, p, p, p],
        "experts_linear8_pack": [p, p, p, p],
        "experts_linear8": [p, *mat, p, p, p, p, p, *mat, *mat, p, i32, i32, p],
        "experts_gated8_quantize": [p, p, p, p, p],
        "experts_gated8_pack": [p, p, p, p, p],
        "experts_gated8": [p, *mat, p, p, p, p, p, *mat, p, i32, i32, p],
    }
    for name, types in args.items():
        fn = getattr(LIB, name)
        fn.argtypes, fn.restype = types, ctypes.c_int
    for op, config in _CONFIG.items():
        fn = getattr(LIB, f"experts_{op}_prepare")
        fn.argtypes, fn.restype = [ctypes.POINTER(config), ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int
        fn = getattr(LIB, f"experts_{op}_destroy")
        fn.argtypes, fn.restype = [p], None
        for call in ("_workspace_bytes", "_packed_bytes"):
            if call in _CALLS[op]:
                fn = getattr(LIB, f"experts_{op}{call}")
                fn.argtypes, fn.restype = [p], ctypes.c_size_t


_declare()


def prepare_raw(op: str, cfg) -> tuple[int, int]:
    """Call experts_<op>_prepare; returns (status, plan handle or 0). cfg may be None."""
    out = ctypes.c_void_p(0)
    st = getattr(LIB, f"experts_{op}_prepare")(ctypes.byref(cfg) if cfg is not None else None,
                                               ctypes.byref(out))
    return st, (out.value or 0)


class _ExpertsPlan(_Plan):
    """A prepared plan (owns the C plan; freed on close/GC)."""

    def _prepare(self, cfg) -> None:
        st, handle = prepare_raw(self.OP, cfg)
        if st != OK:
            raise RouteError(st, f"experts_{self.OP}_prepare")
        self.handle = handle
        self.rows = cfg.rows
        self.device = cfg.device
        for name in ("workspace_bytes", "packed_bytes"):
            if "_" + name in _CALLS[self.OP]:
                setattr(self, name, int(getattr(LIB, f"experts_{self.OP}_{name}")(handle)))

    def close(self) -> None:
        if getattr(self, "handle", 0):
            getattr(LIB, f"experts_{self.OP}_destroy")(self.handle)
            self.handle = 0


class SortPlan(_ExpertsPlan):
    """Up to `rows` rows of `topk` choices, of which those of the experts first
    .. first + experts - 1 are kept."""

    OP = "sort"

    def __init__(self, rows: int, topk: int, experts: int, first: int = 0, device: int | None = None):
        self.topk, self.experts, self.first = topk, experts, first
        self._prepare(SortConfig(ABI_VERSION, _device(device), rows, topk, experts, first))

    def new_workspace(self) -> torch.Tensor:
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=f"cuda:{self.device}")


class CombinePlan(_ExpertsPlan):
    """Up to `rows` rows of `width` values, each with `topk` choices: gather,
    combine and their gradients. These calls need no workspace."""

    OP = "combine"

    def __init__(self, rows: int, topk: int, width: int, dtype=torch.bfloat16, device: int | None = None):
        self.topk, self.width, self.dtype = topk, width, dtype
        self._prepare(CombineConfig(ABI_VERSION, _device(device), rows, topk, width,
                                    _code(DTYPES, dtype, "dtype")))

    def new_workspace(self) -> None:
        return None


class _ProductPlan(_ExpertsPlan):
    def new_workspace(self) -> torch.Tensor:
        """A workspace tensor of the size this plan needs, zero where it has to be."""
        ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=f"cuda:{self.device}")
        ws[:WORKSPACE_ZEROED].zero_()
        return ws


class Linear8Plan(_ProductPlan):
    """y = act(x W[e] + bias[e]) + residual in 8-bit integers, for up to `rows`
    rows of y and `tokens` rows of x (by default as many)."""

    OP = "linear8"

    def __init__(self, rows: int, inputs: int, outputs: int, experts: int = 1, tokens: int | None = None,
                 activation: str = "none", dtype=torch.bfloat16, device: int | None = None):
        self.inputs, self.outputs, self.experts = inputs, outputs, experts
        self.tokens, self.activation, self.dtype = rows if tokens is None else tokens, activation, dtype
        self._prepare(Linear8Config(ABI_VERSION, _device(device), rows, self.tokens, inputs, outputs, experts,
                                    _code(DTYPES, dtype, "dtype"),
                                    _code(ACTIVATIONS, activation, "activation")))


class Gated8Plan(_ProductPlan):
    """h = act(x W_gate[e]) * (x W_up[e]) in 8-bit integers, for up to `rows`
    rows of h and `tokens` rows of x (by default as many)."""

    OP = "gated8"

    def __init__(self, rows: int, inputs: int, inner: int, experts: int = 1, tokens: int | None = None,
                 activation: str = "silu", dtype=torch.bfloat16, device: int | None = None):
        self.inputs, self.inner, self.experts = inputs, inner, experts
        self.tokens, self.activation, self.dtype = rows if tokens is None else tokens, activation, dtype
        self._prepare(Gated8Config(ABI_VERSION, _device(device), rows, self.tokens, inputs, inner, experts,
                                   _code(DTYPES, dtype, "dtype"),
                                   _code(ACTIVATIONS, activation, "activation")))

    @property
    def outputs(self) -> int:
        return self.inner


_I32, _F32, _I8 = torch.int32, torch.float32, torch.int8


# The checks run on every call, in front of kernels of a few microseconds: what
# is as it should be passes here, the rest goes to the checks that name the fault.


def _per_token(t, dtype, plan: _ExpertsPlan, rows: int, name: str) -> int | None:
    """Pointer of a contiguous [rows][topk] tensor; spare rows at the end are allowed."""
    if t is not None and t.dtype is dtype and t.get_device() == plan.device:
        shape = t.shape
        if len(shape) == 2 and shape[1] == plan.topk and shape[0] >= rows and t.is_contiguous():
            return t.data_ptr()
    return _per_row(t, dtype, plan, (rows, plan.topk), name)


def _sorted_rows(t, plan: CombinePlan, name: str) -> tuple[int | None, int, int]:
    """Pointer, row stride and rows of a matrix in sorted order; None has no rows."""
    if t is None:
        return None, plan.width, 0
    shape = t.shape
    if t.dtype is plan.dtype and t.get_device() == plan.device and len(shape) == 2 and shape[1] == plan.width:
        stride = t.stride()
        if stride[1] == 1 and stride[0] >= plan.width and 1 < shape[0] <= MAX_CHOICES:
            return t.data_ptr(), stride[0], shape[0]
    rows = min(shape[0], MAX_CHOICES) if len(shape) == 2 else 0
    return *_rows_of(t, plan.dtype, plan, rows, plan.width, name), rows


def sort(plan: SortPlan, ids, offsets, place, token, workspace, rows: int | None = None, stream=None) -> None:
    """offsets [experts + 1], place [rows][topk] and token [capacity] of the
    choices ids [rows][topk], all int32."""
    rows = ids.shape[0] if rows is None else rows
    shape = token.shape
    if len(shape) != 1:
        raise ValueError(f"token: expected one dimension, got {tuple(shape)}")
    capacity = min(shape[0], MAX_CHOICES)
    _run(LIB.experts_sort, "experts_sort", plan, _per_token(ids, _I32, plan, rows, "ids"),
         _dense(offsets, _I32, plan, (plan.experts + 1,), "offsets"), _per_token(place, _I32, plan, rows, "place"),
         _per_row(token, _I32, plan, (capacity,), "token"), _workspace(plan, workspace), capacity, rows,
         _stream(plan, stream))


def gather(plan: CombinePlan, x, place, xs, rows: int | None = None, stream=None) -> None:
    """xs[place[r, j]] = x[r]; the other rows of xs are left as they are."""
    rows = x.shape[0] if rows is None else rows
    to, ld, capacity = _sorted_rows(xs, plan, "xs")
    _run(LIB.experts_gather, "experts_gather", plan, *_rows_of(x, plan.dtype, plan, rows, plan.width, "x"),
         _per_token(place, _I32, plan, rows, "place"), to, ld, capacity, rows, _stream(plan, stream))


def gather_backward(plan: CombinePlan, dxs, place, dx, rows: int | None = None, stream=None) -> None:
    """dx[r] = sum_j dxs[place[r, j]]."""
    rows = dx.shape[0] if rows is None else rows
    src, ld, capacity = _sorted_rows(dxs, plan, "dxs")
    _run(LIB.experts_gather_backward, "experts_gather_backward", plan, src, ld,
         _per_token(place, _I32, plan, rows, "place"),
         *_rows_of(dx, plan.dtype, plan, rows, plan.width, "dx"), capacity, rows, _stream(plan, stream))


def combine(plan: CombinePlan, ys, place, weights, y, residual=None, rows: int | None = None, stream=None) -> None:
    """y[r] = sum_j weights[r, j] ys[place[r, j]] + residual[r]; `residual` may
    be `y` itself; weights are FP32 [rows][topk]."""
    rows = y.shape[0] if rows is None else rows
    dt, w = plan.dtype, plan.width
    src, ld, capacity = _sorted_rows(ys, plan, "ys")
    _run(LIB.experts_combine, "experts_combine", plan, src, ld, _per_token(place, _I32, plan, rows, "place"),
         _per_token(weights, _F32, plan, rows, "weights"), *_rows_of(residual, dt, plan, rows, w, "residual"),
         *_rows_of(y, dt, plan, rows, w, "y"), capacity, rows, _stream(plan, stream))


def combine_backward(plan: CombinePlan, dy, ys, place, weights, dys, dweights, rows: int | None = None,
                     stream=None) -> None:
    """Gradients of combine (the residual's is dy itself): dys[place[r, j]] =
    weights[r, j] dy[r], other rows left as they are, and dweights [rows][topk]
    FP32. Either may be None (not computed), ys with dweights, weights with dys."""
    rows = dy.shape[0] if rows is None else rows
    if dweights is None:
        ys = None
    src, src_ld, have = _sorted_rows(ys, plan, "ys")
    to, to_ld, room = _sorted_rows(dys, plan, "dys")
    if ys is not None and dys is not None and have != room:
        raise ValueError(f"dys: expected as many rows as ys ({have}), has {room}")
    _run(LIB.experts_combine_backward, "experts_combine_backward", plan,
         *_rows_of(dy, plan.dtype, plan, rows, plan.width, "dy"), src, src_ld,
         _per_token(place, _I32, plan, rows, "place"), _per_token(weights, _F32, plan, rows, "weights"), to, to_ld,
         _per_token(dweights, _F32, plan, rows, "dweights"), max(have, room), rows, _stream(plan, stream))


def quantize(plan: _ProductPlan, w, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """16-bit weights [experts][inputs][outputs] as (int8 of that shape, FP32
    scales [experts][outputs]); once per set of weights."""
    shape = (plan.experts, plan.inputs, plan.outputs)
    ptr = _dense(w, plan.dtype, plan, shape, "w")
    with torch.cuda.stream(stream):  # memory is reused in the order of the stream that it is allocated on
        w8 = torch.empty(shape, dtype=_I8, device=w.device)
        scale = torch.empty(shape[0], shape[2], dtype=_F32, device=w.device)
    name = f"experts_{plan.OP}_quantize"
    _run(getattr(LIB, name), name, plan, ptr, w8.data_ptr(), scale.data_ptr(), _stream(plan, stream))
    return w8, scale


def pack(plan: _ProductPlan, *w, stream=None) -> torch.Tensor:
    """int8 weights [experts][inputs][outputs] (w_gate and w_up for a
    Gated8Plan) in the form that the products read; once per set of weights."""
    if len(w) != (2 if plan.OP == "gated8" else 1):
        raise ValueError(f"pack: {plan.OP} has {2 if plan.OP == 'gated8' else 1} matrices, got {len(w)}")
    ptrs = [_dense(t, _I8, plan, (plan.experts, plan.inputs, plan.outputs), "w") for t in w]
    with torch.cuda.stream(stream):  # as in quantize
        packed = torch.empty(plan.packed_bytes, dtype=torch.uint8, device=w[0].device)
    name = f"experts_{plan.OP}_pack"
    _run(getattr(LIB, name), name, plan, *ptrs, packed.data_ptr(), _stream(plan, stream))
    return packed


def _product_rows(plan: _ProductPlan, x, token, y, rows) -> tuple[int, int]:
    """(tokens, rows) of a product's call."""
    if token is None:
        rows = x.shape[0] if rows is None else rows
        return rows, rows
    return x.shape[0], y.shape[0] if rows is None else rows


def _packed(plan: _ProductPlan, packed) -> int:
    return _dense(packed, torch.uint8, plan, (plan.packed_bytes,), "packed")


def linear8(plan: Linear8Plan, x, packed, scale, y, workspace, offsets=None, token=None, bias=None, residual=None,
            rows: int | None = None, stream=None) -> None:
    """y = act(x W[e] + bias[e]) + residual in 8-bit integers: row p of y is of
    the expert whose range of `offsets` holds p and of row token[p] of x (p
    without token). `residual` may be `y` itself. Rows of y at
    offsets[experts] and beyond are left as they are."""
    tokens, rows = _product_rows(plan, x, token, y, rows)
    dt, n, e = plan.dtype, plan.outputs, plan.experts
    _run(LIB.experts_linear8, "experts_linear8", plan, *_rows_of(x, dt, plan, tokens, plan.inputs, "x"),
         _packed(plan, packed), _dense(scale, _F32, plan, (e, n), "scale"),
         _dense(offsets, _I32, plan, (e + 1,), "offsets"), _per_row(token, _I32, plan, (rows,), "token"),
         _dense(bias, dt, plan, (e, n), "bias"), *_rows_of(residual, dt, plan, rows, n, "residual"),
         *_rows_of(y, dt, plan, rows, n, "y"), _workspace(plan, workspace), tokens, rows, _stream(plan, stream))


def gated8(plan: Gated8Plan, x, packed, scale_gate, scale_up, h, workspace, offsets=None, token=None,
           rows: int | None = None, stream=None) -> None:
    """h = act(x W_gate[e]) * (x W_up[e]) in 8-bit integers, rows as in linear8."""
    tokens, rows = _product_rows(plan, x, token, h, rows)
    dt, n, e = plan.dtype, plan.inner, plan.experts
    _run(LIB.experts_gated8, "experts_gated8", plan, *_rows_of(x, dt, plan, tokens, plan.inputs, "x"),
         _packed(plan, packed), _dense(scale_gate, _F32, plan, (e, n), "scale_gate"),
         _dense(scale_up, _F32, plan, (e, n), "scale_up"), _dense(offsets, _I32, plan, (e + 1,), "offsets"),
         _per_row(token, _I32, plan, (rows,), "token"), *_rows_of(h, dt, plan, rows, n, "h"),
         _workspace(plan, workspace), tokens, rows, _stream(plan, stream))
