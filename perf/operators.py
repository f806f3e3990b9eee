"""The operators that stand around the route in a layer, as cases to be timed
and compared: layer norm, the gated feed-forward product, and the linear
product with bias, activation and residual, each forward ("serve") and as a
training step ("train": forward and backward).

With `own` false every case is computed in its plain form, elementary torch
operations in FP32 rounded once at the end; with `own` true by the library's
kernels (latent_projection_top_amd.block).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def _norm(name, rows, width, train, dtype):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "train": train, "dtype": dtype}


def _gated(name, rows, inputs, inner, train, dtype, act):
    return {"name": name, "op": "gated", "rows": rows, "inputs": inputs, "inner": inner, "train": train,
            "dtype": dtype, "act": act}


def _linear(name, rows, inputs, outputs, train, dtype, act, bias, residual, strided):
    return {"name": name, "op": "linear", "rows": rows, "inputs": inputs, "outputs": outputs,
            "train": train, "dtype": dtype, "act": act, "bias": bias, "residual": residual,
            "strided": strided}


def listed():
    return [
        # one decoded token's hidden row before the route: launch latency
        _norm("norm-serve-1x7168", 1, 7168, False, "bf16"),
        # FP32 training of a small odd width: no vector alignment of the rows
        _norm("norm-train-517x1019-f32", 517, 1019, True, "f32"),
        # the latent's norm in a training step of one chunk
        _norm("norm-train-2048x3584", 2048, 3584, True, "bf16"),
        # the hidden norm over a long training batch: HBM bandwidth
        _norm("norm-train-16384x7168", 16384, 7168, True, "bf16"),
        # one decoded token through an expert on the latent: weight streaming
        _gated("gated-serve-1x3584x2048", 1, 3584, 2048, False, "bf16", "silu"),
        # the widest decode round through a shared expert on the hidden row
        _gated("gated-serve-20x7168x2048", 20, 7168, 2048, False, "bf16", "silu"),
        # a small model's training step, every size odd
        _gated("gated-train-333x1001x777-f16", 333, 1001, 777, True, "f16", "gelu"),
        # a 1024-row prefill chunk
        _gated("gated-serve-1024x3584x4096", 1024, 3584, 4096, False, "bf16", "silu"),
        # a training step over a full batch: the largest
        _gated("gated-train-4096x3584x4096", 4096, 3584, 4096, True, "bf16", "silu"),
        # a decode round's way back to the hidden width, onto the residual
        _linear("linear-serve-8x2048x7168", 8, 2048, 7168, False, "bf16", "none", False, True, False),
        # a prefill chunk with everything in the epilogue, its input a column
        # slice of a wider buffer
        _linear("linear-serve-2048x3584x7168", 2048, 3584, 7168, False, "bf16", "gelu_tanh", True, True,
                True),
        # a training step whose row count fills no tile
        _linear("linear-train-2047x3584x7168", 2047, 3584, 7168, True, "bf16", "silu", True, True, False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over [lo, hi] by its logarithm; three of five are
    multiples of 8 as most models' are, the rest are as drawn."""
    n = _log_int(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(("norm", "gated", "linear"))
    train = rng.random() < 0.5
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "width": _size(rng, 64, 7168), "train": train,
                "dtype": rng.choice(("bf16", "bf16", "f16", "f32"))}
    dtype = rng.choice(("bf16", "bf16", "f16"))
    act = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    rows = _log_int(rng, 1, 4096)
    if op == "gated":
        return {"op": op, "rows": rows, "inputs": _size(rng, 128, 3584), "inner": _size(rng, 128, 4096),
                "train": train, "dtype": dtype, "act": act}
    return {"op": op, "rows": rows, "inputs": _size(rng, 128, 3584), "outputs": _size(rng, 128, 7168),
            "train": train, "dtype": dtype, "act": rng.choice((act, "none")), "bias": rng.random() < 0.5,
            "residual": rng.random() < 0.5, "strided": rng.random() < 0.25}


# ------------------------------------------------------------------ inputs --

def _inputs(case, seed):
    """The tensors of a case: activations N(0, 1) with one channel in a hundred
    ten times larger, as hidden rows have; weights N(0, 1/K); incoming
    gradients N(0, 0.1^2)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    rows = case["rows"]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    def activations(n):
        x = torch.randn(rows, n, generator=gen, device=dev)
        big = torch.rand(n, generator=gen, device=dev) < 0.01
        return torch.where(big, x * 10.0, x).to(dt)

    s = {}
    if case["op"] == "norm":
        w = case["width"]
        s["x"] = (activations(w).float() + normal(rows, 1, dtype=torch.float32)).to(dt)
        s["weight"] = 1.0 + normal(w, scale=0.2, dtype=torch.float32)
        s["bias"] = normal(w, scale=0.1, dtype=torch.float32)
        if case["train"]:
            s["dy"] = normal(rows, w, scale=0.1)
    elif case["op"] == "gated":
        k, n = case["inputs"], case["inner"]
        s["x"] = activations(k)
        s["w_gate"] = normal(k, n, scale=k ** -0.5)
        s["w_up"] = normal(k, n, scale=k ** -0.5)
        if case["train"]:
            s["dh"] = normal(rows, n, scale=0.1)
    else:
        k, n = case["inputs"], case["outputs"]
        x = activations(k)
        if case["strided"]:
            wide = torch.zeros(rows, k + 64, dtype=dt, device=dev)
            wide[:, :k] = x
            x = wide[:, :k]
        s["x"] = x
        s["w"] = normal(k, n, scale=k ** -0.5)
        s["bias"] = normal(n, scale=0.5) if case["bias"] else None
        s["residual"] = activations(n) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(rows, n, scale=0.1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    from latent_projection_top_amd import block

    dt, rows, train = DTYPES[case["dtype"]], case["rows"], case["train"]
    dev = s["x"].device

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev)

    if case["op"] == "norm":
        w = case["width"]
        s["plan"] = block.NormPlan(rows, w, dtype=dt, param_dtype=torch.float32, eps=EPS)
        s["y"] = empty(rows, w)
        if train:
            s.update(mean=empty(rows, dtype=torch.float32), rstd=empty(rows, dtype=torch.float32),
                     dx=empty(rows, w), dweight=empty(w, dtype=torch.float32),
                     dbias=empty(w, dtype=torch.float32))
    elif case["op"] == "gated":
        k, n = case["inputs"], case["inner"]
        s["plan"] = block.GatedPlan(rows, k, n, activation=case["act"], dtype=dt, training=train)
        s["h"] = empty(rows, n)
        if train:
            s.update(d_gate=empty(rows, n), d_up=empty(rows, n), dx=empty(rows, k), dw_gate=empty(k, n),
                     dw_up=empty(k, n))
    else:
        k, n = case["inputs"], case["outputs"]
        s["plan"] = block.LinearPlan(rows, k, n, activation=case["act"], dtype=dt, training=train)
        s["y"] = empty(rows, n)
        if train:
            s.update(slope=empty(rows, n) if case["act"] != "none" else None, dx=empty(rows, k),
                     dw=empty(k, n), dbias=empty(n) if case["bias"] else None)
    s["workspace"] = s["plan"].new_workspace()
    return s


# --------------------------------------------------------------------- run --

def _act(name, z):
    """act(z) and act'(z), FP32."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return z * sg, sg * (1.0 + z * (1.0 - sg))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return (0.5 * z * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z))


def _plain_norm(s, train):
    dt = s["x"].dtype
    x, w, b = s["x"].float(), s["weight"], s["bias"]
    mean = x.mean(dim=1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(dim=1, keepdim=True) + EPS)
    xh = xc * rstd
    out = {"y": (xh * w + b).to(dt)}
    if train:
        dy = s["dy"].float()
        dyw = dy * w
        dx = rstd * (dyw - dyw.mean(dim=1, keepdim=True) - xh * (dyw * xh).mean(dim=1, keepdim=True))
        out.update(mean=mean[:, 0], rstd=rstd[:, 0], dx=dx.to(dt), dweight=(dy * xh).sum(dim=0),
                   dbias=dy.sum(dim=0))
    return out


def _plain_gated(s, act, train):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg, x @ wu
    a, da = _act(act, g)
    out = {"h": (a * u).to(dt)}
    if train:
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        out.update(dx=(dg @ wg.t() + du @ wu.t()).to(dt), dw_gate=(x.t() @ dg).to(dt),
                   dw_up=(x.t() @ du).to(dt))
    return out


def _plain_linear(s, act, train):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w
    if s["bias"] is not None:
        z = z + s["bias"].float()
    a, da = _act(act, z)
    out = {"y": (a if s["residual"] is None else a + s["residual"].float()).to(dt)}
    if train:
        dz = s["dy"].float() * da
        out.update(dx=(dz @ w.t()).to(dt), dw=(x.t() @ dz).to(dt))
        if s["bias"] is not None:
            out["dbias"] = dz.sum(dim=0).to(dt)
    return out


def _own_norm(s, train):
    from latent_projection_top_amd import block

    if not train:
        block.layer_norm(s["plan"], s["x"], s["weight"], s["bias"], s["y"])
        return {"y": s["y"]}
    block.layer_norm(s["plan"], s["x"], s["weight"], s["bias"], s["y"], mean=s["mean"], rstd=s["rstd"])
    block.layer_norm_backward(s["plan"], s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"],
                              s["dweight"], s["dbias"], s["workspace"])
    return {k: s[k] for k in ("y", "mean", "rstd", "dx", "dweight", "dbias")}


def _own_gated(s, train):
    from latent_projection_top_amd import block

    if not train:
        block.gated(s["plan"], s["x"], s["w_gate"], s["w_up"], s["h"], s["workspace"])
        return {"h": s["h"]}
    block.gated(s["plan"], s["x"], s["w_gate"], s["w_up"], s["h"], s["workspace"],
                d_gate=s["d_gate"], d_up=s["d_up"])
    block.gated_backward(s["plan"], s["dh"], s["x"], s["w_gate"], s["w_up"], s["d_gate"], s["d_up"],
                         s["dx"], s["dw_gate"], s["dw_up"], s["workspace"])
    return {k: s[k] for k in ("h", "dx", "dw_gate", "dw_up")}


def _own_linear(s, train):
    from latent_projection_top_amd import block

    if not train:
        block.linear(s["plan"], s["x"], s["w"], s["y"], s["workspace"], bias=s["bias"],
                     residual=s["residual"])
        return {"y": s["y"]}
    block.linear(s["plan"], s["x"], s["w"], s["y"], s["workspace"], bias=s["bias"],
                 residual=s["residual"], slope=s["slope"])
    block.linear_backward(s["plan"], s["dy"], s["x"], s["w"], s["slope"], s["dx"], s["dw"], s["dbias"],
                          s["workspace"])
    return {k: s[k] for k in ("y", "dx", "dw", "dbias") if s[k] is not None}


def run(state):
    case = state["case"]
    op, train = case["op"], case["train"]
    if op == "norm":
        return _own_norm(state, train) if own else _plain_norm(state, train)
    if op == "gated":
        return _own_gated(state, train) if own else _plain_gated(state, case["act"], train)
    return _own_linear(state, train) if own else _plain_linear(state, case["act"], train)


# ------------------------------------------------------------------- exact --

_EXACT_ACT = {
    "none": lambda z: z,
    "relu": torch.relu,
    "silu": torch.nn.functional.silu,
    "gelu": torch.nn.functional.gelu,
    "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
}


def exact(case, seed):
    """The same outputs in FP64: the forward definition, differentiated by
    torch's autograd."""
    s = {k: v.double() if v is not None else None for k, v in _inputs(case, seed).items()}
    train = case["train"]
    names = {"norm": ("x", "weight", "bias"), "gated": ("x", "w_gate", "w_up"),
             "linear": ("x", "w", "bias")}[case["op"]]
    leaves = [s[k] for k in names if s[k] is not None]
    for t in leaves:
        t.requires_grad_(train)
    if case["op"] == "norm":
        var, mean = torch.var_mean(s["x"], dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (s["x"] - mean[:, None]) * rstd[:, None] * s["weight"] + s["bias"]
        if not train:
            return {"y": y}
        dx, dw, db = torch.autograd.grad(y, leaves, s["dy"])
        return {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach(), "dx": dx, "dweight": dw,
                "dbias": db}
    act = _EXACT_ACT[case["act"]]
    if case["op"] == "gated":
        h = act(torch.mm(s["x"], s["w_gate"])) * torch.mm(s["x"], s["w_up"])
        if not train:
            return {"h": h}
        dx, dg, du = torch.autograd.grad(h, leaves, s["dh"])
        return {"h": h.detach(), "dx": dx, "dw_gate": dg, "dw_up": du}
    z = torch.mm(s["x"], s["w"])
    if s["bias"] is not None:
        z = z + s["bias"]
    y = act(z)
    if s["residual"] is not None:
        y = y + s["residual"]
    if not train:
        return {"y": y}
    grads = torch.autograd.grad(y, leaves, s["dy"])
    return dict(zip(("y", "dx", "dw", "dbias"), (y.detach(),) + grads))


# -------------------------------------------------------------------- work --

def work(case):
    """Bytes of every input read once and every output written once, and the
    operations of the products (or, for the norm, of its sums)."""
    e = DTYPES[case["dtype"]].itemsize
    rows, train = case["rows"], case["train"]
    if case["op"] == "norm":
        w = case["width"]
        n = rows * w
        if not train:
            return {"bytes": 2 * n * e + 8 * w, "flops": 8 * n}
        return {"bytes": 4 * n * e + 16 * w + 8 * rows, "flops": 24 * n}
    k = case["inputs"]
    if case["op"] == "gated":
        n = case["inner"]
        if not train:
            return {"bytes": e * (rows * k + 2 * k * n + rows * n), "flops": 4 * rows * k * n}
        return {"bytes": e * (2 * rows * k + 4 * k * n + 2 * rows * n), "flops": 12 * rows * k * n}
    n = case["outputs"]
    extra = e * (n * case["bias"] + rows * n * case["residual"])
    if not train:
        return {"bytes": e * (rows * k + k * n + rows * n) + extra, "flops": 2 * rows * k * n}
    return {"bytes": e * (2 * rows * k + 2 * k * n + 2 * rows * n + n * case["bias"]) + extra,
            "flops": 6 * rows * k * n}
