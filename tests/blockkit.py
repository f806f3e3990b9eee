"""References and derived tolerances for the layer's operators.

Every reference is the operator's definition in FP64 on the same inputs. Two
bounds are checked per output:

worst case, element by element. u is the output type's unit roundoff (BF16
    2^-8, F16 2^-11, FP32 2^-24), e = 2^-24 FP32's, `tiny` half the spacing of
    the type's subnormals. A sum of K products in any FP32 order is off by at
    most (K + 8) e times the sum of the terms' magnitudes (K additions, and
    the product's own rounding); an activation and its derivative are Lipschitz with constants
    below 1.2 and 1.0 and evaluated to 2^-19; each rounding to the output
    type adds u of the value and `tiny`.

root mean square. The roundings to the output type are independent, each with
    an RMS of at most u / sqrt(3) of the value it rounds. A backward product
    goes through three of them (the saved derivative, its product with the
    incoming gradient, the result), which gives at most u times
    sqrt(sum of the squared terms + result^2); 1.5 u is allowed. This one
    finds a lost or doubled term, which is 1/sqrt(K) of the result.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E = 2.0 ** -24
EVAL = 2.0 ** -19

ACT = {
    "none": lambda z: z,
    "relu": lambda z: torch.clamp(z, min=0),
    "silu": lambda z: z / (1 + torch.exp(-z)),
    "gelu": lambda z: 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0))),
    "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))),
}


def slope(act, z):
    """act'(z), written out."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2.0))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def slope_error(act, z, dz):
    """How far act' can be off when z is off by at most dz."""
    if act == "none":
        return torch.zeros_like(z)
    if act == "relu":
        return (z.abs() <= dz).double()
    return dz + EVAL


def check(got, ref, bound, rms_scale, dtype, what):
    """`bound` before the output's own rounding; rms_scale as described above
    (None: no RMS check)."""
    assert got.dtype == dtype, (what, got.dtype)
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: {int((~torch.isfinite(g)).sum())} values not finite"
    err = (g - ref).abs()
    u = UNIT[dtype]
    allowed = bound * (1 + u) + u * ref.abs() + TINY[dtype]
    over = err > allowed
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} outside the bound, worst "
                            f"{float((err / allowed).max()):.3g} of it, first at {over.nonzero()[0].tolist()}")
    if rms_scale is not None:
        r = float(err.square().mean().sqrt())
        s = float(rms_scale.square().mean().sqrt())
        assert r <= 1.5 * u * s + 2 * TINY[dtype], f"{what}: rms error {r:.3g}, scale {s:.3g}, unit {u:.3g}"


def product(a, b):
    """Exact a b, the bound of its FP32 sums and the root of its squared terms."""
    k = a.shape[1]
    return a @ b, (k + 8) * E * (a.abs() @ b.abs()), (a.square() @ b.square()).sqrt()


def rows_like(values, dtype, stride=0, offset=0, fill=float("nan")):
    """`values` as a matrix of rows of the given stride inside a larger buffer
    of `fill`, `offset` elements into it."""
    rows, n = values.shape
    stride = stride or n
    buf = torch.full((offset + rows * stride + 8,), fill, dtype=dtype, device=values.device)
    view = buf[offset:offset + rows * stride].view(rows, stride)[:, :n] if rows else buf[:0].view(0, n)
    view.copy_(values)
    return view, buf


class GatedCase:
    def __init__(self, rows, k, n, act, dtype, seed=0, xs=0, hs=0, offset=0, scale=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, s=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * s).to(dtype)

        self.rows, self.k, self.n, self.act, self.dtype = rows, k, n, act, dtype
        self.x, _ = rows_like(normal(rows, k, s=scale), dtype, xs, offset)
        self.dh, _ = rows_like(normal(rows, n), dtype, hs, offset)
        self.wg = self._weight(normal(k, n, s=k ** -0.5), offset)
        self.wu = self._weight(normal(k, n, s=k ** -0.5), offset)

    def _weight(self, w, offset):
        if not offset:
            return w
        buf = torch.empty(offset + w.numel(), dtype=w.dtype, device="cuda")
        buf[offset:].copy_(w.flatten())
        return buf[offset:].view_as(w)

    def reference(self):
        x, wg, wu, dh = (t.double() for t in (self.x, self.wg, self.wu, self.dh))
        u = UNIT[self.dtype]
        tiny = TINY[self.dtype]
        g, eg, _ = product(x, wg)
        up, eu, _ = product(x, wu)
        a, s = ACT[self.act](g), slope(self.act, g)
        h = a * up
        ea = 1.2 * eg + EVAL * (a.abs() + g.abs())
        out = {"h": (h, ea * (up.abs() + eu) + a.abs() * eu, h.abs() + a.abs() * u)}
        es = slope_error(self.act, g, eg)
        dgl, dul = s * up, a  # the saved derivatives
        edg = es * (up.abs() + eu) + s.abs() * eu
        out["d_gate"] = (dgl, edg, None)
        out["d_up"] = (dul, ea, None)
        dg, du = dh * dgl, dh * dul
        # the derivative rounded once, then its product with dh
        fdg = dh.abs() * (edg * (1 + u) + u * dgl.abs() + tiny) * (1 + u) + u * dg.abs() + tiny
        fdu = dh.abs() * (ea * (1 + u) + u * dul.abs() + tiny) * (1 + u) + u * du.abs() + tiny
        n = self.n
        dx = dg @ wg.t() + du @ wu.t()
        terms = dg.abs() @ wg.abs().t() + du.abs() @ wu.abs().t()
        sq = dg.square() @ wg.square().t() + du.square() @ wu.square().t()
        out["dx"] = (dx, (fdg @ wg.abs().t() + fdu @ wu.abs().t()) * (1 + (2 * n + 8) * E) + (2 * n + 8) * E * terms,
                     (sq + dx.square()).sqrt())
        r = self.rows
        for name, d, f in (("dw_gate", dg, fdg), ("dw_up", du, fdu)):
            dw = x.t() @ d
            out[name] = (dw, x.abs().t() @ f * (1 + (r + 8) * E) + (r + 8) * E * (x.abs().t() @ d.abs()),
                         (x.square().t() @ d.square() + dw.square()).sqrt())
        if self.act == "relu":  # a sign at the edge is allowed either way: no RMS statement
            out = {k: (a, b, None if k[0] == "d" else c) for k, (a, b, c) in out.items()}
        return out


class LinearCase:
    def __init__(self, rows, k, n, act, dtype, bias=True, residual=True, seed=0, xs=0, ys=0, offset=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, s=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * s).to(dtype)

        self.rows, self.k, self.n, self.act, self.dtype = rows, k, n, act, dtype
        self.x, _ = rows_like(normal(rows, k), dtype, xs, offset)
        self.dy, _ = rows_like(normal(rows, n), dtype, ys, offset)
        self.w = GatedCase._weight(self, normal(k, n, s=k ** -0.5), offset)
        self.bias = normal(n, s=0.5) if bias else None
        self.residual = rows_like(normal(rows, n), dtype, ys, offset)[0] if residual else None

    def reference(self):
        x, w, dy = self.x.double(), self.w.double(), self.dy.double()
        u, tiny = UNIT[self.dtype], TINY[self.dtype]
        z, ez, _ = product(x, w)
        if self.bias is not None:
            z = z + self.bias.double()
            ez = ez + 2 * E * z.abs()
        a, s = ACT[self.act](z), slope(self.act, z)
        ea = ez if self.act == "none" else 1.2 * ez + EVAL * (a.abs() + z.abs())
        y = a if self.residual is None else a + self.residual.double()
        out = {"y": (y, ea + 2 * E * y.abs(), y.abs())}
        es = slope_error(self.act, z, ez)
        out["slope"] = (s, es, None)
        dz = dy * s
        if self.act == "none":
            f = torch.zeros_like(dz)
        else:
            f = dy.abs() * (es * (1 + u) + u * s.abs() + tiny) * (1 + u) + u * dz.abs() + tiny
        n, r = self.n, self.rows
        dx = dz @ w.t()
        out["dx"] = (dx, f @ w.abs().t() * (1 + (n + 8) * E) + (n + 8) * E * (dz.abs() @ w.abs().t()),
                     (dz.square() @ w.square().t() + dx.square()).sqrt())
        dw = x.t() @ dz
        out["dw"] = (dw, x.abs().t() @ f * (1 + (r + 8) * E) + (r + 8) * E * (x.abs().t() @ dz.abs()),
                     (x.square().t() @ dz.square() + dw.square()).sqrt())
        db = dz.sum(0)
        out["dbias"] = (db, f.sum(0) * (1 + (r + 8) * E) + (r + 8) * E * dz.abs().sum(0),
                        (dz.square().sum(0) + db.square()).sqrt())
        if self.act == "relu":
            out = {k: (a, b, None if k[0] in "ds" else c) for k, (a, b, c) in out.items()}
        return out


class NormCase:
    def __init__(self, rows, width, dtype, param_dtype=torch.float32, weight=True, bias=True, seed=0,
                 stride=0, offset=0, shift=1.0, eps=1e-5):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, s=1.0, d=dtype):
            return (torch.randn(*shape, generator=gen, device="cuda") * s).to(d)

        self.rows, self.width, self.dtype, self.pdt, self.eps = rows, width, dtype, param_dtype, eps
        x = normal(rows, width, d=torch.float32) + shift * normal(rows, 1, d=torch.float32)
        self.x, _ = rows_like(x.to(dtype), dtype, stride, offset)
        self.dy, _ = rows_like(normal(rows, width), dtype, stride, offset)
        self.weight = (1 + normal(width, s=0.3, d=torch.float32)).to(param_dtype) if weight else None
        self.bias = normal(width, s=0.3, d=param_dtype) if bias else None

    def reference(self):
        x, dy, n = self.x.double(), self.dy.double(), self.width
        w = self.weight.double() if self.weight is not None else torch.ones(n, device="cuda", dtype=torch.float64)
        b = self.bias.double() if self.bias is not None else torch.zeros(n, device="cuda", dtype=torch.float64)
        k = (n + 16) * E
        mean = x.mean(1, keepdim=True)
        emean = k * x.abs().mean(1, keepdim=True)
        xc = x - mean
        var = xc.square().mean(1, keepdim=True)
        rstd = (var + self.eps).rsqrt()
        # the centred squares: relative (n + 16) e, and the mean's error enters
        # through |xc| (2 |xc| emean) and its square
        evar = k * var + 2 * emean * xc.abs().mean(1, keepdim=True) * k + emean.square() + 4 * E * var
        # xc itself is rounded, relative to |xc| (covered by k) and its inputs
        rel = 0.5 * evar * rstd.square() + 8 * E
        erstd = rel * rstd * (1 + rel) * 1.5
        xh = xc * rstd
        exh = (emean + 2 * E * xc.abs()) * (rstd + erstd) + xc.abs() * erstd + 4 * E * xh.abs()
        y = xh * w + b
        out = {"y": (y, w.abs() * exh + 4 * E * ((xh * w).abs() + b.abs()), None),
               "mean": (mean[:, 0], emean[:, 0], None), "rstd": (rstd[:, 0], erstd[:, 0], None)}
        g = w * dy
        c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
        e1 = k * g.abs().mean(1, keepdim=True)
        e2 = (g.abs() * exh).mean(1, keepdim=True) + k * (g * xh).abs().mean(1, keepdim=True)
        inner = g - c1 - xh * c2
        size = g.abs() + c1.abs() + (xh * c2).abs()
        einner = e1 + (xh.abs() + exh) * e2 + c2.abs() * exh + 8 * E * size
        out["dx"] = (rstd * inner, (rstd + erstd) * einner + erstd * inner.abs() + 4 * E * (rstd * inner).abs(), None)
        r = (self.rows + 16) * E
        out["dweight"] = ((dy * xh).sum(0), (dy.abs() * exh).sum(0) + r * (dy * xh).abs().sum(0), None)
        out["dbias"] = (dy.sum(0), r * dy.abs().sum(0), None)
        return out
