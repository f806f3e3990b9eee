"""References and derived tolerances for the routed half of a layer.

Every reference is the operator's definition in FP64 (integers for the sort) on
the same inputs. With u the output type's unit roundoff and e = 2^-24 FP32's:

sums of n products in FP32 in any order are off by at most (n + 2) e times the
    sum of the terms' magnitudes.
8-bit products: the integers are decided exactly and their sum S is exact. What
    the kernel rounds is the row's scale, S as FP32, and two products, 4 e of
    the value; 6 e is allowed; the bias adds e of the sum. Activations as in
    blockkit (1.2 times the argument's error and 2^-19 of the value and the
    argument).
each output is rounded once: u of the value and half the smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

from tests import blockkit as kit

E, EVAL = kit.E, kit.EVAL
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def choices(rows, topk, total, seed=0, liking=0.5):
    """ids [rows][topk], distinct in a row, some experts more often than others."""
    gen = torch.Generator().manual_seed(seed)
    logits = torch.randn(rows, total, generator=gen) + liking * torch.randn(total, generator=gen)
    return torch.topk(logits, topk, dim=1).indices.to(torch.int32).cuda()


def sort_reference(ids, experts, first=0, capacity=None):
    """(offsets, place, token up to the last kept choice) as numpy."""
    flat = ids.cpu().numpy().astype(np.int64).ravel() - first
    kept = np.flatnonzero((flat >= 0) & (flat < experts))
    order = kept[np.argsort(flat[kept], kind="stable")]
    offsets = np.concatenate(([0], np.cumsum(np.bincount(flat[kept], minlength=experts))))
    place = np.full(flat.size, -1)
    place[order] = np.arange(order.size)
    token = order // ids.shape[1]
    return offsets, place.reshape(ids.shape), token if capacity is None else token[:capacity]


def sorted_choices(ids, experts, first=0):
    """The same on the device, token filled up with -1."""
    offsets, place, token = sort_reference(ids, experts, first)
    full = np.full(ids.numel(), -1)
    full[:token.size] = token

    def tensor(a):
        return torch.from_numpy(a.astype(np.int32)).cuda()

    return tensor(offsets), tensor(place), tensor(full)


class RowsCase:
    """Rows, sorted rows and gradients for gather and combine."""

    def __init__(self, rows, topk, width, total, experts, dtype, first=0, seed=0, stride=0, offset=0, whole=False,
                 capacity=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.topk, self.width, self.dtype = rows, topk, width, dtype
        self.ids = choices(rows, topk, total, seed)
        self.offsets, self.place, self.token = sorted_choices(self.ids, experts, first)
        cap = rows * topk if capacity is None else capacity
        self.capacity = cap

        def values(r):
            if whole:  # integers: every sum of products is exact in FP32
                v = torch.randint(-8, 9, (r, width), generator=gen, device="cuda").to(dtype)
            else:
                v = torch.randn(r, width, generator=gen, device="cuda").to(dtype)
            return kit.rows_like(v, dtype, stride, offset)[0]

        self.x, self.dy, self.residual = values(rows), values(rows), values(rows)
        self.ys, self.dxs = values(cap), values(cap)
        w = torch.rand(rows, topk, generator=gen, device="cuda") + 0.25
        self.weights = (w * 8).round() / 4 if whole else w / w.sum(1, keepdim=True)

    def live(self):
        """place with what is dropped or beyond the capacity as -1."""
        p = self.place.long()
        return torch.where((p >= 0) & (p < self.capacity), p, torch.full_like(p, -1))

    def collect(self, values, weights=None, residual=None):
        """(sum, bound) over a row's choices in FP64."""
        at = self.live()
        out = torch.zeros(self.rows, self.width, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        for j in range(self.topk):
            on = at[:, j] >= 0
            v = values[at[on, j]].double()
            if weights is not None:
                v = v * weights[on, j].double()[:, None]
            out[on] += v
            size[on] += v.abs()
        if residual is not None:
            out += residual.double()
            size += residual.double().abs()
        return out, (self.topk + 2) * E * size

    def spread(self, fill, weights=None, rows=None):
        """The sorted buffer after gather (of x) or combine_backward (of dy)."""
        out = fill.double().clone()
        at = self.live()
        for j in range(self.topk):
            on = at[:, j] >= 0
            v = rows[on].double()
            out[at[on, j]] = v if weights is None else v * weights[on, j].double()[:, None]
        return out

    def dweights(self):
        at = self.live()
        out = torch.zeros(self.rows, self.topk, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        for j in range(self.topk):
            on = at[:, j] >= 0
            terms = self.dy[on].double() * self.ys[at[on, j]].double()
            out[on, j], size[on, j] = terms.sum(1), terms.abs().sum(1)
        return out, (self.width + 2) * E * size


def quantised(x):
    """(integers, exact scale) of rows in FP64; rows that hold an infinity or
    NaN get a scale of NaN."""
    x = x.double()
    a = x.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(a)
    q = torch.round(127 * x / torch.where((a > 0) & ~bad, a, torch.ones_like(a)))
    return torch.where(bad, torch.zeros_like(q), q), torch.where(bad, torch.full_like(a, float("nan")), a / 127)


class ProductCase:
    """8-bit products, dense (offsets None) or by expert."""

    def __init__(self, planes, k, n, act, dtype, rows=0, counts=None, tokens=0, bias=False, residual=False, seed=0,
                 xs=0, ys=0, offset=0, spare=0, extreme=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.planes, self.k, self.n, self.act, self.dtype = planes, k, n, act, dtype
        self.counts = [rows] if counts is None else list(counts)
        self.experts = len(self.counts)
        self.kept = sum(self.counts)
        self.rows = self.kept + spare
        self.offsets = None
        if counts is not None:
            self.offsets = torch.tensor([0] + list(np.cumsum(self.counts)), dtype=torch.int32, device="cuda")
        self.tokens = tokens or self.rows
        self.token = None
        if tokens:
            self.token = torch.randint(0, tokens, (self.rows,), generator=gen, device="cuda", dtype=torch.int32)

        def normal(*shape, s=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * s).to(dtype)

        def integers():
            w = (torch.randn(self.experts, k, n, generator=gen, device="cuda") * 40).round().clamp(-128, 127)
            if extreme:
                w = torch.where(w < 0, torch.full_like(w, -128), torch.full_like(w, 127))
            return w.to(torch.int8)

        self.x = kit.rows_like(normal(self.tokens, k), dtype, xs, offset)[0]
        self.w = [integers() for _ in range(planes)]
        self.scale = [(torch.rand(self.experts, n, generator=gen, device="cuda") + 0.5) / (40 * k ** 0.5)
                      for _ in range(planes)]
        self.bias = normal(self.experts, n, s=0.5) if bias else None
        self.residual = kit.rows_like(normal(self.rows, n), dtype, ys, offset)[0] if residual else None

    def plan(self, experts):
        if self.planes == 1:
            return experts.Linear8Plan(max(self.rows, 1), self.k, self.n, experts=self.experts,
                                       tokens=max(self.tokens, 1), activation=self.act, dtype=self.dtype)
        return experts.Gated8Plan(max(self.rows, 1), self.k, self.n, experts=self.experts, tokens=max(self.tokens, 1),
                                  activation=self.act, dtype=self.dtype)

    def run(self, experts, plan, packed, out, workspace, **kw):
        if self.planes == 1:
            experts.linear8(plan, self.x, packed, self.scale[0], out, workspace, offsets=self.offsets,
                            token=self.token, bias=self.bias, residual=self.residual, **kw)
        else:
            experts.gated8(plan, self.x, packed, *self.scale, out, workspace, offsets=self.offsets,
                           token=self.token, **kw)

    def reference(self):
        """(value, bound) of the rows that some expert has."""
        q, s = quantised(self.x)
        out, bound = [], []
        start = 0
        for e, count in enumerate(self.counts):
            i = slice(start, start + count)
            start += count
            at = self.token[i].long() if self.token is not None else torch.arange(i.start, i.stop, device="cuda")
            z = [(q[at] @ w[e].double()) * s[at] * sc[e].double() for w, sc in zip(self.w, self.scale)]
            err = [6 * E * v.abs() for v in z]
            if self.planes == 1:
                v, ev = z[0], err[0]
                if self.bias is not None:
                    v = v + self.bias[e].double()
                    ev = ev + 2 * E * v.abs()
                a = kit.ACT[self.act](v)
                ea = ev if self.act == "none" else 1.2 * ev + EVAL * (a.abs() + v.abs())
                if self.residual is not None:
                    a = a + self.residual[i].double()
                out.append(a)
                bound.append(ea + 2 * E * a.abs())
            else:
                a = kit.ACT[self.act](z[0])
                ea = 1.2 * err[0] + EVAL * (a.abs() + z[0].abs())
                out.append(a * z[1])
                bound.append(ea * (z[1].abs() + err[1]) + a.abs() * err[1] + 2 * E * (a * z[1]).abs())
        return torch.cat(out), torch.cat(bound)

    def check(self, experts, what, fill=7.0, ys=0, offset=0):
        """One call; rows behind the last expert's keep `fill`. Returns y."""
        plan = self.plan(experts)
        packed = experts.pack(plan, *self.w)
        y, _ = kit.rows_like(torch.full((self.rows, self.n), fill, device="cuda").to(self.dtype), self.dtype, ys,
                             offset)
        self.run(experts, plan, packed, y, plan.new_workspace())
        torch.cuda.synchronize()
        ref, bound = self.reference()
        kit.check(y[:self.kept], ref, bound, None, self.dtype, what)
        assert (y[self.kept:].float() == fill).all(), what
        return y
