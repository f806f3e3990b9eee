"""The routed half of a latent MoE layer, as a program would run it.

RoutedRound    one serving round of up to `rows` rows on a rank that holds the
               experts first .. first + experts - 1: the route's choices sorted
               by expert, the experts' gated product and the product back in
               8-bit integers, and the results combined with the route's
               weights onto the residual stream.
RoutedTraining forward and backward pass of the same layer with 16-bit expert
               matrices: gather, one gated and one linear product per expert,
               combine, and every gradient (of the rows, the route's weights
               and the experts' matrices). It reads the experts' row counts
               back to the host between the sort and the products.

Weights and inputs are random; run it on an MI355X with
    python examples/routed_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from latent_projection_top_amd import block, experts, route  # noqa: E402

BF = torch.bfloat16


def matrices(count: int, inputs: int, inner: int, outputs: int, device="cuda", seed: int = 0) -> dict:
    """[count][K][N] BF16 matrices of the experts."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def matrix(k, n):
        return (torch.randn(count, k, n, generator=gen, device=device) * k ** -0.5).to(BF)

    return {"w_gate": matrix(inputs, inner), "w_up": matrix(inputs, inner), "w_down": matrix(inner, outputs)}


class RoutedRound:
    """Plans, packed weights, workspaces and buffers, made once."""

    def __init__(self, rows: int, topk: int, p: dict, first: int = 0):
        count, inputs, inner = p["w_gate"].shape
        outputs, choices = p["w_down"].shape[2], rows * topk
        self.sort = experts.SortPlan(rows, topk, count, first)
        self.gated = experts.Gated8Plan(choices, inputs, inner, experts=count, tokens=rows)
        self.down = experts.Linear8Plan(choices, inner, outputs, experts=count)
        self.combine = experts.CombinePlan(rows, topk, outputs)
        self.ws = [plan.new_workspace() for plan in (self.sort, self.gated, self.down)]
        gate, self.s_gate = experts.quantize(self.gated, p["w_gate"])
        up, self.s_up = experts.quantize(self.gated, p["w_up"])
        down, self.s_down = experts.quantize(self.down, p["w_down"])
        self.w_gated, self.w_down = experts.pack(self.gated, gate, up), experts.pack(self.down, down)

        def empty(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.offsets, self.token = empty(count + 1, dtype=torch.int32), empty(choices, dtype=torch.int32)
        self.place = empty(rows, topk, dtype=torch.int32)
        self.h, self.ys = empty(choices, inner), empty(choices, outputs)

    def __call__(self, x, ids, weights, y) -> None:
        """y += the experts' results for x [rows][inputs], in place. Nothing is
        allocated or read back: the call can be captured into a HIP graph."""
        rows = x.shape[0]
        n = rows * ids.shape[1]
        experts.sort(self.sort, ids, self.offsets, self.place, self.token, self.ws[0])
        experts.gated8(self.gated, x, self.w_gated, self.s_gate, self.s_up, self.h, self.ws[1], self.offsets,
                       self.token, rows=n)
        experts.linear8(self.down, self.h, self.w_down, self.s_down, self.ys, self.ws[2], self.offsets, rows=n)
        experts.combine(self.combine, self.ys, self.place, weights, y, residual=y, rows=rows)


class RoutedTraining:
    """Forward and backward pass of y = x_residual + sum_j w_j expert_j(x)."""

    def __init__(self, rows: int, topk: int, p: dict, first: int = 0):
        count, inputs, inner = p["w_gate"].shape
        outputs, choices = p["w_down"].shape[2], rows * topk
        self.sort = experts.SortPlan(rows, topk, count, first)
        self.into = experts.CombinePlan(rows, topk, inputs)
        self.back = experts.CombinePlan(rows, topk, outputs)
        self.gated = block.GatedPlan(choices, inputs, inner, training=True)
        self.down = block.LinearPlan(choices, inner, outputs, training=True)
        self.ws = [plan.new_workspace() for plan in (self.sort, self.gated, self.down)]

        def empty(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.offsets, self.token = empty(count + 1, dtype=torch.int32), empty(choices, dtype=torch.int32)
        self.place = empty(rows, topk, dtype=torch.int32)
        self.xs, self.dxs = empty(choices, inputs), empty(choices, inputs)
        self.h, self.d_gate, self.d_up, self.dh = (empty(choices, inner) for _ in range(4))
        self.ys, self.dys = empty(choices, outputs), empty(choices, outputs)
        self.y, self.dx = empty(rows, outputs), empty(rows, inputs)
        self.dweights = empty(rows, topk, dtype=torch.float32)
        self.grads = {k: torch.empty_like(v) for k, v in p.items()}

    def _ranges(self):
        return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(self.bounds, self.bounds[1:]))]

    def forward(self, x, ids, weights, residual, p: dict) -> torch.Tensor:
        experts.sort(self.sort, ids, self.offsets, self.place, self.token, self.ws[0])
        experts.gather(self.into, x, self.place, self.xs)
        self.bounds = self.offsets.tolist()
        for e, i in self._ranges():
            block.gated(self.gated, self.xs[i], p["w_gate"][e], p["w_up"][e], self.h[i], self.ws[1], self.d_gate[i],
                        self.d_up[i])
            block.linear(self.down, self.h[i], p["w_down"][e], self.ys[i], self.ws[2])
        experts.combine(self.back, self.ys, self.place, weights, self.y, residual=residual)
        return self.y

    def backward(self, dy, weights, p: dict) -> tuple[torch.Tensor, torch.Tensor, dict]:
        """dx, the gradient of the route's weights and of the matrices (the
        residual's is dy)."""
        g = self.grads
        experts.combine_backward(self.back, dy, self.ys, self.place, weights, self.dys, self.dweights)
        for e, i in self._ranges():
            block.linear_backward(self.down, self.dys[i], self.h[i], p["w_down"][e], None, self.dh[i],
                                  g["w_down"][e], None, self.ws[2])
            block.gated_backward(self.gated, self.dh[i], self.xs[i], p["w_gate"][e], p["w_up"][e], self.d_gate[i],
                                 self.d_up[i], self.dxs[i], g["w_gate"][e], g["w_up"][e], self.ws[1])
        experts.gather_backward(self.into, self.dxs, self.place, self.dx)
        return self.dx, self.dweights, g


def main() -> None:
    # one of 16 ranks: 56 experts; the latent rows of a decode round
    rows, topk, count, inner = 8, route.TOPK, 56, 512
    p = matrices(count, route.LATENT, inner, route.HIDDEN)
    serve = RoutedRound(rows, topk, p, first=112)
    x = torch.randn(rows, route.LATENT, device="cuda").to(BF)
    logits = torch.randn(rows, route.EXPERTS, device="cuda")
    plan = route.Plan(route.MODE_DECODE, rows)
    ids = torch.empty(rows, topk, dtype=torch.int32, device="cuda")
    weights = torch.empty(rows, topk, device="cuda")
    route.topk16(plan, logits, ids, weights)
    y = torch.randn(rows, route.HIDDEN, device="cuda").to(BF)
    before = y.clone()
    serve(x, ids, weights, y)
    torch.cuda.synchronize()
    print(f"serving round: {int(serve.offsets[-1])} of {rows * topk} choices are this rank's, "
          f"|change| / |y| = {float((y - before).float().norm() / before.float().norm()):.3f}")

    rows, topk, count = 256, 4, 8
    p = matrices(count, 512, 256, 512, seed=1)
    train = RoutedTraining(rows, topk, p)
    x, dy = (torch.randn(rows, 512, device="cuda").to(BF) for _ in range(2))
    ids = torch.rand(rows, count, device="cuda").topk(topk).indices.to(torch.int32)
    weights = torch.full((rows, topk), 1.0 / topk, device="cuda")
    train.forward(x, ids, weights, x, p)
    dx, dw, grads = train.backward(dy, weights, p)
    torch.cuda.synchronize()
    print(f"training step: |dx| {float(dx.float().norm()):.3f}, |dweights| {float(dw.norm()):.3f}, "
          f"|dw_gate| {float(grads['w_gate'].float().norm()):.3f}")


if __name__ == "__main__":
    main()
